// sparse.cu -- attention over the key blocks listed for each query block.
//
//   O_i = softmax(Q_i K_L^T / sqrt(d)) V_L,   L = the keys of the 128-token
//   blocks lists[b, h, i, 0 .. counts[b, h, i] - 1];  an empty list gives 0.
//
// The arithmetic is that of the dense kernels (attention.cu), step for step in
// list order, so a list of all blocks in ascending order gives the dense call's
// bits.  QUANT: exact int32 S, dequantized; P8 = e4m3(p * 448) through shared
// memory; O += P8 V8.  BF16: S and O += P V with kind::f16, P in tensor memory
// (D = 64: beside S, D = 128: over S).
//
// Work.  One item is one query block (128 rows) with its list.  A persistent CTA
// per SM runs two lanes, each with Q, K, V, S, P and O of its own: lists differ
// in content and length, so neighbouring query blocks share no tiles, and a lane
// that ends its item goes on to the next without waiting for the other.  Items
// are handed out by a counter (the first two per CTA by position), which evens
// out lists of different lengths.
// Warp roles (12 warps, registers re-split as in attention.cu):
//   warps 0, 2   producer of lane 0, 1: fetches the items, loads Q, K, V by TMA;
//   warps 1, 3   the MMA-issuing thread of lane 0, 1 (warp 1 owns tensor memory);
//   warps 4-7, 8-11   softmax of lane 0, 1, one thread per query row, and the
//                item's epilogue.
// One thread per lane and task, each in blocking waits: one thread polling for
// both lanes added its poll to every step of the BF16 kernel, whose steps are a
// chain S -> P -> PV -> S (a quarter longer).
// Where P has a place of its own (QUANT: shared memory; BF16 with D = 64: the
// tensor memory that the shorter O leaves) the next S is formed while this one is
// in the softmax: a step takes 10% less (BF16, D = 64).  Elsewhere the next S waits
// until PV has read P in its columns (2.3 to 3%; formed in two halves, the one beside P
// ahead of the wait, 9% more: products of half the width).
// The two softmax warpgroups take turns on the exponential phase (an mbarrier
// token, strictly alternating; a lane that has run out of items gives its turns
// away), except in BF16 with D = 64.  Without turns a step of both lanes takes 12%
// (QUANT, D = 64), 15% (QUANT, D = 128) and 11% (BF16, D = 128) longer, but 11% less in
// BF16 with D = 64, where neither the MMAs nor the packing of P hold the other lane up.
// K and V tiles have rings of their own: K_j is free once Q K_j^T is done, a
// whole step before V_j.
// What bounds it: the exponentials' schedule (56% of the SFU rate INT8/FP8, 64% BF16 with
// D = 64), in BF16 with D = 128 the chain of a lane, and the power limit.  Clocks for a step
// of both lanes, items' ends and tail included (time x SM clock x SMs / half the steps; the
// dense kernels by the same reckoning in brackets): INT8/FP8 3,960 (3,470) at D = 128, 4,110
// (3,750) at D = 64; BF16 4,640 (4,190) and 3,600 (3,710).  2,048 of them are the
// exponentials.  Measured, the prepass included: 1 x 40 x 75600 x 128, 59 of 591 blocks a
// row, INT8/FP8 10.5 to 11.0 ms; BF16 1 x 30 x 17776 x 64, 28 of 139 blocks, 720 to 770 us;
// 1 x 12 x 32760 x 128, lists of up to 64 of 256 blocks, 1.02 to 1.04 ms.
//
// A listed index outside [0, ceil(N/128)) adds nothing to its row and a count
// outside [0, width] is clamped to it; both are recorded in the status word and
// read no memory outside the tensors.  Waits are bounded; a softmax warp gives one up as a
// whole, for its tensor-memory accesses and votes need all lanes.
#include <cuda_bf16.h>
#include <algorithm>
#include <cstdint>

#include "attn_tiles.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace sage {

namespace {

struct SparseParams {
  const float* q_scale;
  const float* k_scale;
  const float* v_scale;
  __nv_bfloat16* o;       // [BH, N, D]
  const int* lists;       // [BH, nT, width]
  const int* counts;      // [BH, nT]
  uint32_t* status;
  unsigned* next;         // items handed out after the first two per CTA
  int N, nT, Npad, width, BH, items;
  long long timeout;
  int dbg_flags;          // bit 0: the MMA threads first wait on a barrier nobody arrives on
  int q_per_token;
  int wide;               // o is 32-byte aligned: 32-byte stores
};

// One item as its consumers see it.  steps -1: no more items.
struct Item {
  int bh, qb, steps, bad;           // bad: the count was out of range
};

template <int D, bool QUANT>
struct SparseCfg {
  using C = Cfg<D, QUANT>;
  static constexpr int TILE_BYTES = C::TILE_BYTES;
  static constexpr bool AHEAD = QUANT || D == 64;    // the next S before this step's PV
  static constexpr bool TURNS = QUANT || D == 128;   // the lanes take turns on the exponentials
  // K and V slots of each lane (without AHEAD a second K slot has no use, QK_j+1 follows PV_j)
  static constexpr int KS = AHEAD ? 2 : 1;
  static constexpr int VS = KS;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE_BYTES;                    // [2][KS]
  static constexpr int OFF_V = OFF_K + 2 * KS * TILE_BYTES;       // [2][VS]
  static constexpr int OFF_P = OFF_V + 2 * VS * TILE_BYTES;       // [2], QUANT
  static constexpr int OFF_LANE = OFF_P + 2 * C::P_BYTES;
  static constexpr int LANE_BYTES = 1280;
  static constexpr int SMEM_BYTES = OFF_LANE + 2 * LANE_BYTES + 64 + 1024;   // + 1 KB alignment slack
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// What the threads of one lane share.
template <int KS, int VS>
struct Lane {
  float v_scale[2][128];            // QUANT: of the heads of the items with steps, alternating
  Item item[2];
  uint64_t q_full, q_empty;
  uint64_t k_full[KS], k_empty[KS];
  uint64_t v_full[VS], v_empty[VS];
  uint64_t s_full;                  // S written (MMA commit)
  uint64_t s_free;                  // AHEAD: S read into registers
  uint64_t p_full;                  // P written, O rescaled
  uint64_t o_ready;                 // AHEAD: a PV done; else the item's last PV done
  uint64_t tok;                     // this lane's turn on the exponential phase
  uint64_t p_read;                  // not AHEAD: a PV done, P's columns are free for the next S
  uint64_t item_full[2], item_empty[2];
};

// 32 bytes (32-byte aligned): rows lie 2 D bytes apart, so a warp's store touches 32
// lines whatever its width, and wider stores mean fewer of them.
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

template <int D, bool QUANT>
__global__ void __launch_bounds__(kThreads, 1)
    sparse_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const SparseParams prm) {
  using C = Cfg<D, QUANT>;
  using SC = SparseCfg<D, QUANT>;
  constexpr int KS = SC::KS, VS = SC::VS, TILE = SC::TILE_BYTES;
  constexpr bool AHEAD = SC::AHEAD, TURNS = SC::TURNS;
  using L = Lane<KS, VS>;
  static_assert(sizeof(L) <= SC::LANE_BYTES, "lane struct");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto lane_at = [&](int t) -> L& { return *reinterpret_cast<L*>(smem + SC::OFF_LANE + t * SC::LANE_BYTES); };
  uint64_t* mma_done = reinterpret_cast<uint64_t*>(smem + SC::OFF_LANE + 2 * SC::LANE_BYTES);   // [2]
  uint64_t* never = mma_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* idle = abort_flag + 1;                                 // [2] the lane has no more items

  const int warp = threadIdx.x >> 5, lane_id = threadIdx.x & 31;
  const int N = prm.N, nT = prm.nT;
  const long long limit = prm.timeout;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      L& b = lane_at(t);
      mbar_init(&b.q_full, 1);
      mbar_init(&b.q_empty, 1);
      for (int s = 0; s < KS; ++s) {
        mbar_init(&b.k_full[s], 1);
        mbar_init(&b.k_empty[s], 1);
      }
      for (int s = 0; s < VS; ++s) {
        mbar_init(&b.v_full[s], 1);
        mbar_init(&b.v_empty[s], 1);
      }
      mbar_init(&b.s_full, 1);
      mbar_init(&b.s_free, 128);
      mbar_init(&b.p_full, 128);
      mbar_init(&b.o_ready, 1);
      mbar_init(&b.p_read, 1);
      mbar_init(&b.tok, 128);
      for (int s = 0; s < 2; ++s) {
        mbar_init(&b.item_full[s], 1);
        mbar_init(&b.item_empty[s], 129);              // the softmax warpgroup and the MMA thread
      }
      mbar_init(&mma_done[t], 1);
      idle[t] = 0;
    }
    mbar_init(never, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    regs_release<C::REGS_LOW>();
    const int t = warp >> 1;
    L& b = lane_at(t);
    if ((warp & 1) == 0 && lane_id == 0) {
      // ---------------------------------------------------------- producer of lane t
      if (t == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
      }
      int nq = 0, nk = 0, nv = 0;                      // Q, K, V tiles issued
      // Waits for the slot of the n-th tile of a ring and arms its barrier.
      auto slot_free = [&](int n, int slots, uint64_t* full, uint64_t* empty) {
        const int s = n % slots;
        if (n >= slots && !mbar_wait(&empty[s], ((n / slots) - 1) & 1, abort_flag, limit)) return false;
        mbar_arrive_expect_tx(&full[s], TILE);
        return true;
      };
      auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* full, int bh, int blk, bool v) {
        if constexpr (QUANT) {
          if (v)
            tma_load_2d(dst, map, full, blk * 128, bh * D);
          else
            tma_load_2d(dst, map, full, 0, bh * prm.Npad + blk * 128);
        } else {
#pragma unroll
          for (int a = 0; a < D / 64; ++a) tma_load_3d(dst + a * 16384, map, full, a * 64, blk * 128, bh);
        }
      };
      uint8_t* q_dst = smem + SC::OFF_Q + t * TILE;
      uint8_t* k_dst = smem + SC::OFF_K + t * KS * TILE;
      uint8_t* v_dst = smem + SC::OFF_V + t * VS * TILE;
      const bool more = prm.items > 2 * (int)gridDim.x;
      int id = t * (int)gridDim.x + (int)blockIdx.x;
      for (int n = 0;; ++n) {
        Item it{0, 0, -1, 0};
        if (id < prm.items && SAGE_DCHECK(id, prm.items, kSiteSparseList)) {
          it.bh = id / nT;
          it.qb = id - it.bh * nT;
          const int raw = __ldg(prm.counts + id);
          it.steps = max(0, min(raw, prm.width));
          it.bad = it.steps != raw;
        }
        if (n >= 2 && !mbar_wait(&b.item_empty[n & 1], ((n >> 1) - 1) & 1, abort_flag, limit)) break;
        b.item[n & 1] = it;
        mbar_arrive(&b.item_full[n & 1]);
        const int c = it.steps;
        if (c < 0) break;
        int next = prm.items;                          // without the counter: nothing behind the first two
        if (c == 0) {
          if (more) next = 2 * (int)gridDim.x + (int)atomicAdd(prm.next, 1u);
          id = next;
          continue;
        }
        const long long off = (long long)id * prm.width;
        auto listed = [&](int j, int next) {           // the block `next` places behind j (j + next may pass 2^31)
          return c - j > next && SAGE_DCHECK(off + j + next, (long long)prm.items * prm.width, kSiteSparseList) ? __ldg(prm.lists + off + j + next) : 0;
        };
        // An index outside the sequence: the softmax masks its scores, and V must be zeros
        // (0 * inf would not be 0), which are read behind the end of the tensor.
        auto safe = [&](int x, int otherwise) { return (unsigned)x < (unsigned)nT ? x : otherwise; };
        auto put_k = [&](int x) {
          if (!slot_free(nk, KS, b.k_full, b.k_empty)) return false;
          load(&tmK, k_dst + (nk % KS) * TILE, &b.k_full[nk % KS], it.bh, safe(x, 0), false);
          ++nk;
          return true;
        };
        auto put_v = [&](int x) {
          if (!slot_free(nv, VS, b.v_full, b.v_empty)) return false;
          load(&tmV, v_dst + (nv % VS) * TILE, &b.v_full[nv % VS], it.bh, safe(x, nT), true);
          ++nv;
          return true;
        };
        int cur = listed(0, 0), ahead = listed(0, 1);
        if (!slot_free(nq, 1, &b.q_full, &b.q_empty)) break;
        load(&tmQ, q_dst, &b.q_full, it.bh, it.qb, false);
        ++nq;
        bool go = put_k(cur);
        for (int j = 0; j < c && go; ++j) {
          const int after = listed(j, 2);             // read a step before its load
          // the next item is asked for a few steps before this one's last load: early
          // enough to hide the counter's latency, late enough not to hoard work
          if (more && j == max(0, c - 3)) next = 2 * (int)gridDim.x + (int)atomicAdd(prm.next, 1u);
          // with one K slot, K(j+1) waits for this step's QK, and V(j) must not wait with it
          if (KS > 1 && j + 1 < c) go = put_k(ahead);
          go = go && put_v(cur);
          if (KS == 1 && j + 1 < c) go = go && put_k(ahead);
          cur = ahead;
          ahead = after;
        }
        if (!go) break;
        id = next;
      }
      // drain: every load this thread issued must land before the CTA exits (given its own, long limit:
      // a caller's may be shorter than a load takes)
      volatile int no_abort = 0;
      if (nq > 0) mbar_wait(&b.q_full, (nq - 1) & 1, &no_abort, kDefaultTimeoutCycles);
      for (int i = max(0, nk - KS); i < nk; ++i) mbar_wait(&b.k_full[i % KS], (i / KS) & 1, &no_abort, kDefaultTimeoutCycles);
      for (int i = max(0, nv - VS); i < nv; ++i) mbar_wait(&b.v_full[i % VS], (i / VS) & 1, &no_abort, kDefaultTimeoutCycles);
    } else if ((warp & 1) == 1 && lane_id == 0) {
      // ---------------------------------------------------------- MMA issuer of lane t
      const uint32_t q_s = smem_u32(smem + SC::OFF_Q + t * TILE);
      const uint32_t k_s = smem_u32(smem + SC::OFF_K + t * KS * TILE);
      const uint32_t v_s = smem_u32(smem + SC::OFF_V + t * VS * TILE);
      const uint32_t p_s = smem_u32(smem + SC::OFF_P + t * C::P_BYTES);
      const uint32_t d_s = tmem + t * 128, d_o = tmem + 256 + t * D;
      const uint32_t d_p = AHEAD ? tmem + 384 + t * 64 : d_s;   // BF16
      bool ok = true;
      if (prm.dbg_flags & 1) ok = mbar_wait(never, 0, abort_flag, limit);
      int qk = 0, pv = 0, nq = 0;                      // steps issued, Q tiles taken, over all items
      auto issue_s = [&](bool last_of_item) {          // S = Q K^T of step qk
        if (!mbar_wait(&b.k_full[qk % KS], (qk / KS) & 1, abort_flag, limit)) return false;
        tc_fence_after();
        issue_qk<D, QUANT>(d_s, q_s, k_s + (qk % KS) * TILE);
        mma_commit(&b.s_full);
        mma_commit(&b.k_empty[qk % KS]);
        if (last_of_item) mma_commit(&b.q_empty);
        ++qk;
        return true;
      };
      for (int n = 0; ok; ++n) {
        if (!(ok = mbar_wait(&b.item_full[n & 1], (n >> 1) & 1, abort_flag, limit))) break;
        const int c = *const_cast<volatile int*>(&b.item[n & 1].steps);
        mbar_arrive(&b.item_empty[n & 1]);
        if (c < 0) break;
        if (c == 0) continue;
        ok = mbar_wait(&b.q_full, nq & 1, abort_flag, limit);
        ++nq;
        // the S columns are free: the softmax of the previous item's last S comes before its last
        // PV, which is issued (not AHEAD: done)
        ok = ok && issue_s(c == 1);
        for (int j = 0; j < c && ok; ++j) {
          // AHEAD: the next S as soon as this one is in the softmax warps' registers
          if (AHEAD && j + 1 < c) ok = mbar_wait(&b.s_free, (qk - 1) & 1, abort_flag, limit) && issue_s(j + 2 == c);
          ok = ok && mbar_wait(&b.p_full, pv & 1, abort_flag, limit) &&
               mbar_wait(&b.v_full[pv % VS], (pv / VS) & 1, abort_flag, limit);
          // (an item's first PV overwrites O: p_full comes behind the previous epilogue's reads)
          if (!ok) break;
          tc_fence_after();
          if constexpr (QUANT)
            issue_pv_quant<D>(d_o, p_s, v_s + (pv % VS) * TILE, j > 0 ? 1u : 0u);
          else
            issue_pv_bf16<D>(d_o, d_p, v_s + (pv % VS) * TILE, j > 0 ? 1u : 0u);
          if (AHEAD || j + 1 == c) mma_commit(&b.o_ready);
          mma_commit(&b.v_empty[pv % VS]);
          if constexpr (!AHEAD) {
            // P lies over S, and a product into other columns has no order behind this one (tcgen05
            // gives one only to products that share accumulator and shape): the next S, of the next
            // item too, waits until P is read
            mma_commit(&b.p_read);
            ok = mbar_wait(&b.p_read, pv & 1, abort_flag, limit) && (j + 1 == c || issue_s(j + 2 == c));
          }
          ++pv;
        }
      }
      // drain: every MMA issued must complete before TMEM is released
      mma_commit(&mma_done[t]);
      volatile int no_abort = 0;
      mbar_wait(&mma_done[t], 0, &no_abort, kDefaultTimeoutCycles);
    }
  } else {
    regs_claim<C::REGS_HIGH>();
    // ------------------------------------------------------------ softmax of lane t
    const int t = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane_id;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + t * 128;
    const uint32_t tO = tmem + lane_off + 256 + t * D;
    const uint32_t tP = AHEAD ? tmem + lane_off + 384 + t * 64 : tS;   // BF16
    L& b = lane_at(t);
    uint64_t* give = &lane_at(1 - t).tok;
    int step = 0, done = 0;                              // steps (and turns), items with steps so far
    bool ok = true;
    if (TURNS && t == 1) mbar_arrive(give);              // lane 0 has the first turn
    // int32 S + 0x4B400000 read as a float is 12582912 + S exactly (|S| <= 127*127*128 < 2^22)
    constexpr uint32_t kMagicBits = 0x4B400000u;
    constexpr float kMagic = 12582912.0f;
    // QUANT: p is produced already multiplied by the P scale 448 (2^(s - m + log2 448)),
    // so l accumulates 448 * sum(p) and the epilogue divides by it directly.
    constexpr float kLog2PScale = QUANT ? 8.807354922057604f : 0.f;

    // The item at hand and what its first step needs, read while the previous item is stored.
    Item it{0, 0, -1, 0};
    int blk_next = 0, blk_after = 0;                     // the next two blocks of its list
    float qs = 0.f, ks_next = 0.f, vsc = 0.f;            // QUANT: this row's Q scale, the next block's K scale, a V scale
    auto listed = [&](int j, int next) {                 // the block `next` places behind j (j + next may pass 2^31)
      const long long at = ((long long)it.bh * nT + it.qb) * prm.width + j + next;
      return it.steps - j > next && SAGE_DCHECK(at, (long long)prm.items * prm.width, kSiteSparseList) ? __ldg(prm.lists + at) : 0;
    };
    auto scale_of = [&](int x) {
      const long long ki = (long long)it.bh * nT + ((unsigned)x < (unsigned)nT ? x : 0);
      return QUANT && SAGE_DCHECK(ki, (long long)prm.items, kSiteSparseScale) ? __ldg(prm.k_scale + ki) : 0.f;
    };
    auto take_item = [&](int n) {
      if (!mbar_wait_warp(&b.item_full[n & 1], (n >> 1) & 1, abort_flag, limit)) return false;
      const volatile Item* vi = &b.item[n & 1];
      it = Item{vi->bh, vi->qb, vi->steps, vi->bad};
      mbar_arrive(&b.item_empty[n & 1]);
      blk_next = listed(0, 0);
      blk_after = listed(0, 1);
      if (QUANT && it.steps > 0) {
        const size_t qi = prm.q_per_token ? (size_t)it.bh * prm.Npad + it.qb * 128 + row : (size_t)it.bh * nT + it.qb;
        if (SAGE_DCHECK(qi, (long long)prm.BH * (prm.q_per_token ? prm.Npad : nT), kSiteSparseScale)) qs = __ldg(prm.q_scale + qi);
        if (row < D && SAGE_DCHECK((size_t)it.bh * D + row, (long long)prm.BH * D, kSiteSparseScale))
          vsc = __ldg(prm.v_scale + (size_t)it.bh * D + row);
      }
      return true;
    };
    ok = take_item(0);
    ks_next = scale_of(blk_next);
    for (int n = 0; ok; ++n) {
      const int c = it.steps;
      if (c < 0) break;
      // Every thread's value reaches the others through p_full, the MMA thread and o_ready,
      // and the item with steps before this one has had all threads past the one before it.
      if (QUANT && c > 0 && row < D) b.v_scale[done & 1][row] = vsc;
      float m = -INFINITY, l = 0.f;
      // A lane whose wait ran out goes on, on scores that mean nothing, to the end of its step: the warp
      // leaves as a whole.  (A vote at every wait costs 1.5 to 2%.)
      int steps = c;
      for (int j = 0; __all_sync(0xffffffffu, j < steps); ++j) {
        const int blk = blk_next;
        const float sc = QUANT ? __fmul_rn(__fmul_rn(qs, ks_next), softmax_c(D)) : softmax_c(D);
        blk_next = blk_after;
        blk_after = listed(j, 2);
        ks_next = scale_of(blk_next);
        const int valid = (unsigned)blk < (unsigned)nT ? min(128, N - blk * 128) : 0;
        it.bad |= valid == 0;
        if (!mbar_wait(&b.s_full, step & 1, abort_flag, limit)) steps = 0;
        tc_fence_after();
        // the whole S row in registers (one wait for four loads)
        uint32_t sr[128];
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) tmem_ld32(tS + ch * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[ch * 32]));
        tmem_wait_ld();
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) regs_after_wait(*reinterpret_cast<uint32_t(*)[32]>(&sr[ch * 32]));
        if constexpr (AHEAD) {
          tc_fence_before();
          mbar_arrive(&b.s_free);     // the S columns may now take the next QK
        }
        const bool whole = valid == 128;
        // QUANT: scores as 12582912 + S (exact) until after the max
        float f[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) f[i] = __uint_as_float(QUANT ? sr[i] + kMagicBits : sr[i]);
        // row max of the raw scores (s is monotone in f since sc >= 0)
        float mx;
        if (whole) {
          float a0 = f[0], a1 = f[1], a2 = f[2], a3 = f[3];
#pragma unroll
          for (int i = 4; i + 8 <= 128; i += 8) {   // columns 4 .. 123
            a0 = fmax3(a0, f[i], f[i + 1]);
            a1 = fmax3(a1, f[i + 2], f[i + 3]);
            a2 = fmax3(a2, f[i + 4], f[i + 5]);
            a3 = fmax3(a3, f[i + 6], f[i + 7]);
          }
          mx = fmaxf(fmax3(a0, a1, f[124]), fmax3(a2, a3, fmax3(f[125], f[126], f[127])));
        } else {
          mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < 128; ++i) mx = fmaxf(mx, i < valid ? f[i] : -INFINITY);
        }
        if constexpr (QUANT) {
          mx = __fsub_rn(mx, kMagic);                       // exact: the integer max as a float
#pragma unroll
          for (int i = 0; i < 128; i += 2) {                // exact: back to S as a float
            const float2 v = fadd2(make_float2(f[i], f[i + 1]), make_float2(-kMagic, -kMagic));
            f[i] = v.x;
            f[i + 1] = v.y;
          }
        }
        // a block outside the sequence has no maximum (0 * -inf is not a number)
        const float m_new = valid > 0 ? fmaxf(m, __fmul_rn(mx, sc)) : m;
        const float alpha = (m == -INFINITY) ? 0.f : ex2_approx(__fsub_rn(m, m_new));
        const float bias = __fsub_rn(kLog2PScale, m_new);   // x = f * sc + bias = s - m_new (+ log2 448)
        if (TURNS && !mbar_wait(&b.tok, step & 1, abort_flag, limit)) steps = 0;
        // p = 2^x, row sum (two packed accumulators), P packed for the PV MMA; `mask` zeroes the keys
        // >= N of a last block.  Two copies of the loop, so whole blocks carry no masking at all.
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
        uint32_t pk[QUANT ? 32 : 64];
        auto group = [&](int g, bool mask) {
          const float2 x01 = ffma2(f[4 * g], f[4 * g + 1], sc, bias);
          const float2 x23 = ffma2(f[4 * g + 2], f[4 * g + 3], sc, bias);
          float p0 = ex2_approx(x01.x), p1 = ex2_approx(x01.y), p2 = ex2_approx(x23.x), p3 = ex2_approx(x23.y);
          if (mask) {
            p0 = 4 * g + 0 < valid ? p0 : 0.f;
            p1 = 4 * g + 1 < valid ? p1 : 0.f;
            p2 = 4 * g + 2 < valid ? p2 : 0.f;
            p3 = 4 * g + 3 < valid ? p3 : 0.f;
          }
          acc0 = fadd2(acc0, make_float2(p0, p1));
          acc1 = fadd2(acc1, make_float2(p2, p3));
          if constexpr (QUANT) {
            pk[g] = pack_e4m3x4(p0, p1, p2, p3);
          } else {
            pk[2 * g] = pack_bf16x2(p0, p1);
            pk[2 * g + 1] = pack_bf16x2(p2, p3);
          }
        };
        if (whole) {
#pragma unroll
          for (int g = 0; g < 32; ++g) group(g, false);
        } else {
#pragma unroll
          for (int g = 0; g < 32; ++g) group(g, true);
        }
        if constexpr (TURNS) mbar_arrive(give);   // hand the exponential phase to the other lane
        const bool grew = j > 0 && __any_sync(0xffffffffu, m_new > m);
        if (AHEAD && j > 0) {         // the previous PV has read the P tile, O is stable
          if (!mbar_wait(&b.o_ready, (step - 1) & 1, abort_flag, limit)) steps = 0;
          tc_fence_after();
        }
        if constexpr (QUANT) {
          uint8_t* p_row = smem + SC::OFF_P + t * C::P_BYTES + row * 128;   // this row of the swizzled P tile
#pragma unroll
          for (int cc = 0; cc < 8; ++cc)
            *reinterpret_cast<uint4*>(p_row + ((cc ^ (row & 7)) << 4)) =
                make_uint4(pk[4 * cc], pk[4 * cc + 1], pk[4 * cc + 2], pk[4 * cc + 3]);
          fence_proxy_async_smem();   // generic-proxy writes -> visible to the MMA
        } else {
          tmem_st32(tP, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
          tmem_st32(tP + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[QUANT ? 0 : 32]));
        }
        // rescale O by alpha where the max grew (without AHEAD O is complete: the commit
        // after this step's QK covers the previous PV)
        if (grew) {
#pragma unroll
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t r[32];
            tmem_ld32(tO + ch * 32, r);
            tmem_wait_ld_regs(r);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 v = fmul2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), alpha);
              r[i] = __float_as_uint(v.x);
              r[i + 1] = __float_as_uint(v.y);
            }
            tmem_st32(tO + ch * 32, r);
          }
          if constexpr (QUANT) tmem_wait_st();
        }
        if constexpr (!QUANT) tmem_wait_st();
        const float2 acc = fadd2(acc0, acc1);
        l = __fadd_rn(__fmul_rn(l, alpha), __fadd_rn(acc.x, acc.y));
        m = m_new;
        tc_fence_before();
        mbar_arrive(&b.p_full);
        ++step;
      }
      if (!(ok = __all_sync(0xffffffffu, steps == c))) break;
      if (it.bad && row == 0) atomicOr(prm.status, kStatusBadIndex);
      const int gq = it.qb * 128 + row;
      const long long orow = ((long long)it.bh * N + gq) * D;
      if (!(ok = take_item(n + 1))) break;
      if (c > 0) {
        if (!(ok = mbar_wait_warp(&b.o_ready, (AHEAD ? step - 1 : done) & 1, abort_flag, limit))) break;
        ++done;
        tc_fence_after();
      }
      ks_next = scale_of(blk_next);
      // ---------------------------------------------------------- epilogue
      // bf16(a / l) for 32 columns at a time without 32 divisions: 1 / l lies between
      // the two neighbours of its rounded value, so a / l rounds between the products
      // with them; where both give the same bf16 that is the result, else divide.
      const float rl = __frcp_rn(l);
      const float rlo = __uint_as_float(__float_as_uint(rl) - 1u), rhi = __uint_as_float(__float_as_uint(rl) + 1u);
      const float4* vs4 = reinterpret_cast<const float4*>(b.v_scale[(done - 1) & 1]);
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t w[16];
        if (c > 0) {
          uint32_t r[32];
          tmem_ld32(tO + ch * 32, r);
          tmem_wait_ld_regs(r);
          float2 a[16];
#pragma unroll
          for (int g = 0; g < 16; ++g) a[g] = make_float2(__uint_as_float(r[2 * g]), __uint_as_float(r[2 * g + 1]));
          if constexpr (QUANT) {
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const float4 v4 = vs4[ch * 8 + g];
              a[2 * g] = fmul2v(a[2 * g], make_float2(v4.x, v4.y));
              a[2 * g + 1] = fmul2v(a[2 * g + 1], make_float2(v4.z, v4.w));
            }
          }
          uint32_t apart = 0;
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            const float2 lo = fmul2(a[g], rlo), hi = fmul2(a[g], rhi);
            w[g] = pack_bf16x2(lo.x, lo.y);
            apart |= w[g] ^ pack_bf16x2(hi.x, hi.y);
          }
          if (apart)
#pragma unroll
            for (int g = 0; g < 16; ++g) {
              const float2 hi = fmul2(a[g], rhi);
              if (w[g] != pack_bf16x2(hi.x, hi.y))
                w[g] = pack_bf16x2(__fdiv_rn(a[g].x, l), __fdiv_rn(a[g].y, l));   // QUANT: l holds 448 * sum(p)
            }
        }
        if (c == 0 || l == 0.f)                  // no block, or none inside the sequence
#pragma unroll
          for (int g = 0; g < 16; ++g) w[g] = 0u;
        if (gq < N && SAGE_DCHECK((orow + ch * 32) / 8 + 3, (long long)prm.BH * N * D / 8, kSiteSparseOut)) {
          __nv_bfloat16* dst = prm.o + orow + ch * 32;
          if (prm.wide) {
            store32(dst, w);
            store32(dst + 16, w + 8);
          } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              reinterpret_cast<uint4*>(dst)[v] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
          }
        }
      }
    }
    // A lane without items keeps giving its turns away until the other has ended, too.
    idle[t] = 1;
    while (TURNS && ok && !idle[1 - t]) {
      const long long t0 = clock64();
      while (!mbar_try_wait(&b.tok, step & 1) && !idle[1 - t] && ok) {
        if (clock64() - t0 > limit) *abort_flag = 1;
        ok = !*abort_flag;
      }
      mbar_arrive(give);
      ++step;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if (threadIdx.x == 0 && *abort_flag) atomicOr(prm.status, kStatusTimeout);
}

template <int D, bool QUANT>
cudaError_t launch_sparse_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const SparseParams& prm,
                            cudaStream_t stream) {
  using C = Cfg<D, QUANT>;
  using SC = SparseCfg<D, QUANT>;
  auto kern = sparse_kernel<D, QUANT>;
  // the setmaxnreg split must fit in the registers the block is launched with,
  // or the increase would wait forever
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * kThreads < 128 * C::REGS_LOW + 256 * C::REGS_HIGH) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SC::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return e;
  const int grid = std::min(sms, prm.items);
  if (prm.items > 2 * grid && (e = cudaMemsetAsync(prm.next, 0, sizeof(*prm.next), stream)) != cudaSuccess) return e;
  kern<<<grid, kThreads, SC::SMEM_BYTES, stream>>>(tq, tk, tv, prm);
  return cudaGetLastError();
}

}  // namespace

unsigned debug_take_sparse(unsigned long long* first) {
#ifdef SAGE_DEBUG
  return debug_take_tu(first);
#else
  (void)first;
  return 0;
#endif
}

// The item counter lies in the status region, behind the status word.
constexpr int kNextWord = 16;

cudaError_t launch_sparse_i8f8(const int8_t* q_i8, const float* q_scale, const int8_t* k_i8, const float* k_scale,
                               const uint8_t* v_f8t, const float* v_scale, void* o, int BH, int N, int d,
                               const int* lists, const int* counts, int width, uint32_t* status,
                               long long timeout_cycles, int dbg_flags, cudaStream_t stream, bool q_per_token) {
  const int nT = num_tiles(N), Npad = nT * kTile;
  alignas(64) CUtensorMap tq, tk, tv;
  const CUtensorMapSwizzle qk_sw = d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!encode_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, q_i8, d, (uint64_t)BH * Npad, d, d, 128, qk_sw) ||
      !encode_tmap_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, k_i8, d, (uint64_t)BH * Npad, d, d, 128, qk_sw) ||
      !encode_tmap_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, v_f8t, Npad, (uint64_t)BH * d, Npad, 128, d,
                      CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const SparseParams prm{q_scale, k_scale, v_scale, static_cast<__nv_bfloat16*>(o), lists, counts, status,
                         status + kNextWord, N, nT, Npad, width, BH, BH * nT, timeout_cycles, dbg_flags,
                         q_per_token ? 1 : 0, (reinterpret_cast<uintptr_t>(o) & 31u) == 0};
  return d == 128 ? launch_sparse_d<128, true>(tq, tk, tv, prm, stream)
                  : launch_sparse_d<64, true>(tq, tk, tv, prm, stream);
}

cudaError_t launch_sparse_bf16(const void* q, const void* k, const void* v, void* o, int BH, int N, int d,
                               const int* lists, const int* counts, int width, uint32_t* status,
                               long long timeout_cycles, int dbg_flags, cudaStream_t stream) {
  const int nT = num_tiles(N);
  alignas(64) CUtensorMap tq, tk, tv;
  const uint64_t s1 = (uint64_t)d * 2, s2 = (uint64_t)N * d * 2;
  if (!encode_tmap_3d(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q, d, N, BH, s1, s2, 64, 128, 1,
                      CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap_3d(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, k, d, N, BH, s1, s2, 64, 128, 1,
                      CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap_3d(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, v, d, N, BH, s1, s2, 64, 128, 1,
                      CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const SparseParams prm{nullptr, nullptr, nullptr, static_cast<__nv_bfloat16*>(o), lists, counts, status,
                         status + kNextWord, N, nT, nT * kTile, width, BH, BH * nT, timeout_cycles, dbg_flags, 0,
                         (reinterpret_cast<uintptr_t>(o) & 31u) == 0};
  return d == 128 ? launch_sparse_d<128, false>(tq, tk, tv, prm, stream)
                  : launch_sparse_d<64, false>(tq, tk, tv, prm, stream);
}

}  // namespace sage
