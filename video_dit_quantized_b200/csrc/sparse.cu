// sparse.cu -- attention over the key blocks listed for each query block.
//
//   O_i = softmax(Q_i K_L^T / sqrt(d)) V_L,   L = the keys of the 128-token
//   blocks lists[b, h, i, 0 .. counts[b, h, i] - 1];  an empty list gives 0.
//
// Two kernels with the arithmetic of the dense ones (attention.cu), step for
// step in list order, so a list of all blocks in ascending order gives the dense
// call's bits:
//   sparse_i8f8_kernel: exact int32 S, dequantized; P8 = e4m3(p * 448) through
//                       shared memory; O += P8 V8.
//   sparse_bf16_kernel: S and O += P V with kind::f16; P in tensor memory.
// One CTA = two neighbouring 128-row query blocks of one (b, h), twelve warps as
// in attention.cu (TMA producer, MMA issuer, two softmax warpgroups that take
// turns on the exponential phase).  The two query blocks have lists of their
// own, of any two lengths, so K and V tiles are fetched per query block: twice
// the L2-to-SM traffic of the dense kernels, which the steps' length covers
// (64 KB per 128 x 128 step of the BF16 kernel at d = 128).
//
// A listed index outside [0, ceil(N/128)) adds nothing to its row and a count
// outside [0, width] is clamped to it; both are recorded in the status word and
// read no memory outside the tensors.  Waits are bounded as in attention.cu.
#include <cuda_bf16.h>
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
  int N, nT, Npad, width;
  long long timeout;
  int dbg_flags;          // bit 0: MMA thread first waits on a barrier nobody arrives on
  int q_per_token;
};

// The block list of one query block.
struct BlockList {
  const int* at;
  long long off, ext;     // of the list and of the whole buffer, for the checks of a debug build
  int n, nT;
  bool bad;               // the count lies outside [0, width]; n is clamped to it
  __device__ __forceinline__ int raw(int j) const {
    return j < n && SAGE_DCHECK(off + j, ext, kSiteSparseList) ? __ldg(at + off + j) : 0;
  }
  // The block to load at step j: an index outside the sequence loads block 0,
  // whose scores the softmax then masks.
  __device__ __forceinline__ int block(int j) const {
    const int b = raw(j);
    return (unsigned)b < (unsigned)nT ? b : 0;
  }
};

__device__ __forceinline__ BlockList block_list(const SparseParams& p, int bh, int qt) {
  BlockList l;
  l.at = p.lists;
  l.nT = p.nT;
  l.n = 0;
  l.bad = false;
  l.off = 0;
  l.ext = (long long)gridDim.y * p.nT * p.width;
  if (qt < p.nT) {
    const long long row = (long long)bh * p.nT + qt;
    l.off = row * p.width;
    if (SAGE_DCHECK(row, (long long)gridDim.y * p.nT, kSiteSparseList)) {
      const int c = __ldg(p.counts + row);
      l.n = max(0, min(c, p.width));
      l.bad = c != l.n;
    }
  }
  return l;
}

// ---------------------------------------------------------------- BF16
// Shared memory: the two Q tiles, then a ring of one-tile slots through which K
// and V tiles pass in the order the MMA thread uses them:
//   K_0(0) K_1(0) | V_0(0) K_0(1) | V_1(0) K_1(1) | V_0(1) K_0(2) | ...
// Slots of one tile instead of (K, V) pairs per query block: at d = 128 only
// five 32 KB tiles fit beside Q, and a pair ring would hold two.
template <int D>
struct SparseBf16Cfg {
  using C = Cfg<D, false>;
  static constexpr int TILE_BYTES = C::TILE_BYTES;
  static constexpr int SLOTS = D == 128 ? 5 : 12;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_R = 2 * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_R + SLOTS * TILE_BYTES;
  static constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert((1 + 2 * SLOTS + 8 + 2) * 8 + 8 <= 512, "barriers");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    sparse_bf16_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const SparseParams prm) {
  using C = Cfg<D, false>;
  using SC = SparseBf16Cfg<D>;
  constexpr int SLOTS = SC::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SC::OFF_BAR);
  uint64_t* q_full = bars + 0;
  uint64_t* full = bars + 1;                          // [SLOTS]
  uint64_t* empty = full + SLOTS;                     // [SLOTS]
  uint64_t* s_full = empty + SLOTS;                   // [2] S_t written (MMA commit)
  uint64_t* p_full = s_full + 2;                      // [2] P_t written, O_t rescaled
  uint64_t* o_ready = p_full + 2;                     // [2] the last PV_t done
  uint64_t* tok = o_ready + 2;                        // [2] exp-phase token of softmax warpgroup t
  uint64_t* mma_done = tok + 2;
  uint64_t* never = mma_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.y;
  const int N = prm.N, nT = prm.nT;
  const int qt0 = 2 * blockIdx.x;
  const long long limit = prm.timeout;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 128);
      mbar_init(&o_ready[t], 1);
      mbar_init(&tok[t], 128);
    }
    mbar_init(mma_done, 1);
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
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      const BlockList l0 = block_list(prm, bh, qt0), l1 = block_list(prm, bh, qt0 + 1);
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      mbar_arrive_expect_tx(q_full, 2 * SC::TILE_BYTES);
      for (int t = 0; t < 2; ++t) {
        uint8_t* dst = smem + SC::OFF_Q + t * SC::TILE_BYTES;
#pragma unroll
        for (int a = 0; a < D / 64; ++a) tma_load_3d(dst + a * 16384, &tmQ, q_full, a * 64, (qt0 + t) * 128, bh);
      }
      int u = 0;                                       // tiles issued
      auto load = [&](const CUtensorMap* map, int blk) {
        const int s = u % SLOTS;
        if (u >= SLOTS && !mbar_wait(&empty[s], ((u / SLOTS) - 1) & 1, abort_flag, limit)) return false;
        mbar_arrive_expect_tx(&full[s], SC::TILE_BYTES);
        uint8_t* dst = smem + SC::OFF_R + s * SC::TILE_BYTES;
#pragma unroll
        for (int a = 0; a < D / 64; ++a) tma_load_3d(dst + a * 16384, map, &full[s], a * 64, blk * 128, bh);
        ++u;
        return true;
      };
      // blocks of this step (V) and of the next one (K), read a step ahead
      int v0 = l0.block(0), v1 = l1.block(0), k0 = l0.block(1), k1 = l1.block(1);
      bool go = (l0.n == 0 || load(&tmK, v0)) && (l1.n == 0 || load(&tmK, v1));
      const int steps = max(l0.n, l1.n);
      for (int j = 0; j < steps && go; ++j) {
        const int n0 = l0.block(j + 2), n1 = l1.block(j + 2);
        if (j < l0.n) go = load(&tmV, v0) && (j + 1 >= l0.n || load(&tmK, k0));
        if (go && j < l1.n) go = load(&tmV, v1) && (j + 1 >= l1.n || load(&tmK, k1));
        v0 = k0;
        v1 = k1;
        k0 = n0;
        k1 = n1;
      }
      // drain: every load this thread issued must land before the CTA exits
      volatile int no_abort = 0;
      mbar_wait(q_full, 0, &no_abort, limit);
      for (int i = u - SLOTS < 0 ? 0 : u - SLOTS; i < u; ++i)
        mbar_wait(&full[i % SLOTS], (i / SLOTS) & 1, &no_abort, limit);
    } else if (warp == 1 && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      const int c0 = block_list(prm, bh, qt0).n, c1 = block_list(prm, bh, qt0 + 1).n;
      const uint32_t q_s = smem_u32(smem + SC::OFF_Q);
      const uint32_t r_s = smem_u32(smem + SC::OFF_R);
      int u = 0;                                       // tiles consumed
      auto wait_tile = [&]() { return mbar_wait(&full[u % SLOTS], (u / SLOTS) & 1, abort_flag, limit); };
      auto qk = [&](int t) {
        if (!wait_tile()) return false;
        tc_fence_after();
        issue_qk<D, false>(tmem + t * 128, q_s + t * SC::TILE_BYTES, r_s + (u % SLOTS) * SC::TILE_BYTES);
        mma_commit(&s_full[t]);
        mma_commit(&empty[u % SLOTS]);
        ++u;
        return true;
      };
      auto step = [&](int t, int j, int c) {           // PV_t(j), then QK_t(j+1) over the same S columns
        if (!mbar_wait(&p_full[t], j & 1, abort_flag, limit) || !wait_tile()) return false;
        tc_fence_after();
        issue_pv_bf16<D>(tmem + 256 + t * D, tmem + t * 128, r_s + (u % SLOTS) * SC::TILE_BYTES, j > 0 ? 1u : 0u);
        mma_commit(&empty[u % SLOTS]);
        ++u;
        if (j + 1 < c) return qk(t);
        mma_commit(&o_ready[t]);
        return true;
      };
      bool ok = true;
      if (prm.dbg_flags & 1) ok = mbar_wait(never, 0, abort_flag, limit);
      ok = ok && mbar_wait(q_full, 0, abort_flag, limit);
      ok = ok && (c0 == 0 || qk(0)) && (c1 == 0 || qk(1));
      const int steps = max(c0, c1);
      for (int j = 0; j < steps && ok; ++j) ok = (j >= c0 || step(0, j, c0)) && (j >= c1 || step(1, j, c1));
      // drain: every MMA issued must complete before TMEM is released
      mma_commit(mma_done);
      volatile int no_abort = 0;
      mbar_wait(mma_done, 0, &no_abort, limit);
    }
  } else {
    regs_claim<C::REGS_HIGH>();
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + t * 128;
    const uint32_t tO = tmem + lane_off + 256 + t * D;
    const int qt = qt0 + t;
    const BlockList mine = block_list(prm, bh, qt);
    const int c_other = block_list(prm, bh, qt0 + 1 - t).n;
    const float sc = softmax_c(D);
    float m = -INFINITY, l = 0.f;
    bool ok = true, bad = mine.bad;
    int blk_next = mine.raw(0);
    for (int j = 0; j < mine.n; ++j) {
      const int blk = blk_next;
      blk_next = mine.raw(j + 1);
      const bool in = (unsigned)blk < (unsigned)nT;
      bad = bad || !in;
      const int valid = in ? min(128, N - blk * 128) : 0;
      if (!mbar_wait(&s_full[t], j & 1, abort_flag, limit)) { ok = false; break; }
      tc_fence_after();
      // the whole S row in registers (one wait for four loads)
      uint32_t sr[128];
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) tmem_ld32(tS + ch * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[ch * 32]));
      tmem_wait_ld();
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) regs_after_wait(*reinterpret_cast<uint32_t(*)[32]>(&sr[ch * 32]));
      float f[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) f[i] = __uint_as_float(sr[i]);
      const bool whole = valid == 128;
      // row max of the raw scores (s is monotone in f since sc > 0)
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
      const float m_new = fmaxf(m, __fmul_rn(mx, sc));
      const float alpha = (m == -INFINITY) ? 0.f : ex2_approx(__fsub_rn(m, m_new));
      const float bias = __fsub_rn(0.f, m_new);         // x = f * sc + bias = s - m_new
      // The warpgroups take turns on the exponential phase while both have
      // steps: 0 first, then they alternate.  Nobody waits for a turn that the
      // other, out of blocks, will not take.
      if (t == 0 ? (j > 0 && j - 1 < c_other) : j < c_other) {
        if (!mbar_wait(&tok[t], (t == 0 ? (j - 1) : j) & 1, abort_flag, limit)) { ok = false; break; }
      }
      // p = 2^x, row sum (two packed accumulators), P packed as bf16 for the PV MMA
      float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
      uint32_t pk[64];
      if (whole) {
#pragma unroll
        for (int g = 0; g < 32; ++g) {
          const float2 x01 = ffma2(f[4 * g], f[4 * g + 1], sc, bias);
          const float2 x23 = ffma2(f[4 * g + 2], f[4 * g + 3], sc, bias);
          const float p0 = ex2_approx(x01.x), p1 = ex2_approx(x01.y), p2 = ex2_approx(x23.x), p3 = ex2_approx(x23.y);
          acc0 = fadd2(acc0, make_float2(p0, p1));
          acc1 = fadd2(acc1, make_float2(p2, p3));
          pk[2 * g] = pack_bf16x2(p0, p1);
          pk[2 * g + 1] = pack_bf16x2(p2, p3);
        }
      } else {
#pragma unroll
        for (int g = 0; g < 32; ++g) {
          const float2 x01 = ffma2(f[4 * g], f[4 * g + 1], sc, bias);
          const float2 x23 = ffma2(f[4 * g + 2], f[4 * g + 3], sc, bias);
          const float p0 = 4 * g + 0 < valid ? ex2_approx(x01.x) : 0.f;
          const float p1 = 4 * g + 1 < valid ? ex2_approx(x01.y) : 0.f;
          const float p2 = 4 * g + 2 < valid ? ex2_approx(x23.x) : 0.f;
          const float p3 = 4 * g + 3 < valid ? ex2_approx(x23.y) : 0.f;
          acc0 = fadd2(acc0, make_float2(p0, p1));
          acc1 = fadd2(acc1, make_float2(p2, p3));
          pk[2 * g] = pack_bf16x2(p0, p1);
          pk[2 * g + 1] = pack_bf16x2(p2, p3);
        }
      }
      mbar_arrive(&tok[1 - t]);     // hand the exponential phase to the other warpgroup
      const bool grew = j > 0 && __any_sync(0xffffffffu, m_new > m);
      tmem_st32(tS, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
      tmem_st32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
      // rescale O_t by alpha where the max grew (O_t is complete: the commit
      // after QK_t(j) covers PV_t(j-1))
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
      }
      tmem_wait_st();
      const float2 acc = fadd2(acc0, acc1);
      l = __fadd_rn(__fmul_rn(l, alpha), __fadd_rn(acc.x, acc.y));
      m = m_new;
      tc_fence_before();
      mbar_arrive(&p_full[t]);
    }
    if (bad && row == 0) atomicOr(prm.status, kStatusBadIndex);
    // ---------------------------------------------------------- epilogue
    if (ok && (mine.n == 0 || mbar_wait(&o_ready[t], 0, abort_flag, limit))) {
      tc_fence_after();
      const int gq = qt * 128 + row;
      const long long orow = ((long long)bh * N + gq) * D;
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t w[16];
        if (mine.n > 0) {
          uint32_t r[32];
          tmem_ld32(tO + ch * 32, r);
          tmem_wait_ld_regs(r);
#pragma unroll
          for (int g = 0; g < 16; ++g) w[g] = pack_bf16x2(__fdiv_rn(__uint_as_float(r[2 * g]), l), __fdiv_rn(__uint_as_float(r[2 * g + 1]), l));
        }
        if (mine.n == 0 || l == 0.f)
#pragma unroll
          for (int g = 0; g < 16; ++g) w[g] = 0u;
        if (qt < nT && gq < N) {
          uint4* dst = reinterpret_cast<uint4*>(prm.o + orow + ch * 32);
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (SAGE_DCHECK((orow + ch * 32) / 8 + v, (long long)gridDim.y * N * D / 8, kSiteSparseOut))
              dst[v] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if (threadIdx.x == 0 && *abort_flag) atomicOr(prm.status, kStatusTimeout);
}

// ---------------------------------------------------------------- INT8/FP8
// Shared memory: the two Q tiles, a ring of STAGES (K, V) pairs for each query
// block, the two P tiles.
template <int D>
struct SparseI8Cfg {
  using C = Cfg<D, true>;
  static constexpr int TILE_BYTES = C::TILE_BYTES;
  static constexpr int STAGES = D == 128 ? 2 : 4;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE_BYTES;                        // [2][STAGES]
  static constexpr int OFF_V = OFF_K + 2 * STAGES * TILE_BYTES;       // [2][STAGES]
  static constexpr int OFF_P = OFF_V + 2 * STAGES * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_P + 2 * C::P_BYTES;
  static constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert((1 + 4 * STAGES + 10 + 2) * 8 + 8 <= 512, "barriers");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    sparse_i8f8_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const SparseParams prm) {
  using C = Cfg<D, true>;
  using SC = SparseI8Cfg<D>;
  constexpr int STAGES = SC::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SC::OFF_BAR);
  uint64_t* q_full = bars + 0;
  uint64_t* kv_full = bars + 1;                       // [2][STAGES]
  uint64_t* kv_empty = kv_full + 2 * STAGES;          // [2][STAGES]
  uint64_t* s_full = kv_empty + 2 * STAGES;           // [2] S_t written (MMA commit)
  uint64_t* s_free = s_full + 2;                      // [2] S_t read into registers
  uint64_t* p_full = s_free + 2;                      // [2] P_t written, O_t rescaled
  uint64_t* o_ready = p_full + 2;                     // [2] PV_t done
  uint64_t* tok = o_ready + 2;                        // [2] exp-phase token of softmax warpgroup t
  uint64_t* mma_done = tok + 2;
  uint64_t* never = mma_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.y;
  const int N = prm.N, nT = prm.nT;
  const int qt0 = 2 * blockIdx.x;
  const long long limit = prm.timeout;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < 2 * STAGES; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&s_free[t], 128);
      mbar_init(&p_full[t], 128);
      mbar_init(&o_ready[t], 1);
      mbar_init(&tok[t], 128);
    }
    mbar_init(mma_done, 1);
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
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      const BlockList l0 = block_list(prm, bh, qt0), l1 = block_list(prm, bh, qt0 + 1);
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      mbar_arrive_expect_tx(q_full, 2 * SC::TILE_BYTES);
      for (int t = 0; t < 2; ++t)
        tma_load_2d(smem + SC::OFF_Q + t * SC::TILE_BYTES, &tmQ, q_full, 0, bh * prm.Npad + (qt0 + t) * 128);
      auto load = [&](int t, int j, int blk) {
        const int s = t * STAGES + j % STAGES;
        if (j >= STAGES && !mbar_wait(&kv_empty[s], ((j / STAGES) - 1) & 1, abort_flag, limit)) return false;
        mbar_arrive_expect_tx(&kv_full[s], 2 * SC::TILE_BYTES);
        tma_load_2d(smem + SC::OFF_K + s * SC::TILE_BYTES, &tmK, &kv_full[s], 0, bh * prm.Npad + blk * 128);
        tma_load_2d(smem + SC::OFF_V + s * SC::TILE_BYTES, &tmV, &kv_full[s], blk * 128, bh * D);
        return true;
      };
      int done0 = 0, done1 = 0;                        // steps issued
      int b0 = l0.block(0), b1 = l1.block(0);
      const int steps = max(l0.n, l1.n);
      bool go = true;
      for (int j = 0; j < steps && go; ++j) {
        const int n0 = l0.block(j + 1), n1 = l1.block(j + 1);
        if (j < l0.n && (go = load(0, j, b0))) done0 = j + 1;
        if (go && j < l1.n && (go = load(1, j, b1))) done1 = j + 1;
        b0 = n0;
        b1 = n1;
      }
      // drain: every load this thread issued must land before the CTA exits
      volatile int no_abort = 0;
      mbar_wait(q_full, 0, &no_abort, limit);
      for (int t = 0; t < 2; ++t) {
        const int done = t == 0 ? done0 : done1;
        for (int j = done - STAGES < 0 ? 0 : done - STAGES; j < done; ++j)
          mbar_wait(&kv_full[t * STAGES + j % STAGES], (j / STAGES) & 1, &no_abort, limit);
      }
    } else if (warp == 1 && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      const int cnt[2] = {block_list(prm, bh, qt0).n, block_list(prm, bh, qt0 + 1).n};
      const uint32_t q_s = smem_u32(smem + SC::OFF_Q);
      const uint32_t k_s = smem_u32(smem + SC::OFF_K);
      const uint32_t v_s = smem_u32(smem + SC::OFF_V);
      const uint32_t p_s = smem_u32(smem + SC::OFF_P);
      bool ok = true;
      if (prm.dbg_flags & 1) ok = mbar_wait(never, 0, abort_flag, limit);
      ok = ok && mbar_wait(q_full, 0, abort_flag, limit);
      // Event driven, as in attn_i8f8_kernel, each query block with its own
      // tiles:  QK_t(j) needs s_free_t(j-1) (S_t(j-1) read out) and its K/V pair
      // loaded;  PV_t(j) needs p_full_t(j) (P_t(j) stored, O_t rescaled).
      int qk_next[2] = {0, 0}, pv_next[2] = {0, 0};
      long long last = clock64();
      while (ok && (pv_next[0] < cnt[0] || pv_next[1] < cnt[1])) {
        bool progressed = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int jq = qk_next[t];
          if (jq < cnt[t] && (jq == 0 || mbar_test(&s_free[t], (jq - 1) & 1)) &&
              mbar_test(&kv_full[t * STAGES + jq % STAGES], (jq / STAGES) & 1)) {
            tc_fence_after();
            issue_qk<D, true>(tmem + t * 128, q_s + t * SC::TILE_BYTES, k_s + (t * STAGES + jq % STAGES) * SC::TILE_BYTES);
            mma_commit(&s_full[t]);
            qk_next[t] = jq + 1;
            progressed = true;
          }
          const int jp = pv_next[t];
          if (jp < qk_next[t] && mbar_test(&p_full[t], jp & 1)) {
            tc_fence_after();
            issue_pv_quant<D>(tmem + 256 + t * D, p_s + t * C::P_BYTES, v_s + (t * STAGES + jp % STAGES) * SC::TILE_BYTES,
                              jp > 0 ? 1u : 0u);
            mma_commit(&o_ready[t]);
            mma_commit(&kv_empty[t * STAGES + jp % STAGES]);
            pv_next[t] = jp + 1;
            progressed = true;
          }
        }
        if (progressed) {
          last = clock64();
        } else if (*abort_flag || clock64() - last > limit) {
          *abort_flag = 1;
          ok = false;
        } else {
          __nanosleep(20);   // leave the issue slots to the softmax warps on this SMSP
        }
      }
      // drain: every MMA issued must complete before TMEM is released
      mma_commit(mma_done);
      volatile int no_abort = 0;
      mbar_wait(mma_done, 0, &no_abort, limit);
    }
  } else {
    regs_claim<C::REGS_HIGH>();
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + t * 128;
    const uint32_t tO = tmem + lane_off + 256 + t * D;
    uint8_t* p_row = smem + SC::OFF_P + t * C::P_BYTES + row * 128;   // this row of the swizzled P tile
    const int qt = qt0 + t;
    const BlockList mine = block_list(prm, bh, qt);
    const int c_other = block_list(prm, bh, qt0 + 1 - t).n;
    const float c = softmax_c(D);
    float qs = 0.f;
    if (qt < nT) {
      const size_t qi = prm.q_per_token ? (size_t)bh * prm.Npad + qt * 128 + row : (size_t)bh * nT + qt;
      const long long qe = (long long)gridDim.y * (prm.q_per_token ? prm.Npad : nT);
      qs = SAGE_DCHECK(qi, qe, kSiteSparseScale) ? prm.q_scale[qi] : 0.f;
      (void)qe;
    }
    // p is produced already multiplied by the P scale 448 (2^(s - m + log2 448)),
    // so l accumulates 448 * sum(p) and the epilogue divides by it directly.
    constexpr float kLog2PScale = 8.807354922057604f;
    // int32 S + 0x4B400000 read as a float is 12582912 + S exactly (|S| <= 127*127*128 < 2^22)
    constexpr uint32_t kMagicBits = 0x4B400000u;
    constexpr float kMagic = 12582912.0f;
    const long long ks_ext = (long long)gridDim.y * nT;
    (void)ks_ext;
    auto k_scale_of = [&](int blk) {
      const size_t ki = (size_t)bh * nT + ((unsigned)blk < (unsigned)nT ? blk : 0);
      return SAGE_DCHECK(ki, ks_ext, kSiteSparseScale) ? __ldg(prm.k_scale + ki) : 0.f;
    };
    // the next step's block and scale, and the block after it, are read ahead
    int blk_next = mine.raw(0), blk_after = mine.raw(1);
    float ks_next = k_scale_of(blk_next);
    float m = -INFINITY, l = 0.f;
    bool ok = true, bad = mine.bad;
    uint32_t sr[128];
    for (int j = 0; j < mine.n && ok; ++j) {
      const int blk = blk_next;
      const float sc = __fmul_rn(__fmul_rn(qs, ks_next), c);
      blk_next = blk_after;
      blk_after = mine.raw(j + 2);
      ks_next = k_scale_of(blk_next);
      const bool in = (unsigned)blk < (unsigned)nT;
      bad = bad || !in;
      const int valid = in ? min(128, N - blk * 128) : 0;
      if (!mbar_wait(&s_full[t], j & 1, abort_flag, limit)) { ok = false; break; }
      tc_fence_after();
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) tmem_ld32(tS + ch * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[ch * 32]));
      tmem_wait_ld();
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) regs_after_wait(*reinterpret_cast<uint32_t(*)[32]>(&sr[ch * 32]));
      tc_fence_before();
      mbar_arrive(&s_free[t]);     // the S columns may now take QK_t(j+1)
      const bool whole = valid == 128;
      // scores as 12582912 + S (exact) until after the max
      float f[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) f[i] = __uint_as_float(sr[i] + kMagicBits);
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
      mx = __fsub_rn(mx, kMagic);                       // exact: the integer max as a float
#pragma unroll
      for (int i = 0; i < 128; i += 2) {                // exact: back to S as a float
        const float2 v = fadd2(make_float2(f[i], f[i + 1]), make_float2(-kMagic, -kMagic));
        f[i] = v.x;
        f[i + 1] = v.y;
      }
      // a block outside the sequence has no maximum: 0 * -inf is not a number
      const float m_new = in ? fmaxf(m, __fmul_rn(mx, sc)) : m;
      const float alpha = (m == -INFINITY) ? 0.f : ex2_approx(__fsub_rn(m, m_new));
      const float bias = __fsub_rn(kLog2PScale, m_new);  // x = s * sc + bias = s - m_new + log2 448
      // the warpgroups take turns on the exponential phase while both have
      // steps: 0 first, then they alternate
      if (t == 0 ? (j > 0 && j - 1 < c_other) : j < c_other) {
        if (!mbar_wait(&tok[t], (t == 0 ? (j - 1) : j) & 1, abort_flag, limit)) { ok = false; break; }
      }
      float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
      uint32_t pk[32];
      // one group of four scores: 2^x, row sum, e4m3 pack; `mask` zeroes the keys >= N of a last
      // block.  Two copies of the loop, so whole blocks carry no masking at all.
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
        pk[g] = pack_e4m3x4(p0, p1, p2, p3);
      };
      if (whole) {
#pragma unroll
        for (int g = 0; g < 32; ++g) group(g, false);
      } else {
#pragma unroll
        for (int g = 0; g < 32; ++g) group(g, true);
      }
      mbar_arrive(&tok[1 - t]);     // hand the exponential phase to the other warpgroup
      const bool grew = j > 0 && __any_sync(0xffffffffu, m_new > m);
      if (j > 0) {
        if (!mbar_wait(&o_ready[t], (j - 1) & 1, abort_flag, limit)) { ok = false; break; }
        tc_fence_after();
      }
#pragma unroll
      for (int cc = 0; cc < 8; ++cc)
        *reinterpret_cast<uint4*>(p_row + ((cc ^ (row & 7)) << 4)) = make_uint4(pk[4 * cc], pk[4 * cc + 1], pk[4 * cc + 2], pk[4 * cc + 3]);
      fence_proxy_async_smem();    // generic-proxy writes -> visible to the MMA
      // rescale O_t by alpha where the max grew (PV_t(j-1) is done)
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
        tmem_wait_st();
      }
      const float2 acc = fadd2(acc0, acc1);
      l = __fadd_rn(__fmul_rn(l, alpha), __fadd_rn(acc.x, acc.y));
      m = m_new;
      tc_fence_before();
      mbar_arrive(&p_full[t]);
    }
    if (bad && row == 0) atomicOr(prm.status, kStatusBadIndex);
    // ---------------------------------------------------------- epilogue
    if (ok && (mine.n == 0 || mbar_wait(&o_ready[t], (uint32_t)((mine.n - 1) & 1), abort_flag, limit))) {
      tc_fence_after();
      const int gq = qt * 128 + row;
      const long long orow = ((long long)bh * N + gq) * D;
      const float* vs = prm.v_scale + (size_t)bh * D;
      const bool vs_ok = SAGE_DCHECK((size_t)bh * D + D - 1, (long long)gridDim.y * D, kSiteSparseScale);
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t w[16];
        if (mine.n > 0) {
          uint32_t r[32];
          tmem_ld32(tO + ch * 32, r);
          tmem_wait_ld_regs(r);
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            const float a0 = __fmul_rn(__uint_as_float(r[2 * g]), vs_ok ? vs[ch * 32 + 2 * g] : 0.f);
            const float a1 = __fmul_rn(__uint_as_float(r[2 * g + 1]), vs_ok ? vs[ch * 32 + 2 * g + 1] : 0.f);
            w[g] = pack_bf16x2(__fdiv_rn(a0, l), __fdiv_rn(a1, l));   // l holds 448 * sum(p)
          }
        }
        if (mine.n == 0 || l == 0.f)
#pragma unroll
          for (int g = 0; g < 16; ++g) w[g] = 0u;
        if (qt < nT && gq < N) {
          uint4* dst = reinterpret_cast<uint4*>(prm.o + orow + ch * 32);
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (SAGE_DCHECK((orow + ch * 32) / 8 + v, (long long)gridDim.y * N * D / 8, kSiteSparseOut))
              dst[v] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if (threadIdx.x == 0 && *abort_flag) atomicOr(prm.status, kStatusTimeout);
}

// The setmaxnreg split must fit in the registers the block is launched with, or
// the increase would wait forever.
template <typename K>
cudaError_t launch_split(K kern, int regs_low, int regs_high, int smem, const CUtensorMap& tq, const CUtensorMap& tk,
                         const CUtensorMap& tv, const SparseParams& prm, int BH, cudaStream_t stream) {
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * kThreads < 128 * regs_low + 256 * regs_high) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3((prm.nT + 1) / 2, BH), kThreads, smem, stream>>>(tq, tk, tv, prm);
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
  const SparseParams prm{q_scale, k_scale, v_scale, static_cast<__nv_bfloat16*>(o), lists, counts, status, N, nT, Npad,
                         width, timeout_cycles, dbg_flags, q_per_token ? 1 : 0};
  if (d == 128)
    return launch_split(sparse_i8f8_kernel<128>, Cfg<128, true>::REGS_LOW, Cfg<128, true>::REGS_HIGH,
                        SparseI8Cfg<128>::SMEM_BYTES, tq, tk, tv, prm, BH, stream);
  return launch_split(sparse_i8f8_kernel<64>, Cfg<64, true>::REGS_LOW, Cfg<64, true>::REGS_HIGH,
                      SparseI8Cfg<64>::SMEM_BYTES, tq, tk, tv, prm, BH, stream);
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
  const SparseParams prm{nullptr, nullptr, nullptr, static_cast<__nv_bfloat16*>(o), lists, counts, status, N, nT,
                         nT * kTile, width, timeout_cycles, dbg_flags, 0};
  if (d == 128)
    return launch_split(sparse_bf16_kernel<128>, Cfg<128, false>::REGS_LOW, Cfg<128, false>::REGS_HIGH,
                        SparseBf16Cfg<128>::SMEM_BYTES, tq, tk, tv, prm, BH, stream);
  return launch_split(sparse_bf16_kernel<64>, Cfg<64, false>::REGS_LOW, Cfg<64, false>::REGS_HIGH,
                      SparseBf16Cfg<64>::SMEM_BYTES, tq, tk, tv, prm, BH, stream);
}

}  // namespace sage
