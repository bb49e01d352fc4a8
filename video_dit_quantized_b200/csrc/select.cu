// select.cu -- the key blocks each query block attends to, chosen by a cheap
// score.
//
//   qbar_i, kbar_j = mean over the real rows of a 128-token block: summed in fp64
//                    (rows r, r + 8, r + 16, .. for each r < 8, then the eight
//                    sums), divided in fp64, rounded once to fp32.  Where a
//                    channel's nonzero values lie within a factor of 2^38 of each
//                    other the sum is exact, and the order does not matter;
//   s_ij           = sum_c qbar_i[c] * kbar_j[c] in fp64;
//   kept           = the `keep` largest s_ij of a row, ties to the lower j;
//                    blocks j < first and |i - j| <= window rank above all.
// The result is a set: over the 23,640 rows of the 720p sequence some pairs at the
// border differ by less than fp32 rounding, hence the fp64 definition.  But scores
// with a bound on their error decide nearly every row, and tensor cores give
// them in exact integers: every mean is split into three 8-bit slices,
//   x = step * (a0 + a1 / 2^7 + a2 / 2^14) + r,   step = amax / 127,   |r| <= 2^-14 step,
// and the six products of weight up to 2^-14 are summed in int32 (tcgen05 kind::i8).  (All
// scores in fp64: 864 us at 1 x 40 x 75600 x 128; in fp32 on the FMA pipe, bound by
// shared-memory wavefronts: 247 us; so: 98 us.)  Of the keys, token 0's values are
// subtracted first, which shifts a row's scores alike and makes amax, and with it the error,
// small where channels carry an offset.
//
// Two kernels.  pool: one CTA per (block, head, tensor), HBM-bound, q and k are
// read once; it writes the means, their slices, steps and norms.  score: one CTA
// per (16 query blocks, head) forms its rows of scores against every key block of
// the head in shared memory (the score matrix never reaches HBM), then one warp per
// row looks for a threshold with n scores at or above it.  What bounds it: latency (two
// CTAs of 8 warps per SM by shared memory); of 30,000 clocks a CTA the tiles take 14,000,
// a third of it the products' reads of the key slices from shared memory (each slice is
// read once for all query slices: the products took twice as long with one each), and
// a row's selection 5,000, 13,000 where scores are refined.
// The call at 1 x 40 x 75600 x 128: 363 to 366 us (4.3 TB/s), the pool kernel of it 262
// (5.9 TB/s, 0.90 of a copy); 1 x 30 x 17776 x 64: 47 us, 44 on the device.
//   |computed - exact| <= E = 3 step_q max step_k + 2^-23 |qbar| max |kbar|:
//   the products left out are below 0.51 step_q step_k (128 * 2 * 64 * 64 * 2^-21), the
//   remainders r below 128 * 127 * 2 * 4.7e-5 = 1.53, four fp32 roundings of at most
//   2.1e6 below 0.5, that of kbar - token 0 below 0.13; the second term is the rounding
//   of kbar in the definition.
//   a = the smallest kept, b = the largest left out: a - b > 2 E decides the row.
//   Else the rows' order is open only among scores in [a - 2 E, b + 2 E]: up to 32 of
//   them are computed in fp64 by the warp and ranked (9% of the rows); more (equal or
//   all-zero blocks, values that are not finite) send the row to a second pass, in
//   which the CTA computes the whole row in fp64 and bisects over its bits.  Its rows go one
//   after another: with all blocks equal the call above takes 4.9 ms, with the last quarter
//   of the tokens zero 3.3 ms.
#include <cuda_bf16.h>
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/sage_sparse.h"
#include "internal.h"
#include "sm100.cuh"

namespace sage {

namespace {

// One thread a channel: few threads with many loads each keep more bytes in flight per
// thread slot than the long tail of sums costs (280 us with 256 threads at 1 x 40 x 75600
// x 128, 262 with 128; 1 x 30 x 17776 x 64: 37 with 256, 28 with 64).
template <int D>
constexpr int kPoolThreads = D;

// What the pool kernel leaves in the scratch: the rounded means [2][BH][nT][D] (q, then
// k), their slices [2][3][BH][nT][D], steps and norms (a little rounded up) [2][BH][nT].
struct Pooled {
  float* mean;
  int8_t* slices;
  float* step;
  float* norm;
};

// grid (nT, BH, 2): z = 0 pools q, z = 1 pools k
template <int D>
__global__ void __launch_bounds__(kPoolThreads<D>) pool_blocks_kernel(const uint4* __restrict__ q,
                                                                   const uint4* __restrict__ k, int N, int nT,
                                                                   const Pooled out) {
  constexpr int V8 = D / 8, GROUPS = kPoolThreads<D> / V8, PER_T = kTile / GROUPS;
  __shared__ double part[GROUPS][D + 2];
  __shared__ float norm_part[D / 32], amax_part[D / 32];
  // the score kernel's blocks may take their places once every block of this grid has started
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int blk = blockIdx.x, bh = blockIdx.y;
  const int n0 = blk * kTile, nr = min(kTile, N - n0);
  const uint4* src = (blockIdx.z == 0 ? q : k);
  const size_t base = ((size_t)bh * N + n0) * V8;
  const long long ext = (long long)gridDim.y * N * V8;
  (void)ext;
  const int g = threadIdx.x / V8, v = threadIdx.x % V8;
  uint4 u[PER_T];
#pragma unroll
  for (int i = 0; i < PER_T; ++i) {
    const int row = i * GROUPS + g;
    u[i] = make_uint4(0, 0, 0, 0);
    if (row < nr && SAGE_DCHECK(base + (size_t)row * V8 + v, ext, kSitePoolIn)) u[i] = src[base + (size_t)row * V8 + v];
  }
  double s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < PER_T; ++i) {
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      s[2 * c] += (double)__uint_as_float(w[c] << 16);
      s[2 * c + 1] += (double)__uint_as_float(w[c] & 0xFFFF0000u);
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) part[g][v * 8 + c] = s[c];
  __syncthreads();
  const int c = threadIdx.x;
  const long long row = ((long long)blockIdx.z * gridDim.y + bh) * nT + blk, rows = 2LL * gridDim.y * nT;
  (void)rows;
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) t += part[i][c];
  t /= (double)nr;
  const float mean = __double2float_rn(t);
  if (SAGE_DCHECK(row * D + c, rows * D, kSitePoolOut)) out.mean[row * D + c] = mean;
  float x = mean;                         // what is sliced
  if (blockIdx.z == 1) {
    const size_t at = (size_t)bh * N * D + c;      // token 0 of the head
    if (SAGE_DCHECK(at / 8, ext, kSitePoolIn))
      x = __double2float_rn(t - (double)__bfloat162float(reinterpret_cast<const __nv_bfloat16*>(k)[at]));
  }
  float sq = mean * mean, am = fabsf(x) < INFINITY ? fabsf(x) : INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sq += __shfl_xor_sync(0xffffffffu, sq, o);
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  }
  if ((c & 31) == 0) {
    norm_part[c >> 5] = sq;
    amax_part[c >> 5] = am;
  }
  __syncthreads();
  sq = norm_part[0];
  am = amax_part[0];
#pragma unroll
  for (int i = 1; i < D / 32; ++i) {
    sq += norm_part[i];
    am = fmaxf(am, amax_part[i]);
  }
  // Not finite, or so small that squares and the reciprocal leave the normal range: an
  // infinite step, and with it an infinite error bound, sends the rows to the second pass.
  if (am > 0.f && am < 1e-15f) am = INFINITY;
  const float y = am > 0.f && am < INFINITY ? fminf(fmaxf(x * (127.f / am), -127.f), 127.f) : 0.f;
  const float a0 = rintf(y), r1 = (y - a0) * 128.f, a1 = rintf(r1), a2 = rintf((r1 - a1) * 128.f);
  const long long slice = (long long)gridDim.y * nT * D;             // elements of one slice of one tensor
  const long long at = blockIdx.z * 3 * slice + ((long long)bh * nT + blk) * D + c;
  if (SAGE_DCHECK(at + 2 * slice, 6 * slice, kSitePoolOut)) {
    out.slices[at] = (int8_t)a0;
    out.slices[at + slice] = (int8_t)a1;
    out.slices[at + 2 * slice] = (int8_t)a2;
  }
  if (c == 0 && SAGE_DCHECK(row, rows, kSitePoolOut)) {
    out.step[row] = am / 127.f;
    out.norm[row] = sqrtf(sq) * 1.001f;
  }
}

// Bits of a score in an order that unsigned comparison follows: negative scores
// below positive ones, -0 equal to +0, NaN below everything.
__device__ __forceinline__ unsigned long long ordered_bits(double s) {
  if (s != s) return 0ull;
  if (s == 0.0) s = 0.0;
  const unsigned long long b = (unsigned long long)__double_as_longlong(s);
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// s_ij in fp64, channels ascending: equal means give equal scores.
template <int D>
__device__ __forceinline__ double exact_score(const float* __restrict__ q, const float* __restrict__ k) {
  double s = 0.0;
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    const float4 a = *reinterpret_cast<const float4*>(q + c), b = *reinterpret_cast<const float4*>(k + c);
    s = fma((double)a.x, (double)b.x, s);
    s = fma((double)a.y, (double)b.y, s);
    s = fma((double)a.z, (double)b.z, s);
    s = fma((double)a.w, (double)b.w, s);
  }
  return s;
}

// The same by eight lanes, D / 8 channels each (q: this lane's) and a fixed tree: equal
// means give equal scores here, too.
template <int D>
__device__ __forceinline__ double exact_score_lanes(const float4 (&q)[D / 32], const float* __restrict__ k, int lane) {
  double s = 0.0;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const float4 b = *reinterpret_cast<const float4*>(k + c * 32 + (lane & 7) * 4);
    s = fma((double)q[c].x, (double)b.x, s);
    s = fma((double)q[c].y, (double)b.y, s);
    s = fma((double)q[c].z, (double)b.z, s);
    s = fma((double)q[c].w, (double)b.w, s);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

constexpr int kScoreThreads = 256;
constexpr int kRowRegs = 5;                // float4 of a row that a lane holds in registers
constexpr int kKeys = 128;                 // key blocks of one tile: the MMA's M
constexpr int kRows = 16;                  // query blocks of one tile: its N
// Tensor-memory columns of the product of key slice sl and query slice qs: 48, 32 and 16 for the key slices.
__host__ __device__ constexpr int acc_col(int sl, int qs) { return (sl * (7 - sl) / 2 + qs) * kRows; }
constexpr uint32_t kAccCols = 128;
static_assert(acc_col(1, 0) == 3 * kRows && acc_col(2, 0) == 5 * kRows && acc_col(2, 1) <= (int)kAccCols, "three products");
__host__ __device__ constexpr uint32_t score_idesc(int slices) { return make_idesc(kFmtS32Acc, kFmtS8, kFmtS8, 0, kKeys, slices * kRows); }
// Shared memory: 3 slices of a key tile (in the second pass: a row of 64-bit scores),
// 3 slices of the query tile, the fp32 scores of ROWS <= 16 rows.
template <int D>
struct ScoreCfg {
  static constexpr int KEY_BYTES = kKeys * D, ROW_BYTES = kRows * D;
  static constexpr uint32_t LAYOUT = D == 128 ? kLayoutSW128 : kLayoutSW64;
  static constexpr int OFF_Q = 3 * 128 * 128, OFF_SCORES = OFF_Q + 3 * ROW_BYTES;
  static constexpr size_t smem(int rows, int nTp) { return OFF_SCORES + sizeof(float) * (size_t)rows * nTp + 1024; }
  static_assert(8 * SAGE_SELECT_MAX_BLOCKS <= OFF_Q, "the second pass's row must fit");
};

// Smallest and largest of a warp's floats (no NaN) by the integer reductions: the bits
// of a negative float, all but the sign inverted, follow integer order, and back.
__device__ __forceinline__ int int_order(int bits) { return bits ^ (bits >> 31 & 0x7FFFFFFF); }
__device__ __forceinline__ float warp_min(float v) {
  return __int_as_float(int_order(__reduce_min_sync(0xffffffffu, int_order(__float_as_int(v)))));
}
__device__ __forceinline__ float warp_max(float v) {
  return __int_as_float(int_order(__reduce_max_sync(0xffffffffu, int_order(__float_as_int(v)))));
}

struct SelectParams {
  Pooled pooled;
  int nT, nTp, keep, first, window;              // nTp: nT rounded up to an odd multiple of 128
  float z, slope;         // of a normal row: (threshold - mean) / sigma, and blocks per sigma there
  int* lists;             // [BH, nT, keep]
  int* counts;            // [BH, nT]
  __device__ __forceinline__ bool forced(int i, int j) const {
    return j < first || (window >= 0 && abs(i - j) <= window);
  }
};

// A warp shares a row in 32 stretches of nTp / 32 consecutive blocks, one a lane; an
// odd number of float4 each, so that 16-byte reads of eight lanes meet no bank twice.
// Exclusive prefix of c over the lanes.
__device__ __forceinline__ int lane_prefix(int c, int lane) {
  const int own = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) c += x;
  }
  return c - own;
}

// The 4-bit mask of pred over a float4.
template <typename F>
__device__ __forceinline__ unsigned mask4(const float4& v, F pred) {
  return (pred(v.x) ? 1u : 0u) | (pred(v.y) ? 2u : 0u) | (pred(v.z) ? 4u : 0u) | (pred(v.w) ? 8u : 0u);
}

// One row's list as a warp writes it: each lane the blocks of its stretch, behind those of
// the lanes before it.
struct ListOut {
  const SelectParams& p;
  long long row, ext, count;
  int at, done;
  __device__ __forceinline__ ListOut(const SelectParams& p_, int bh, int i)
      : p(p_), row(((long long)bh * p_.nT + i) * p_.keep), ext((long long)gridDim.y * p_.nT * p_.keep),
        count((long long)bh * p_.nT + i) {}
  __device__ __forceinline__ void start(int c, int lane) {
    at = lane_prefix(c, lane);
    done = __shfl_sync(0xffffffffu, at + c, 31);
  }
  __device__ __forceinline__ void put(unsigned m, int j0) {
    while (m) {
      if (at < p.keep && SAGE_DCHECK(row + at, ext, kSiteSelectOut)) p.lists[row + at] = j0 + __ffs(m) - 1;
      ++at;
      m &= m - 1;
    }
  }
  __device__ __forceinline__ void end(int lane) {
    // unsigned: a signed counter would wrap where keep is near 2^31
    for (unsigned s = done + lane; s < (unsigned)p.keep; s += 32)
      if (SAGE_DCHECK(row + s, ext, kSiteSelectOut)) p.lists[row + s] = -1;
    if (lane == 0) p.counts[count] = done;
  }
};

// Writes one row's list by a warp.  make() gives a function of j0 that returns the mask
// of the kept blocks among j0 .. j0 + 3, called for a lane's stretch in order; it is
// made twice, to count and to write.
template <typename F>
__device__ __forceinline__ void write_list(const SelectParams& p, int bh, int i, int lane, F make) {
  ListOut out(p, bh, i);
  const int from = lane * (p.nTp / 32), to = from + p.nTp / 32;
  int c = 0;
  auto counted = make();
  for (int j0 = from; j0 < to; j0 += 4) c += __popc(counted(j0));
  out.start(c, lane);
  auto written = make();
  for (int j0 = from; j0 < to; j0 += 4) out.put(written(j0), j0);
  out.end(lane);
}

// The same for stretches of at most 32 blocks, block j0 + e of a lane kept where bit e of m is set.
__device__ __forceinline__ void write_bits(const SelectParams& p, int bh, int i, int lane, int j0, unsigned m) {
  ListOut out(p, bh, i);
  out.start(__popc(m), lane);
  out.put(m, j0);
  out.end(lane);
}

// One row from its 64-bit ordered scores (two arrays of halves), by one warp.  The
// kept set is {hi > th} plus, among hi == th, the `need` largest by (lo descending,
// j ascending): {lo > tl} plus the first `ties` of lo == tl.  th is built bit by bit
// as the largest value with at least n scores at or above it; once exactly n are,
// the set is known.
__device__ __noinline__ void select_exact(const SelectParams& p, int bh, int i, int lane, const uint32_t* h,
                                          const uint32_t* w) {
  const int nT = p.nT, n = min(p.keep, nT);
  auto count = [&](auto pred) {
    int c = 0;
    for (int j = lane; j < nT; j += 32) c += pred(j) ? 1 : 0;
    return __reduce_add_sync(0xffffffffu, c);
  };
  uint32_t th = 0, tl = 0;
  int ge = nT;                                   // scores with hi >= th
  for (int bit = 31; bit >= 0 && ge != n; --bit) {
    const uint32_t t = th | (1u << bit);
    const int c = count([&](int j) { return h[j] >= t; });
    if (c >= n) {
      th = t;
      ge = c;
    }
  }
  int ties = nT;
  if (ge != n) {                                 // several scores share the high half at the border
    const int need = n - count([&](int j) { return h[j] > th; });
    int eq = ge - (n - need);                    // with hi == th and lo >= tl
    for (int bit = 31; bit >= 0 && eq != need; --bit) {
      const uint32_t t = tl | (1u << bit);
      const int c = count([&](int j) { return h[j] == th && w[j] >= t; });
      if (c >= need) {
        tl = t;
        eq = c;
      }
    }
    if (eq != need)                              // full ties: the lowest j first
      ties = need - count([&](int j) { return h[j] == th && w[j] > tl; });
  }
  const int from = lane * (p.nTp / 32), to = from + p.nTp / 32;
  int tie = 0;
  for (int j = from; j < min(to, nT); ++j) tie += h[j] == th && w[j] == tl ? 1 : 0;
  const int before = lane_prefix(tie, lane);     // ties in front of this lane's stretch
  write_list(p, bh, i, lane, [&] {
    return [&, at = before](int j0) mutable {
      unsigned m = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j0 + e < nT) {
          const uint32_t hv = h[j0 + e], lv = w[j0 + e];
          const bool t = hv == th && lv == tl;
          if (hv > th || (hv == th && lv > tl) || (t && at < ties)) m |= 1u << e;
          at += t ? 1 : 0;
        }
      return m;
    };
  });
}

// A row's scores as a warp goes through them, lane by lane its stretch of nv float4.
// NV > 0: held in registers (-inf behind the stretch); 0: read from shared memory.
template <int NV>
struct Row {
  const float4* s4;
  int nv;
  float4 v[NV > 0 ? NV : 1];
  __device__ __forceinline__ Row(const float* s, int lane, int nv_) : s4(reinterpret_cast<const float4*>(s) + lane * nv_), nv(nv_) {
    if constexpr (NV > 0) {
#pragma unroll
      for (int x = 0; x < NV; ++x) v[x] = x < nv ? s4[x] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if constexpr (NV > 0) {
#pragma unroll
      for (int x = 0; x < NV; ++x) f(x, v[x]);
    } else {
#pragma unroll 4
      for (int x = 0; x < nv; ++x) f(x, s4[x]);
    }
  }
};

// Writes a row's list; make() as in write_list, its function taking (x, scores).
template <int NV, typename F>
__device__ __forceinline__ void write_row(const SelectParams& p, int bh, int i, int lane, const Row<NV>& row, F make) {
  if constexpr (NV > 0) {
    static_assert(4 * NV <= 32, "a lane's stretch as the bits of one word");
    unsigned m = 0;
    auto kept = make();
    row.each([&](int x, const float4& v) { m |= kept(x, v) << (4 * x); });
    write_bits(p, bh, i, lane, lane * row.nv * 4, m);
  } else {
    write_list(p, bh, i, lane, [&] {
      return [&, kept = make()](int j0) mutable {
        const int x = j0 / 4 - lane * row.nv;
        return kept(x, row.s4[x]);
      };
    });
  }
}

// One row from its fp32 scores (forced blocks +inf, -inf behind the last), by one
// warp; false: the order at the border is open among more than 32 blocks.  cand: 32
// integers of the warp's own.
template <int D, int NV>
__device__ __forceinline__ bool select_row(const SelectParams& p, int bh, int i, int lane, const float* s, float E,
                                           const float* qrow, const float* kp, int* cand) {
  const int nT = p.nT, n = min(p.keep, nT), nv = p.nTp / 128;
  const Row<NV> row(s, lane, nv);
  if (n == nT) {
    write_row<NV>(p, bh, i, lane, row, [&] {
      return [&](int x, const float4&) {
        const int j0 = (lane * nv + x) * 4;
        return x >= nv || j0 >= nT ? 0u : j0 + 3 < nT ? 15u : (1u << (nT - j0)) - 1u;
      };
    });
    return true;
  }
  // blocks with a score of at least t
  auto count = [&](float t) {
    float c = 0.f;
    row.each([&](int, const float4& v) {
      c += (v.x >= t ? 1.f : 0.f) + (v.y >= t ? 1.f : 0.f);
      c += (v.z >= t ? 1.f : 0.f) + (v.w >= t ? 1.f : 0.f);
    });
    return __reduce_add_sync(0xffffffffu, (int)c);
  };
  float mn = INFINITY, mx = -INFINITY, sum = 0.f, sq = 0.f;
  row.each([&](int, const float4& v) {
    const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = fabsf(y[e]) < INFINITY;
      mn = fminf(mn, in ? y[e] : INFINITY);
      mx = fmaxf(mx, in ? y[e] : -INFINITY);
      sum += in ? y[e] : 0.f;
      sq += in ? y[e] * y[e] : 0.f;
    }
  });
  mn = warp_min(mn);
  mx = warp_max(mx);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sq += __shfl_xor_sync(0xffffffffu, sq, o);
  }
  const int head = min(p.first, nT);
  const int forced = head + (p.window < 0 ? 0 : max(0, min(nT - 1, i + p.window) - max(head, i - p.window) + 1));
  // A threshold with count(s >= lo) > n > count(s >= hi) around it.  The first steps are
  // Newton's on a normal distribution of the row's mean and width, which meets n in about
  // five steps where halving takes eleven; from the eighth step on the bracket is halved, so
  // any row ends, at n or where only equal scores are left between.
  float lo = mn, hi = mx + fabsf(mx) * 2.4e-7f + 1e-37f, T = 0.f;
  bool found = false;
  if (forced == n) {                             // the forced blocks alone
    T = hi;
    found = true;
  }
  const float mean = sum / (float)(nT - forced), sigma = sqrtf(fmaxf(sq / (float)(nT - forced) - mean * mean, 0.f));
  float mid = mean + p.z * sigma;
  for (int it = 0; it < 72 && !found; ++it) {
    if (!(mid > lo && mid < hi) || it >= 8) mid = 0.5f * lo + 0.5f * hi;
    if (!(mid > lo && mid < hi)) break;
    const int c = count(mid);
    if (c == n) {
      T = mid;
      found = true;
    } else if (c > n) {
      lo = mid;
    } else {
      hi = mid;
    }
    mid += (float)(c - n) / p.slope * sigma;
  }
  // a: the smallest kept, b: the largest left out (where no threshold was found, b >= a)
  const float split = found ? T : hi;
  float a = INFINITY, b = -INFINITY;
  row.each([&](int, const float4& v) {
    const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a = fminf(a, y[e] >= split ? y[e] : INFINITY);
      b = fmaxf(b, y[e] >= split ? -INFINITY : y[e]);
    }
  });
  b = warp_max(b);
  a = found ? warp_min(a) : lo;
  if (found && a - b > 2.f * E) {
    write_row<NV>(p, bh, i, lane, row, [&] { return [&](int, const float4& v) { return mask4(v, [&](float y) { return y >= T; }); }; });
    return true;
  }
  const float from = a - 2.f * E, to = b + 2.f * E;
  auto is_open = [&](float v) { return v >= from && v <= to; };
  int above = 0, mine = 0;
  row.each([&](int, const float4& v) {
    above += __popc(mask4(v, [&](float y) { return y > to; }));
    mine += __popc(mask4(v, is_open));
  });
  above = __reduce_add_sync(0xffffffffu, above);
  const int open = __reduce_add_sync(0xffffffffu, mine);
  if (open > 32) return false;
  // lane r gets the r-th open block's score in fp64
  const int before = lane_prefix(mine, lane);    // open blocks in front of this lane's stretch
  int at = before;
  row.each([&](int x, const float4& v) {
    unsigned m = mask4(v, is_open);
    while (m) {
      cand[at++] = (lane * nv + x) * 4 + __ffs(m) - 1;
      m &= m - 1;
    }
  });
  __syncwarp();
  // four at a time, eight lanes each
  double v = -INFINITY;
  float4 qv[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) qv[c] = *reinterpret_cast<const float4*>(qrow + c * 32 + (lane & 7) * 4);
  for (int r = 0; r < open; r += 4) {
    const double x = exact_score_lanes<D>(qv, kp + (size_t)cand[min(r + (lane >> 3), open - 1)] * D, lane);
    const double y = __shfl_sync(0xffffffffu, x, (lane & 3) * 8);
    if (lane >= r && lane < min(r + 4, open)) v = y;
  }
  int rank = 0;
  for (int r = 0; r < open; ++r) {
    const double o = __shfl_sync(0xffffffffu, v, r);
    rank += o > v || (o == v && r < lane) ? 1 : 0;
  }
  const unsigned kept = __ballot_sync(0xffffffffu, lane < open && rank < n - above);
  write_row<NV>(p, bh, i, lane, row, [&] {
    return [&, r = before](int, const float4& y) mutable {
      const unsigned m = mask4(y, is_open);
      unsigned take = mask4(y, [&](float u) { return u > to; });
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (m >> e & 1u) take |= (kept >> r++ & 1u) << e;
      return take;
    };
  });
  return true;
}

// grid (ceil(nT / ROWS), BH)
template <int D, int ROWS, int NV>
__global__ void __launch_bounds__(kScoreThreads, ROWS == kRows ? 2 : 1)
    score_select_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                        const SelectParams p) {
  using C = ScoreCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ float kmax_part[2][4];
  __shared__ int later[kRows];                   // rows for the second pass
  __shared__ int cand[kScoreThreads / 32][32];
  __shared__ __align__(8) uint64_t full, done;
  __shared__ uint32_t tmem_slot;
  __shared__ int gave_up;
  float* scores = reinterpret_cast<float*>(sm + C::OFF_SCORES);
  const int nT = p.nT, bh = blockIdx.y, i0 = blockIdx.x * ROWS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t qrow = (size_t)bh * nT, krow = ((size_t)gridDim.y + bh) * nT;
  const float* qp = p.pooled.mean + qrow * D;
  const float* kp = p.pooled.mean + krow * D;
  const int ntiles = (nT + kKeys - 1) / kKeys;

  // A tile's three slices; rows behind the head's last belong to the next head (or are
  // zeros behind the tensor) and their scores are not used.
  auto fetch_keys = [&](int x) {
    mbar_arrive_expect_tx(&full, 3 * C::KEY_BYTES + (x == 0 ? 3 * C::ROW_BYTES : 0));
#pragma unroll
    for (int sl = 0; sl < 3; ++sl)
      tma_load_2d(sm + sl * C::KEY_BYTES, &tmK, &full, 0, ((3 + sl) * (int)gridDim.y + bh) * nT + x * kKeys);
  };
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kAccCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmQ);
    mbar_init(&full, 1);
    mbar_init(&done, 1);
    gave_up = 0;
    fence_mbar_init();
  }
  // launched while the pool kernel still runs: nothing of it is read before this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) {
    fetch_keys(0);
#pragma unroll
    for (int sl = 0; sl < 3; ++sl)
      tma_load_2d(sm + C::OFF_Q + sl * C::ROW_BYTES, &tmQ, &full, 0, (sl * (int)gridDim.y + bh) * nT + i0);
  }
  // each half of the block turns the accumulators into scores for half the rows
  constexpr int RH = ROWS / 2;
  const int r0 = warp < 4 ? 0 : RH;
  float sq[RH];
#pragma unroll
  for (int r = 0; r < RH; ++r) sq[r] = i0 + r0 + r < nT ? p.pooled.step[qrow + i0 + r0 + r] : 0.f;
  bool ok = true;
  int fetched = 1, committed = 0;                 // thread 0: tiles asked for, tiles given to the tensor cores
  for (int x = 0; x < ntiles; ++x) {
    tc_fence_before();
    if (!__syncthreads_and(ok)) break;            // the accumulators are read
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int j = x * kKeys + (threadIdx.x & 127);            // this thread's key block
    const float sk = j < nT ? p.pooled.step[krow + j] : 0.f;
    if (threadIdx.x == 0) {
      ok = mbar_wait(&full, x & 1, &gave_up, kDefaultTimeoutCycles);
      tc_fence_after();
      const uint32_t a = smem_u32(sm), b = smem_u32(sm + C::OFF_Q);
      // Key slice sl times query slices 0 .. 2 - sl, side by side as the columns of one product.  Each has
      // columns of its own: products of other widths into the same columns have no order among them.
      if (ok)
#pragma unroll
        for (int sl = 0; sl < 3; ++sl)
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_ss<kKindI8>(tmem + acc_col(sl, 0), make_sdesc(a + sl * C::KEY_BYTES + k * 32, 16, 8 * D, C::LAYOUT),
                            make_sdesc(b + k * 32, 16, 8 * D, C::LAYOUT), score_idesc(3 - sl), k > 0 ? 1u : 0u);
      mma_commit(&done);
      ++committed;
    }
    if (x == 0 && warp >= 4) {
      // meanwhile: the largest norm and step of the head's keys, for the error bound
      float kn = 0.f, ks = 0.f;
      for (int j = threadIdx.x - 128; j < nT; j += 128) {
        kn = fmaxf(kn, p.pooled.norm[krow + j]);
        ks = fmaxf(ks, p.pooled.step[krow + j]);
      }
      kn = warp_max(kn);
      ks = warp_max(ks);
      if (lane == 0) {
        kmax_part[0][warp - 4] = kn;
        kmax_part[1][warp - 4] = ks;
      }
    }
    ok = __all_sync(0xffffffffu, mbar_wait(&done, x & 1, &gave_up, kDefaultTimeoutCycles) && ok);
    tc_fence_after();
    if (threadIdx.x == 0 && ok && x + 1 < ntiles) {
      fetch_keys(x + 1);
      ++fetched;
    }
    if (ok) {
      const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + r0;
      uint32_t c[3][3][8];                        // key slice, query slice
#pragma unroll
      for (int sl = 0; sl < 3; ++sl)
#pragma unroll
        for (int qs = 0; qs < 3 - sl; ++qs) tmem_ld8(at + acc_col(sl, qs), c[sl][qs]);
#pragma unroll
      for (int sl = 0; sl < 3; ++sl)
#pragma unroll
        for (int qs = 0; qs < 3 - sl; ++qs) tmem_wait_ld_regs8(c[sl][qs]);
      // by weight 2^-7w: key slice + query slice = w
      uint32_t (&l0)[8] = c[0][0], l1[8], l2[8];
#pragma unroll
      for (int r = 0; r < RH; ++r) {
        l1[r] = c[0][1][r] + c[1][0][r];
        l2[r] = c[0][2][r] + c[1][1][r] + c[2][0][r];
      }
      float* to = scores + (size_t)r0 * p.nTp + j;
      if (j < p.nTp)
#pragma unroll
        for (int r = 0; r < RH; r += 2) {
          // l0 (below 2^21) as a float by way of 12582912 + l0, whose bits are an integer sum
          constexpr float kMagic = 12582912.f;
          const float2 h = fadd2(make_float2(__uint_as_float(l0[r] + 0x4B400000u), __uint_as_float(l0[r + 1] + 0x4B400000u)),
                                 make_float2(-kMagic, -kMagic));
          const float2 m = make_float2((float)((int)l1[r] * 128 + (int)l2[r]), (float)((int)l1[r + 1] * 128 + (int)l2[r + 1]));
          const float2 v = fmul2v(ffma2v(m, make_float2(0x1p-14f, 0x1p-14f), h),
                                  fmul2v(make_float2(sq[r], sq[r + 1]), make_float2(sk, sk)));
          to[(size_t)r * p.nTp] = j < nT ? v.x : -INFINITY;
          to[(size_t)(r + 1) * p.nTp] = j < nT ? v.y : -INFINITY;
        }
    }
  }
  for (int j = ntiles * kKeys + threadIdx.x; j < p.nTp; j += kScoreThreads)
    for (int r = 0; r < ROWS; ++r) scores[(size_t)r * p.nTp + j] = -INFINITY;
  if (threadIdx.x == 0 && gave_up) {              // what is under way ends before its memory is used again
    volatile int no_abort = 0;
    mbar_wait(&full, (fetched - 1) & 1, &no_abort, kDefaultTimeoutCycles);
    if (committed > 0) mbar_wait(&done, (committed - 1) & 1, &no_abort, kDefaultTimeoutCycles);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_slot, kAccCols);
  float kn = kmax_part[0][0], ks = kmax_part[1][0];
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    kn = fmaxf(kn, kmax_part[0][w]);
    ks = fmaxf(ks, kmax_part[1][w]);
  }

  // a wait that ran out leaves no scores: every row goes to the second pass
  const bool usable = gave_up == 0;
  for (int rr = warp; rr < ROWS; rr += kScoreThreads / 32) {
    const int i = i0 + rr;
    if (i >= nT) continue;
    const float E = 3.f * p.pooled.step[qrow + i] * ks + 1.1920929e-7f * p.pooled.norm[qrow + i] * kn + 1e-37f;
    float* row = scores + (size_t)rr * p.nTp;
    for (int j = lane; j < min(p.first, nT); j += 32) row[j] = INFINITY;
    for (int j = max(0, i - p.window) + lane; j <= min(nT - 1, i + p.window); j += 32) row[j] = INFINITY;
    __syncwarp();
    // below this limit on E, steps and scores are finite
    const bool sure = usable && E < 1e31f &&
                      select_row<D, NV>(p, bh, i, lane, row, E, qp + (size_t)i * D, kp, cand[warp]);
    __syncwarp();
    if (lane == 0) later[rr] = sure ? 0 : 1;
  }
  __syncthreads();

  // second pass: a whole row in fp64
  uint32_t* hi = reinterpret_cast<uint32_t*>(sm);
  uint32_t* lo = hi + nT;
  for (int rr = 0; rr < ROWS; ++rr) {
    const int i = i0 + rr;
    if (i >= nT || later[rr] == 0) continue;      // the same for all threads
    for (int j = threadIdx.x; j < nT; j += kScoreThreads) {
      const unsigned long long o = p.forced(i, j) ? ~0ull : ordered_bits(exact_score<D>(qp + (size_t)i * D, kp + (size_t)j * D));
      hi[j] = (uint32_t)(o >> 32);
      lo[j] = (uint32_t)o;
    }
    __syncthreads();
    if (warp == 0) select_exact(p, bh, i, lane, hi, lo);
    __syncthreads();
  }
}

constexpr size_t kSmemMax = 232448 - 2048;       // beside the static arrays
// 4-row CTAs hold the longest rows
static_assert(ScoreCfg<128>::smem(4, SAGE_SELECT_MAX_BLOCKS) <= kSmemMax, "the longest row must fit in shared memory");

template <int D, int ROWS, int NV>
cudaError_t score_launch(const SelectParams& p, int BH, cudaStream_t stream) {
  alignas(64) CUtensorMap tk, tq;
  const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  const uint64_t rows = 6ull * BH * p.nT;
  if (!encode_tmap_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.pooled.slices, D, rows, D, D, kKeys, sw) ||
      !encode_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.pooled.slices, D, rows, D, D, kRows, sw))
    return cudaErrorInvalidValue;
  auto kern = score_select_kernel<D, ROWS, NV>;
  const int smem = (int)ScoreCfg<D>::smem(ROWS, p.nTp);
  // The limit is the function's, not the launch's: this call's own size, set by two host threads at
  // once, could lower it between the other's setting and launch.
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
  if (e != cudaSuccess) return e;
  // its blocks may start, and set themselves up, while the pool kernel's last ones run
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.nT + ROWS - 1) / ROWS, BH);
  cfg.blockDim = dim3(kScoreThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tk, tq, p);
}

Pooled pooled_carve(void* base, int BH, int nT, int d) {
  const size_t rows = 2 * (size_t)BH * nT;
  char* p = static_cast<char*>(base);
  Pooled o;
  o.mean = reinterpret_cast<float*>(p);
  p += align_up(rows * d * 4, 256);
  o.slices = reinterpret_cast<int8_t*>(p);
  p += align_up(rows * 3 * d, 256);
  o.step = reinterpret_cast<float*>(p);
  p += align_up(rows * 4, 256);
  o.norm = reinterpret_cast<float*>(p);
  return o;
}

template <int D>
cudaError_t select_d(const void* q, const void* k, int BH, int N, int keep, int first, int window, int* lists,
                     int* counts, void* scratch, cudaStream_t stream) {
  const int nT = num_tiles(N);
  const Pooled pooled = pooled_carve(scratch, BH, nT, D);
  pool_blocks_kernel<D><<<dim3(nT, BH, 2), kPoolThreads<D>, 0, stream>>>(static_cast<const uint4*>(q),
                                                                      static_cast<const uint4*>(k), N, nT, pooled);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // where a normal row of nT scores has its n-th largest, by Newton's method on the
  // normal distribution function, and its density there
  const double share = std::min(std::max((double)std::min(keep, nT) / nT, 1e-6), 1.0 - 1e-6);
  double z = 0.0;
  for (int it = 0; it < 20; ++it) {
    const double density = std::exp(-0.5 * z * z) / 2.5066282746310002;
    z += std::min(std::max((0.5 * std::erfc(z / 1.4142135623730951) - share) / density, -0.5), 0.5);
  }
  const float slope = (float)std::max(1.0, nT * std::exp(-0.5 * z * z) / 2.5066282746310002);
  const int nTp = ((nT + 127) / 128 | 1) * 128;
  const SelectParams p{pooled, nT, nTp, keep, first, std::min(window, nT), (float)z, slope, lists, counts};
  // A warp's row in registers while a lane's stretch is at most 20 blocks (read again for
  // every threshold the call takes 401 us at 1 x 40 x 75600 x 128, in registers 375);
  // sixteen rows a CTA, two CTAs per SM, while their scores fit; four for longer rows (1 x 4 x
  // 332800 x 128, 2600 blocks, sixteen rows: 414 us; 1 x 4 x 384000 x 128, four: 634 us).
  if (nTp <= 128 * kRowRegs) return score_launch<D, kRows, kRowRegs>(p, BH, stream);
  if (ScoreCfg<D>::smem(kRows, nTp) <= kSmemMax) return score_launch<D, kRows, 0>(p, BH, stream);
  return score_launch<D, 4, 0>(p, BH, stream);
}

}  // namespace

unsigned debug_take_select(unsigned long long* first) {
#ifdef SAGE_DEBUG
  return debug_take_tu(first);
#else
  (void)first;
  return 0;
#endif
}

size_t select_scratch_bytes(int BH, int N, int d) {
  const size_t rows = 2 * (size_t)BH * num_tiles(N);
  return align_up(rows * d * 4, 256) + align_up(rows * 3 * d, 256) + 2 * align_up(rows * 4, 256);
}

cudaError_t launch_select_blocks(const void* q, const void* k, int BH, int N, int d, int keep, int first, int window,
                                 int* lists, int* counts, void* scratch, cudaStream_t stream) {
  return d == 128 ? select_d<128>(q, k, BH, N, keep, first, window, lists, counts, scratch, stream)
                  : select_d<64>(q, k, BH, N, keep, first, window, lists, counts, scratch, stream);
}

}  // namespace sage
