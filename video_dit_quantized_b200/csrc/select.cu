// select.cu -- the key blocks each query block attends to, chosen by a cheap
// score.
//
//   qbar_i, kbar_j = mean over the real rows of a 128-token block: exact sums
//                    in fp64 (128 bf16 values span far less than 53 bits),
//                    divided in fp64, rounded once to fp32;
//   s_ij           = sum_c qbar_i[c] * kbar_j[c] in fp64;
//   kept           = the `keep` largest s_ij of a row, ties to the lower j;
//                    blocks j < first and |i - j| <= window rank above all.
// The result is a set: over the 23,640 rows of the 720p sequence some pairs at the
// border differ by less than fp32 rounding, hence the fp64 definition.  But scores
// with a bound on their error decide nearly every row, and tensor cores give
// them in exact integers: every mean is split into three 8-bit slices,
//   x = step * (a0 + a1 / 2^7 + a2 / 2^14) + r,   step = amax / 127,   |r| <= 2^-14 step,
// and the six products of weight up to 2^-14 are summed in int32 (tcgen05 kind::i8,
// one accumulator a weight).  (All scores in fp64: 864 us at 1 x 40 x 75600 x 128; in
// fp32 on the FMA pipe, bound by shared-memory wavefronts: 247 us.)  Of the keys,
// token 0's values are subtracted first, which shifts a row's scores alike and
// makes amax, and with it the error, small where channels carry an offset.
//
// Two kernels.  pool: one CTA per (block, head, tensor), HBM-bound, q and k are
// read once; it writes the means, their slices, steps and norms.  score: one CTA
// per (16 query blocks, head) forms its rows of scores against every key block of
// the head in shared memory (the score matrix never reaches HBM), then one warp per
// row looks for a threshold with n scores at or above it.
//   |computed - exact| <= E = 3 step_q max step_k + 2^-23 |qbar| max |kbar|:
//   the products left out are below 0.51 step_q step_k (128 * 2 * 64 * 64 * 2^-21), the
//   remainders r below 128 * 127 * 2 * 4.7e-5 = 1.53, six fp32 roundings of at most
//   2.1e6 below 0.75, that of kbar - token 0 below 0.13; the second term is the rounding
//   of kbar in the definition.
//   a = the smallest kept, b = the largest left out: a - b > 2 E decides the row.
//   Else the rows' order is open only among scores in [a - 2 E, b + 2 E]: up to 32 of
//   them are computed in fp64 by the warp and ranked (9% of the rows); more (equal or
//   all-zero blocks, values that are not finite) send the row to a second pass, in
//   which the CTA computes the whole row in fp64 and bisects over its bits.
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
  float x = 0.f;                          // what is sliced
  if (c < D) {
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) t += part[i][c];
    t /= (double)nr;
    const float mean = __double2float_rn(t);
    if (SAGE_DCHECK(row * D + c, rows * D, kSitePoolOut)) out.mean[row * D + c] = mean;
    x = mean;
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
  }
  __syncthreads();
  if (c < D) {
    float sq = norm_part[0], am = amax_part[0];
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

// The same by a warp, four (D = 64: two) channels a lane and a fixed tree: equal means
// give equal scores here, too.
template <int D>
__device__ __forceinline__ double exact_score_warp(const float* __restrict__ q, const float* __restrict__ k, int lane) {
  double s = 0.0;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) s = fma((double)q[c * 32 + lane], (double)k[c * 32 + lane], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

constexpr int kScoreThreads = 256;
constexpr int kKeys = 128;                 // key blocks of one tile: the MMA's M
constexpr int kRows = 16;                  // query blocks of one tile: its N
constexpr uint32_t kScoreIdesc = make_idesc(kFmtS32Acc, kFmtS8, kFmtS8, 0, kKeys, kRows);
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

__device__ __forceinline__ float warp_min(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fminf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
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

// Writes one row's list by a warp.  make() gives a function of j0 that returns the mask
// of the kept blocks among j0 .. j0 + 3, called for a lane's stretch in order; it is
// made twice, to count and to write.
template <typename F>
__device__ __forceinline__ void write_list(const SelectParams& p, int bh, int i, int lane, F make) {
  const long long row = ((long long)bh * p.nT + i) * p.keep, ext = (long long)gridDim.y * p.nT * p.keep;
  (void)ext;
  const int from = lane * (p.nTp / 32), to = from + p.nTp / 32;
  int c = 0;
  auto counted = make();
  for (int j0 = from; j0 < to; j0 += 4) c += __popc(counted(j0));
  int at = lane_prefix(c, lane);
  const int done = __shfl_sync(0xffffffffu, at + c, 31);
  auto written = make();
  for (int j0 = from; j0 < to; j0 += 4) {
    unsigned m = written(j0);
    while (m) {
      if (at < p.keep && SAGE_DCHECK(row + at, ext, kSiteSelectOut)) p.lists[row + at] = j0 + __ffs(m) - 1;
      ++at;
      m &= m - 1;
    }
  }
  for (int s = done + lane; s < p.keep; s += 32)
    if (SAGE_DCHECK(row + s, ext, kSiteSelectOut)) p.lists[row + s] = -1;
  if (lane == 0) p.counts[(long long)bh * p.nT + i] = done;
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

// One row from its fp32 scores (forced blocks +inf, -inf behind the last), by one
// warp; false: the order at the border is open among more than 32 blocks.  cand: 32
// integers of the warp's own.
template <int D>
__device__ __forceinline__ bool select_row(const SelectParams& p, int bh, int i, int lane, const float* s, float E,
                                           const float* qrow, const float* kp, int* cand) {
  const int nT = p.nT, n = min(p.keep, nT), nv = p.nTp / 128;
  const float4* s4 = reinterpret_cast<const float4*>(s) + lane * nv;
  auto load4 = [&](int j0) { return *reinterpret_cast<const float4*>(s + j0); };
  if (n == nT) {
    write_list(p, bh, i, lane, [&] {
      return [&](int j0) { return j0 + 3 < nT ? 15u : j0 < nT ? (1u << (nT - j0)) - 1u : 0u; };
    });
    return true;
  }
  // blocks with a score of at least t
  auto count = [&](float t) {
    float c = 0.f;
#pragma unroll 4
    for (int x = 0; x < nv; ++x) {
      const float4 v = s4[x];
      c += (v.x >= t ? 1.f : 0.f) + (v.y >= t ? 1.f : 0.f);
      c += (v.z >= t ? 1.f : 0.f) + (v.w >= t ? 1.f : 0.f);
    }
    return __reduce_add_sync(0xffffffffu, (int)c);
  };
  float mn = INFINITY, mx = -INFINITY, sum = 0.f, sq = 0.f;
  int forced = 0;
#pragma unroll 4
  for (int x = 0; x < nv; ++x) {
    const float4 v = s4[x];
    const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = fabsf(y[e]) < INFINITY;
      mn = fminf(mn, in ? y[e] : INFINITY);
      mx = fmaxf(mx, in ? y[e] : -INFINITY);
      sum += in ? y[e] : 0.f;
      sq += in ? y[e] * y[e] : 0.f;
      forced += y[e] == INFINITY ? 1 : 0;
    }
  }
  mn = warp_min(mn);
  mx = warp_max(mx);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sq += __shfl_xor_sync(0xffffffffu, sq, o);
  }
  forced = __reduce_add_sync(0xffffffffu, forced);
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
#pragma unroll 4
  for (int x = 0; x < nv; ++x) {
    const float4 v = s4[x];
    const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a = fminf(a, y[e] >= split ? y[e] : INFINITY);
      b = fmaxf(b, y[e] >= split ? -INFINITY : y[e]);
    }
  }
  b = warp_max(b);
  a = found ? warp_min(a) : lo;
  if (found && a - b > 2.f * E) {
    write_list(p, bh, i, lane, [&] { return [&](int j0) { return mask4(load4(j0), [&](float v) { return v >= T; }); }; });
    return true;
  }
  const float from = a - 2.f * E, to = b + 2.f * E;
  auto is_open = [&](float v) { return v >= from && v <= to; };
  int above = 0, mine = 0;
  for (int x = 0; x < nv; ++x) {
    above += __popc(mask4(s4[x], [&](float v) { return v > to; }));
    mine += __popc(mask4(s4[x], is_open));
  }
  above = __reduce_add_sync(0xffffffffu, above);
  const int open = __reduce_add_sync(0xffffffffu, mine);
  if (open > 32) return false;
  // lane r gets the r-th open block's score in fp64
  const int before = lane_prefix(mine, lane);    // open blocks in front of this lane's stretch
  int at = before;
  for (int x = 0; x < nv; ++x) {
    unsigned m = mask4(s4[x], is_open);
    while (m) {
      cand[at++] = (lane * nv + x) * 4 + __ffs(m) - 1;
      m &= m - 1;
    }
  }
  __syncwarp();
  double v = -INFINITY;
#pragma unroll 4
  for (int r = 0; r < open; ++r) {
    const double x = exact_score_warp<D>(qrow, kp + (size_t)cand[r] * D, lane);
    if (lane == r) v = x;
  }
  int rank = 0;
  for (int r = 0; r < open; ++r) {
    const double o = __shfl_sync(0xffffffffu, v, r);
    rank += o > v || (o == v && r < lane) ? 1 : 0;
  }
  const unsigned kept = __ballot_sync(0xffffffffu, lane < open && rank < n - above);
  write_list(p, bh, i, lane, [&] {
    return [&, r = before](int j0) mutable {
      const float4 y = load4(j0);
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
template <int D, int ROWS>
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
    tmem_alloc(&tmem_slot, 128);                   // two sets of accumulators
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
  if (threadIdx.x < kRows) later[threadIdx.x] = 0;
  float sq[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) sq[r] = i0 + r < nT ? p.pooled.step[qrow + i0 + r] : 0.f;
  bool ok = true;
  int fetched = 1, committed = 0;                 // thread 0: tiles asked for, tiles given to the tensor cores
  for (int x = 0; x < ntiles; ++x) {
    tc_fence_before();
    if (!__syncthreads_and(ok)) break;            // the accumulators of tile x - 2 are read
    tc_fence_after();
    const uint32_t tmem = tmem_slot + (x & 1) * 64;
    if (threadIdx.x == 0) {
      ok = mbar_wait(&full, x & 1, &gave_up, kDefaultTimeoutCycles);
      tc_fence_after();
      const uint32_t a = smem_u32(sm), b = smem_u32(sm + C::OFF_Q);
      if (ok)
#pragma unroll
        for (int w = 0; w < 3; ++w)               // accumulator of weight 2^-7w
#pragma unroll
          for (int sl = 0; sl <= w; ++sl)         // key slice sl, query slice w - sl
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              mma_ss<kKindI8>(tmem + w * kRows, make_sdesc(a + sl * C::KEY_BYTES + k * 32, 16, 8 * D, C::LAYOUT),
                              make_sdesc(b + (w - sl) * C::ROW_BYTES + k * 32, 16, 8 * D, C::LAYOUT), kScoreIdesc,
                              sl > 0 || k > 0 ? 1u : 0u);
      mma_commit(&done);
      ++committed;
    }
    if (x == 0 && warp < 4) {
      // meanwhile: the largest norm and step of the head's keys, for the error bound
      float kn = 0.f, ks = 0.f;
      for (int j = threadIdx.x; j < nT; j += 128) {
        kn = fmaxf(kn, p.pooled.norm[krow + j]);
        ks = fmaxf(ks, p.pooled.step[krow + j]);
      }
      kn = warp_max(kn);
      ks = warp_max(ks);
      if (lane == 0) {
        kmax_part[0][warp] = kn;
        kmax_part[1][warp] = ks;
      }
    }
    ok = __all_sync(0xffffffffu, mbar_wait(&done, x & 1, &gave_up, kDefaultTimeoutCycles) && ok);
    tc_fence_after();
    if (threadIdx.x == 0 && ok && x + 1 < ntiles) {
      fetch_keys(x + 1);
      ++fetched;
    }
    if (ok && warp >= 4) {
      // thread = key block, columns = query blocks
      const int j = x * kKeys + threadIdx.x - 128;
      const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      uint32_t l0[16], l1[16], l2[16];
      tmem_ld16(at, l0);
      tmem_ld16(at + kRows, l1);
      tmem_ld16(at + 2 * kRows, l2);
      const float sk = j < nT ? p.pooled.step[krow + j] : 0.f;
      tmem_wait_ld_regs16(l0);
      tmem_wait_ld_regs16(l1);
      tmem_wait_ld_regs16(l2);
      if (j < p.nTp)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          // the sums are exact in fp32 (below 2^22)
          const float v = fmaf(fmaf((float)(int)l2[r], 0.0078125f, (float)(int)l1[r]), 0.0078125f, (float)(int)l0[r]) *
                          (sq[r] * sk);
          const bool forced = j < nT && p.forced(i0 + r, j);
          if (j < nT && !forced && !(fabsf(v) < INFINITY)) later[r] = 1;
          scores[(size_t)r * p.nTp + j] = j >= nT ? -INFINITY : forced ? INFINITY : v;
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
  if (warp == 1) tmem_dealloc(tmem_slot, 128);
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
    const bool sure = usable && later[rr] == 0 && E < 1e37f &&
                      select_row<D>(p, bh, i, lane, scores + (size_t)rr * p.nTp, E, qp + (size_t)i * D, kp, cand[warp]);
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

template <int D, int ROWS>
cudaError_t score_launch(const SelectParams& p, int BH, cudaStream_t stream) {
  alignas(64) CUtensorMap tk, tq;
  const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  const uint64_t rows = 6ull * BH * p.nT;
  if (!encode_tmap_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.pooled.slices, D, rows, D, D, kKeys, sw) ||
      !encode_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.pooled.slices, D, rows, D, D, kRows, sw))
    return cudaErrorInvalidValue;
  auto kern = score_select_kernel<D, ROWS>;
  const int smem = (int)ScoreCfg<D>::smem(ROWS, p.nTp);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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

constexpr size_t kSmemMax = 232448 - 2048;       // beside the static arrays
// 4-row CTAs hold the longest rows
static_assert(ScoreCfg<128>::smem(4, SAGE_SELECT_MAX_BLOCKS) <= kSmemMax, "the longest row must fit in shared memory");

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
  const SelectParams p{pooled, nT, nTp, keep, first, window, (float)z, slope, lists, counts};
  // sixteen rows a CTA, two CTAs per SM, while their scores fit; four for longer rows
  if (ScoreCfg<D>::smem(kRows, nTp) <= kSmemMax) return score_launch<D, kRows>(p, BH, stream);
  return score_launch<D, 4>(p, BH, stream);
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
