// select.cu -- the key blocks each query block attends to, chosen by a cheap
// score.
//
//   qbar_i, kbar_j = mean over the real rows of a 128-token block: exact sums
//                    in fp64 (128 bf16 values span far less than 53 bits),
//                    divided in fp64, rounded once to fp32;
//   s_ij           = sum_c qbar_i[c] * kbar_j[c] in fp64;
//   kept           = the `keep` largest s_ij of a row, ties to the lower j;
//                    blocks j < first and |i - j| <= window rank above all.
// The result is a set, and fp32 scores do not decide it: over the 23,640 rows of
// the 720p sequence some pairs at the border differ by less than fp32 rounding.
// But fp32 scores with a bound on their error decide nearly every row, so fp64
// is kept for the rest (all-fp64 scores took 864 us at 1 x 40 x 75600 x 128, this
// form 286).
//
// Two kernels.  pool: one CTA per (block, head, tensor), HBM-bound, q and k are
// read once; it also writes the norm of every mean.  score: one CTA per (R query
// blocks, head) forms its rows of scores against every key block of the head in
// shared memory (the score matrix never reaches HBM), then one warp per row
// bisects for a threshold with n scores at or above it:
//   |computed - exact| <= E = 20 * 2^-24 * |qbar| * max |kbar|  (eight products a
//   partial sum, eight partial sums a half, two halves: 17 roundings deep; Cauchy);
//   a = the smallest kept, b = the largest left out: a - b > 2 E decides the row.
//   Else the rows' order is open only among scores in [a - 2 E, b + 2 E]: up to 32 of
//   them are computed in fp64 by the warp, one a lane, and ranked; more (equal or
//   all-zero blocks, scores that are not finite) send the row to a second pass, in
//   which the CTA computes the whole row in fp64 and bisects over its bits.
#include <cuda_bf16.h>
#include <cstdint>

#include "../../include/sage_sparse.h"
#include "internal.h"
#include "sm100.cuh"

namespace sage {

namespace {

constexpr int kPoolThreads = 256;

// grid (nT, BH, 2): z = 0 pools q, z = 1 pools k; pooled [2][BH][nT][D], norms
// [2][BH][nT] (of the rounded means, rounded up a little)
template <int D>
__global__ void __launch_bounds__(kPoolThreads) pool_blocks_kernel(const uint4* __restrict__ q,
                                                                   const uint4* __restrict__ k, int N, int nT,
                                                                   float* __restrict__ pooled,
                                                                   float* __restrict__ norms) {
  constexpr int V8 = D / 8, GROUPS = kPoolThreads / V8, PER_T = kTile / GROUPS;
  __shared__ double part[GROUPS][D + 2];
  __shared__ float norm_part[D / 32];
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
  if (threadIdx.x < D) {
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) t += part[i][threadIdx.x];
    const long long blk_row = ((long long)blockIdx.z * gridDim.y + bh) * nT + blk;
    const float mean = __double2float_rn(t / (double)nr);
    if (SAGE_DCHECK(blk_row * D + threadIdx.x, 2LL * gridDim.y * nT * D, kSitePoolOut))
      pooled[blk_row * D + threadIdx.x] = mean;
    float sq = mean * mean;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if ((threadIdx.x & 31) == 0) norm_part[threadIdx.x >> 5] = sq;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float sq = norm_part[0];
#pragma unroll
    for (int i = 1; i < D / 32; ++i) sq += norm_part[i];
    const long long blk_row = ((long long)blockIdx.z * gridDim.y + bh) * nT + blk;
    if (SAGE_DCHECK(blk_row, 2LL * gridDim.y * nT, kSitePoolOut)) norms[blk_row] = sqrtf(sq) * 1.001f;
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

constexpr int kScoreThreads = 256;
constexpr int kDepth = 16;                 // channels of one tile
constexpr int kStages = 3;                 // tiles in shared memory
constexpr int kTileRow = kDepth + 4;       // floats; 80-byte rows keep 16-byte reads of 8 rows conflict-free

// Tile shape: a warp covers 4 * RT rows x 32 keys (thread: RT x 4), the eight warps
// WR row groups x 8 / WR key groups.
template <int RT, int WR>
struct ScoreCfg {
  static constexpr int ROWS = 4 * RT * WR, KEYS = 32 * 8 / WR;
  static constexpr int TILE = (KEYS + ROWS) * kTileRow;                 // floats
  // the tiles, which the second pass reuses for a row of 64-bit scores, and the fp32 scores
  static __host__ __device__ constexpr size_t tiles(int nTp) {
    return kStages * TILE * sizeof(float) > 8 * (size_t)nTp ? kStages * TILE * sizeof(float) : 8 * (size_t)nTp;
  }
  static __host__ __device__ constexpr size_t smem(int nTp) { return tiles(nTp) + sizeof(float) * (size_t)ROWS * nTp; }
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool live) {
  // src-size 0 writes zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}

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
  const float* pooled;    // [2][BH][nT][D]
  const float* norms;     // [2][BH][nT]
  int nT, nTp, keep, first, window;              // nTp: nT rounded up to 128
  int* lists;             // [BH, nT, keep]
  int* counts;            // [BH, nT]
  __device__ __forceinline__ bool forced(int i, int j) const {
    return j < first || (window >= 0 && abs(i - j) <= window);
  }
};

// A warp walks a row 128 blocks at a time, lane l holding blocks 4 l .. 4 l + 3.
// Exclusive prefix over the lanes of the number of set bits of m (4 bits), and the
// warp's total.
__device__ __forceinline__ int lane_prefix(unsigned m, int lane, int& total) {
  int c = __popc(m);
  const int own = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) c += x;
  }
  total = __shfl_sync(0xffffffffu, c, 31);
  return c - own;
}

// Writes one row's list by a warp: take(j0) gives the 4-bit mask of the kept blocks
// among j0 .. j0 + 3; called by all lanes together.
template <typename F>
__device__ __forceinline__ void write_list(const SelectParams& p, int bh, int i, int lane, F take) {
  const long long row = ((long long)bh * p.nT + i) * p.keep, ext = (long long)gridDim.y * p.nT * p.keep;
  (void)ext;
  int done = 0;
  for (int jb = 0; jb < p.nTp; jb += 128) {
    const int j0 = jb + 4 * lane;
    const unsigned m = take(j0);
    int total, at = done + lane_prefix(m, lane, total);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m >> e & 1u) {
        if (at < p.keep && SAGE_DCHECK(row + at, ext, kSiteSelectOut)) p.lists[row + at] = j0 + e;
        ++at;
      }
    done += total;
  }
  for (int s = done + lane; s < p.keep; s += 32)
    if (SAGE_DCHECK(row + s, ext, kSiteSelectOut)) p.lists[row + s] = -1;
  if (lane == 0) p.counts[(long long)bh * p.nT + i] = done;
}

// The 4-bit mask of pred over a float4.
template <typename F>
__device__ __forceinline__ unsigned mask4(const float4& v, F pred) {
  return (pred(v.x) ? 1u : 0u) | (pred(v.y) ? 2u : 0u) | (pred(v.z) ? 4u : 0u) | (pred(v.w) ? 8u : 0u);
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
  int tied = 0;
  write_list(p, bh, i, lane, [&](int j0) {
    unsigned sure = 0, tie = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j0 + e < nT) {
        const uint32_t hv = h[j0 + e], lv = w[j0 + e];
        if (hv > th || (hv == th && lv > tl)) sure |= 1u << e;
        if (hv == th && lv == tl) tie |= 1u << e;
      }
    int total, before = tied + lane_prefix(tie, lane, total);
    tied += total;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (tie >> e & 1u && before++ < ties) sure |= 1u << e;
    return sure;
  });
}

// One row from its fp32 scores (forced blocks +inf, -inf behind the last), by one
// warp; false: the order at the border is open among more than 32 blocks.  cand: 32
// integers of the warp's own.
template <int D>
__device__ __forceinline__ bool select_row(const SelectParams& p, int bh, int i, int lane, const float* s, float E,
                                           const float* qrow, const float* kp, int* cand) {
  const int nT = p.nT, n = min(p.keep, nT), nv = p.nTp / 128;
  const float4* s4 = reinterpret_cast<const float4*>(s) + lane;
  if (n == nT) {
    write_list(p, bh, i, lane, [&](int j0) { return j0 + 3 < nT ? 15u : j0 < nT ? (1u << (nT - j0)) - 1u : 0u; });
    return true;
  }
  auto count = [&](auto pred) {
    int c = 0;
#pragma unroll 4
    for (int t = 0; t < nv; ++t) c += __popc(mask4(s4[t * 32], pred));
    return __reduce_add_sync(0xffffffffu, c);
  };
  float mn = INFINITY, mx = -INFINITY;
#pragma unroll 4
  for (int t = 0; t < nv; ++t) {
    const float4 v = s4[t * 32];
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (fabsf(x[e]) < INFINITY) {
        mn = fminf(mn, x[e]);
        mx = fmaxf(mx, x[e]);
      }
  }
  mn = warp_min(mn);
  mx = warp_max(mx);
  // bisection over the values with count(s >= lo) > n > count(s >= hi); it ends at a
  // threshold with n scores, or where only equal scores are left between
  float lo = mn, hi = mx + fabsf(mx) * 2.4e-7f + 1e-37f, T = 0.f;
  bool found = false;
  if (count([&](float v) { return v >= hi; }) == n) {        // the forced blocks alone
    T = hi;
    found = true;
  }
  int clo = nT, chi = 0;
  for (int it = 0; it < 64 && !found; ++it) {
    // the middle in every third step, between where the counts say n would lie
    const float w = it % 3 == 2 ? 0.5f : fminf(fmaxf((float)(clo - n) / (float)(clo - chi), 0.06f), 0.94f);
    const float mid = lo + w * (hi - lo);
    if (!(mid > lo && mid < hi)) break;
    const int c = count([&](float v) { return v >= mid; });
    if (c == n) {
      T = mid;
      found = true;
    } else if (c > n) {
      lo = mid;
      clo = c;
    } else {
      hi = mid;
      chi = c;
    }
  }
  // a: the smallest kept, b: the largest left out (where no threshold was found, b >= a)
  const float split = found ? T : hi;
  float a = INFINITY, b = -INFINITY;
#pragma unroll 4
  for (int t = 0; t < nv; ++t) {
    const float4 v = s4[t * 32];
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (x[e] >= split)
        a = fminf(a, x[e]);
      else
        b = fmaxf(b, x[e]);
    }
  }
  b = warp_max(b);
  a = found ? warp_min(a) : lo;
  if (found && a - b > 2.f * E) {
    write_list(p, bh, i, lane, [&](int j0) {
      return mask4(*reinterpret_cast<const float4*>(s + j0), [&](float v) { return v >= T; });
    });
    return true;
  }
  const float from = a - 2.f * E, to = b + 2.f * E;
  const int above = count([&](float v) { return v > to; });
  auto is_open = [&](float v) { return v >= from && v <= to; };
  const int open = count(is_open);
  if (open > 32) return false;
  // lane r computes the r-th open block's score in fp64
  int seen = 0;
  for (int t = 0; t < nv; ++t) {
    const unsigned m = mask4(s4[t * 32], is_open);
    int total, at = seen + lane_prefix(m, lane, total);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m >> e & 1u) cand[at++] = t * 128 + 4 * lane + e;
    seen += total;
  }
  __syncwarp();
  const double v = lane < open ? exact_score<D>(qrow, kp + (size_t)cand[lane] * D) : -INFINITY;
  int rank = 0;
  for (int r = 0; r < open; ++r) {
    const double o = __shfl_sync(0xffffffffu, v, r);
    rank += o > v || (o == v && r < lane) ? 1 : 0;
  }
  const unsigned kept = __ballot_sync(0xffffffffu, lane < open && rank < n - above);
  int base = 0;
  write_list(p, bh, i, lane, [&](int j0) {
    const float4 x = *reinterpret_cast<const float4*>(s + j0);
    const unsigned m = mask4(x, is_open);
    unsigned take = mask4(x, [&](float y) { return y > to; });
    int total, at = base + lane_prefix(m, lane, total);
    base += total;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m >> e & 1u) take |= (kept >> at++ & 1u) << e;
    return take;
  });
  return true;
}

// grid (ceil(nT / ROWS), BH)
template <int D, int RT, int WR>
__global__ void __launch_bounds__(kScoreThreads, WR == 1 ? 1 : 3) score_select_kernel(const SelectParams p) {
  using C = ScoreCfg<RT, WR>;
  extern __shared__ __align__(16) unsigned char sm[];
  __shared__ float kmax_part[kScoreThreads / 32];
  __shared__ int later[C::ROWS];                 // rows for the second pass
  __shared__ int cand[kScoreThreads / 32][32];
  float* tile = reinterpret_cast<float*>(sm);
  float* scores = reinterpret_cast<float*>(sm + C::tiles(p.nTp));
  const int nT = p.nT, bh = blockIdx.y, i0 = blockIdx.x * C::ROWS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = (warp % WR) * 4 * RT + (lane >> 3) * RT;    // this thread's rows and first key of a tile
  const int key0 = (warp / WR) * 32 + (lane & 7);
  const float* qp = p.pooled + (size_t)bh * nT * D;
  const float* kp = p.pooled + ((size_t)gridDim.y + bh) * nT * D;

  // the largest norm of the head's pooled keys, for the error bound
  float km = 0.f;
  for (int j = threadIdx.x; j < nT; j += kScoreThreads) km = fmaxf(km, p.norms[((size_t)gridDim.y + bh) * nT + j]);
  km = warp_max(km);
  if (lane == 0) kmax_part[warp] = km;
  for (int r = threadIdx.x; r < C::ROWS; r += kScoreThreads) later[r] = 0;

  constexpr int CHUNKS = D / kDepth;
  const int ntiles = (nT + C::KEYS - 1) / C::KEYS, total = ntiles * CHUNKS;
  auto fetch = [&](int x) {                       // tile x: keys x / CHUNKS, channels x % CHUNKS
    float* dst = tile + x % kStages * C::TILE;
    const int j0 = x / CHUNKS * C::KEYS, c0 = x % CHUNKS * kDepth;
    for (int e = threadIdx.x; e < (C::KEYS + C::ROWS) * (kDepth / 4); e += kScoreThreads) {
      const int row = e / (kDepth / 4), part = e % (kDepth / 4);
      const bool is_k = row < C::KEYS;
      const int j = is_k ? j0 + row : i0 + row - C::KEYS;
      const bool live = j < nT;
      cp_async16(dst + row * kTileRow + part * 4, (is_k ? kp : qp) + (size_t)(live ? j : 0) * D + c0 + part * 4, live);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(0);
  if (total > 1) fetch(1);
  float2 tot[RT][4];
  for (int x = 0; x < total; ++x) {
    if (x % CHUNKS == 0)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int y = 0; y < 4; ++y) tot[r][y] = make_float2(0.f, 0.f);
    if (x + 1 < total)
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();                              // tile x has landed, tile x - 1 is read
    if (x + 2 < total) fetch(x + 2);
    const float* kt = tile + x % kStages * C::TILE;
    const float* qt = kt + C::KEYS * kTileRow;
    float2 acc[RT][4];
#pragma unroll
    for (int c = 0; c < kDepth; c += 4) {
      float4 a[RT], b[4];
#pragma unroll
      for (int r = 0; r < RT; ++r) a[r] = *reinterpret_cast<const float4*>(qt + (row0 + r) * kTileRow + c);
#pragma unroll
      for (int y = 0; y < 4; ++y) b[y] = *reinterpret_cast<const float4*>(kt + (key0 + y * 8) * kTileRow + c);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float2 z = c == 0 ? make_float2(0.f, 0.f) : acc[r][y];
          acc[r][y] = ffma2v(make_float2(a[r].x, a[r].y), make_float2(b[y].x, b[y].y), z);
          acc[r][y] = ffma2v(make_float2(a[r].z, a[r].w), make_float2(b[y].z, b[y].w), acc[r][y]);
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int y = 0; y < 4; ++y) tot[r][y] = fadd2(tot[r][y], acc[r][y]);
    if (x % CHUNKS == CHUNKS - 1) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int j = x / CHUNKS * C::KEYS + key0 + y * 8, i = i0 + row0 + r;
          if (j < p.nTp) {
            const float v = tot[r][y].x + tot[r][y].y;
            const bool forced = j < nT && p.forced(i, j);
            if (!forced && !(fabsf(v) < INFINITY)) later[row0 + r] = 1;
            scores[(size_t)(row0 + r) * p.nTp + j] = j >= nT ? -INFINITY : forced ? INFINITY : v;
          }
        }
    }
  }
  __syncthreads();
  km = kmax_part[0];
#pragma unroll
  for (int w = 1; w < kScoreThreads / 32; ++w) km = fmaxf(km, kmax_part[w]);

  for (int rr = warp; rr < C::ROWS; rr += kScoreThreads / 32) {
    const int i = i0 + rr;
    if (i >= nT) continue;
    // 20 roundings of the largest possible sum of magnitudes, and what subnormal products lose
    const float E = 20.f * 5.9604645e-8f * p.norms[(size_t)bh * nT + i] * km + 1e-37f;
    const bool sure = later[rr] == 0 && E < 1e37f &&
                      select_row<D>(p, bh, i, lane, scores + (size_t)rr * p.nTp, E, qp + (size_t)i * D, kp, cand[warp]);
    __syncwarp();
    if (lane == 0) later[rr] = sure ? 0 : 1;
  }
  __syncthreads();

  // second pass: a whole row in fp64
  uint32_t* hi = reinterpret_cast<uint32_t*>(sm);
  uint32_t* lo = hi + p.nTp;
  for (int rr = 0; rr < C::ROWS; ++rr) {
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

template <int D, int RT, int WR>
cudaError_t score_launch(const SelectParams& p, int BH, cudaStream_t stream) {
  using C = ScoreCfg<RT, WR>;
  auto kern = score_select_kernel<D, RT, WR>;
  const int smem = (int)C::smem(p.nTp);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3((p.nT + C::ROWS - 1) / C::ROWS, BH), kScoreThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

constexpr size_t kSmemMax = 232448 - 2048;       // beside the static arrays
// 4-row CTAs hold the longest rows
static_assert(ScoreCfg<1, 1>::smem(SAGE_SELECT_MAX_BLOCKS) <= kSmemMax, "the longest row must fit in shared memory");

template <int D>
cudaError_t select_d(const void* q, const void* k, int BH, int N, int keep, int first, int window, int* lists,
                     int* counts, float* pooled, cudaStream_t stream) {
  const int nT = num_tiles(N);
  float* norms = pooled + 2 * (size_t)BH * nT * D;
  pool_blocks_kernel<D><<<dim3(nT, BH, 2), kPoolThreads, 0, stream>>>(static_cast<const uint4*>(q),
                                                                      static_cast<const uint4*>(k), N, nT, pooled,
                                                                      norms);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const SelectParams p{pooled, norms, nT, (nT + 127) & ~127, keep, first, window, lists, counts};
  // sixteen rows a CTA while their scores fit beside the tiles, else four
  if (ScoreCfg<2, 2>::smem(p.nTp) <= kSmemMax) return score_launch<D, 2, 2>(p, BH, stream);
  return score_launch<D, 1, 1>(p, BH, stream);
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

// pooled means and their norms
size_t select_scratch_bytes(int BH, int N, int d) {
  return align_up(2 * (size_t)BH * num_tiles(N) * (d + 1) * 4, 256);
}

cudaError_t launch_select_blocks(const void* q, const void* k, int BH, int N, int d, int keep, int first, int window,
                                 int* lists, int* counts, void* scratch, cudaStream_t stream) {
  float* pooled = static_cast<float*>(scratch);
  return d == 128 ? select_d<128>(q, k, BH, N, keep, first, window, lists, counts, pooled, stream)
                  : select_d<64>(q, k, BH, N, keep, first, window, lists, counts, pooled, stream);
}

}  // namespace sage
