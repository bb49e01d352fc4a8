// select.cu -- the key blocks each query block attends to, chosen by a cheap
// score.
//
//   qbar_i, kbar_j = mean over the real rows of a 128-token block: exact sums
//                    in fp64 (128 bf16 values span far less than 53 bits),
//                    divided in fp64, rounded once to fp32;
//   s_ij           = sum_c qbar_i[c] * kbar_j[c] in fp64;
//   kept           = the `keep` largest s_ij of a row, ties to the lower j;
//                    blocks j < first and |i - j| <= window rank above all.
// fp64 because the result is a set: with fp32 sums a run over the 720p sequence
// (23,640 rows) meets pairs at the border whose order the rounding decides.
//
// Two kernels.  pool: one CTA per (block, head, tensor), HBM-bound, q and k are
// read once.  score: one CTA per (R query blocks, head) forms its rows of
// scores against every key block of the head in shared memory (the score matrix
// never reaches HBM), then one warp per row finds the keep-th largest by
// bisection on the bits of the ordered scores and writes the kept indices
// ascending.
#include <cuda_bf16.h>
#include <cstdint>

#include "../../include/sage_sparse.h"
#include "internal.h"
#include "sm100.cuh"

namespace sage {

namespace {

constexpr int kPoolThreads = 256;

// grid (nT, BH, 2): z = 0 pools q, z = 1 pools k; out [2][BH][nT][D]
template <int D>
__global__ void __launch_bounds__(kPoolThreads) pool_blocks_kernel(const uint4* __restrict__ q,
                                                                   const uint4* __restrict__ k, int N, int nT,
                                                                   float* __restrict__ pooled) {
  constexpr int V8 = D / 8, GROUPS = kPoolThreads / V8, PER_T = kTile / GROUPS;
  __shared__ double part[GROUPS][D + 2];
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
    const long long out = (((long long)blockIdx.z * gridDim.y + bh) * nT + blk) * D + threadIdx.x;
    if (SAGE_DCHECK(out, 2LL * gridDim.y * nT * D, kSitePoolOut)) pooled[out] = __double2float_rn(t / (double)nr);
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

constexpr int kScoreThreads = 256;
constexpr int kKeyTile = 256;              // key blocks of one inner tile
constexpr int kDepth = 16;                 // channels of one inner tile
constexpr int kTileRow = kDepth + 2;       // doubles; 144-byte rows keep 16-byte reads of 8 rows conflict-free

// Shared memory: k tile [256][18] and q tile [R][18] doubles, then the scores of
// R rows as two arrays of 32-bit halves, [R][nTp] each.
template <int RT>
__host__ __device__ constexpr size_t score_smem(int nTp) {
  return sizeof(double) * (size_t)(kKeyTile + 4 * RT) * kTileRow + 2 * sizeof(uint32_t) * (size_t)(4 * RT) * nTp;
}

// One warp: how many of n values v(j) satisfy v(j) >= t
__device__ __forceinline__ int count_ge(const uint32_t* v, int n, uint32_t t, int lane) {
  int c = 0;
  for (int j = lane; j < n; j += 32) c += v[j] >= t ? 1 : 0;
  return __reduce_add_sync(0xffffffffu, c);
}

// grid (ceil(nT / R), BH), R = 4 * RT rows.  Thread (row group 0..3, key lane):
// a warp covers the R rows x 32 keys, eight warps 256 keys.
template <int D, int RT>
__global__ void __launch_bounds__(kScoreThreads) score_select_kernel(const float* __restrict__ pooled, int nT, int nTp,
                                                                     int keep, int first, int window,
                                                                     int* __restrict__ lists, int* __restrict__ counts) {
  constexpr int R = 4 * RT;
  extern __shared__ __align__(16) unsigned char sm[];
  double* kt = reinterpret_cast<double*>(sm);
  double* qt = kt + kKeyTile * kTileRow;
  uint32_t* hi = reinterpret_cast<uint32_t*>(qt + R * kTileRow);
  uint32_t* lo = hi + (size_t)R * nTp;
  const int bh = blockIdx.y, i0 = blockIdx.x * R;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = lane >> 3, kl = lane & 7;
  const float* qp = pooled + (size_t)bh * nT * D;
  const float* kp = pooled + ((size_t)gridDim.y + bh) * nT * D;

  for (int j0 = 0; j0 < nT; j0 += kKeyTile) {
    double acc[RT][4];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[a][b] = 0.0;
    for (int c0 = 0; c0 < D; c0 += kDepth) {
      __syncthreads();
      // 4 float4 a key row of the tile, key rows behind nT as zeros
      for (int e = threadIdx.x; e < (kKeyTile + R) * (kDepth / 4); e += kScoreThreads) {
        const int row = e / (kDepth / 4), part = e % (kDepth / 4);
        const bool is_k = row < kKeyTile;
        const int j = is_k ? j0 + row : i0 + row - kKeyTile;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < nT) x = *reinterpret_cast<const float4*>((is_k ? kp : qp) + (size_t)j * D + c0 + part * 4);
        double* dst = kt + row * kTileRow + part * 4;     // the q tile follows the k tile
        dst[0] = x.x; dst[1] = x.y; dst[2] = x.z; dst[3] = x.w;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kDepth; c += 2) {
        double2 a[RT], b[4];
#pragma unroll
        for (int x = 0; x < RT; ++x) a[x] = *reinterpret_cast<const double2*>(qt + (rg * RT + x) * kTileRow + c);
#pragma unroll
        for (int x = 0; x < 4; ++x) b[x] = *reinterpret_cast<const double2*>(kt + (warp * 32 + x * 8 + kl) * kTileRow + c);
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            acc[x][y] = fma(a[x].x, b[y].x, acc[x][y]);
            acc[x][y] = fma(a[x].y, b[y].y, acc[x][y]);
          }
      }
    }
#pragma unroll
    for (int x = 0; x < RT; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int j = j0 + warp * 32 + y * 8 + kl, i = i0 + rg * RT + x;
        if (j < nT) {
          const bool forced = j < first || (window >= 0 && abs(i - j) <= window);
          const unsigned long long o = forced ? ~0ull : ordered_bits(acc[x][y]);
          hi[(rg * RT + x) * nTp + j] = (uint32_t)(o >> 32);
          lo[(rg * RT + x) * nTp + j] = (uint32_t)o;
        }
      }
  }
  __syncthreads();

  // one warp per row
  const long long ext = (long long)gridDim.y * nT * keep;
  (void)ext;
  for (int rr = warp; rr < R; rr += kScoreThreads / 32) {
    const int i = i0 + rr;
    if (i >= nT) continue;
    const uint32_t* h = hi + (size_t)rr * nTp;
    const uint32_t* w = lo + (size_t)rr * nTp;
    const int n = min(keep, nT);
    // The kept set is {hi > th} plus, among hi == th, the `need` largest by
    // (lo descending, j ascending): {lo > tl} plus the first `ties` of lo == tl.
    // th is built bit by bit as the largest value with at least n scores at or
    // above it; once exactly n are, the set is known.
    uint32_t th = 0, tl = 0;
    int ge = nT;                                   // scores with hi >= th
    for (int bit = 31; bit >= 0 && ge != n; --bit) {
      const uint32_t t = th | (1u << bit);
      const int c = count_ge(h, nT, t, lane);
      if (c >= n) {
        th = t;
        ge = c;
      }
    }
    int ties = nT;
    if (ge != n) {                                 // several scores share the high half at the border
      int above = 0;
      for (int j = lane; j < nT; j += 32) above += h[j] > th ? 1 : 0;
      const int need = n - __reduce_add_sync(0xffffffffu, above);
      int eq = ge - (n - need);                    // with hi == th and lo >= tl
      for (int bit = 31; bit >= 0 && eq != need; --bit) {
        const uint32_t t = tl | (1u << bit);
        int c = 0;
        for (int j = lane; j < nT; j += 32) c += h[j] == th && w[j] >= t ? 1 : 0;
        c = __reduce_add_sync(0xffffffffu, c);
        if (c >= need) {
          tl = t;
          eq = c;
        }
      }
      if (eq != need) {                            // full ties: the lowest j first
        int gt = 0;
        for (int j = lane; j < nT; j += 32) gt += h[j] == th && w[j] > tl ? 1 : 0;
        ties = need - __reduce_add_sync(0xffffffffu, gt);
      }
    }
    const long long row = ((long long)bh * nT + i) * keep;
    int done = 0, tied = 0;
    for (int jb = 0; jb < nT; jb += 32) {
      const int j = jb + lane;
      const uint32_t hv = j < nT ? h[j] : 0u, lv = j < nT ? w[j] : 0u;
      const bool in = j < nT;
      const bool tie = in && hv == th && lv == tl;
      const unsigned tm = __ballot_sync(0xffffffffu, tie);
      const bool take = in && (hv > th || (hv == th && lv > tl) ||
                               (tie && tied + __popc(tm & ((1u << lane) - 1u)) < ties));
      const unsigned m = __ballot_sync(0xffffffffu, take);
      const int at = done + __popc(m & ((1u << lane) - 1u));
      if (take && at < keep && SAGE_DCHECK(row + at, ext, kSiteSelectOut)) lists[row + at] = j;
      done += __popc(m);
      tied += __popc(tm);
    }
    for (int s = done + lane; s < keep; s += 32)
      if (SAGE_DCHECK(row + s, ext, kSiteSelectOut)) lists[row + s] = -1;
    if (lane == 0) counts[(long long)bh * nT + i] = done;
  }
}

template <int D, int RT>
cudaError_t score_launch(const float* pooled, int BH, int nT, int keep, int first, int window, int* lists, int* counts,
                         cudaStream_t stream) {
  const int nTp = (nT + 31) & ~31;
  const size_t smem = score_smem<RT>(nTp);
  auto kern = score_select_kernel<D, RT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3((nT + 4 * RT - 1) / (4 * RT), BH), kScoreThreads, smem, stream>>>(pooled, nT, nTp, keep, first, window,
                                                                                lists, counts);
  return cudaGetLastError();
}

constexpr size_t kSmemMax = 232448;
// 4-row CTAs hold the longest rows
static_assert(score_smem<1>(SAGE_SELECT_MAX_BLOCKS) <= kSmemMax, "the longest row must fit in shared memory");

template <int D>
cudaError_t select_d(const void* q, const void* k, int BH, int N, int keep, int first, int window, int* lists,
                     int* counts, float* pooled, cudaStream_t stream) {
  const int nT = num_tiles(N);
  pool_blocks_kernel<D><<<dim3(nT, BH, 2), kPoolThreads, 0, stream>>>(static_cast<const uint4*>(q),
                                                                      static_cast<const uint4*>(k), N, nT, pooled);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // sixteen rows a CTA while their scores fit beside the tiles, else four
  if (score_smem<4>((nT + 31) & ~31) <= kSmemMax)
    return score_launch<D, 4>(pooled, BH, nT, keep, first, window, lists, counts, stream);
  return score_launch<D, 1>(pooled, BH, nT, keep, first, window, lists, counts, stream);
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

size_t select_scratch_bytes(int BH, int N, int d) { return align_up(2 * (size_t)BH * num_tiles(N) * d * 4, 256); }

cudaError_t launch_select_blocks(const void* q, const void* k, int BH, int N, int d, int keep, int first, int window,
                                 int* lists, int* counts, void* scratch, cudaStream_t stream) {
  float* pooled = static_cast<float*>(scratch);
  return d == 128 ? select_d<128>(q, k, BH, N, keep, first, window, lists, counts, pooled, stream)
                  : select_d<64>(q, k, BH, N, keep, first, window, lists, counts, pooled, stream);
}

}  // namespace sage
