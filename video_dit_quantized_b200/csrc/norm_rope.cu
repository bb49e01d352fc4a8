// norm_rope.cu -- the norm of queries and keys with the position rotation in
// the same pass, written straight into the layout the attention path reads.
//
// Per token and tensor, x[h][c] (bf16):
//   RMS:    y = x * r * w,           r = 1 / sqrt(mean(x^2) + eps)
//   LAYER:  y = (x - mu) * r * w + b, r = 1 / sqrt(mean((x - mu)^2) + eps)
//   rotation of the channel pair (a, b) of pair index i at table row
//   n - begin:  a' = a cos - b sin,  b' = a sin + b cos
// over one head's d channels or over all H * d channels of the token.  All
// arithmetic in fp32 (the centred sum of squares of LAYER is a second pass over
// registers, not E[x^2] - mu^2, which loses the small variance of a large
// mean); one rounding to bf16 at the end.
//
// What bounds it: HBM.  Every element is read once and written once; the
// tables add d * 4 bytes a token, shared by the heads and the two tensors.  A
// token's row stays in registers between the sums and the rotation, so the
// norm over all heads needs no second read.  TPT threads own one token, each
// CH chunks of eight channels, TPT chunks apart, so a thread always sees the
// same channels of a head: its cos and sin values are read once a token.
// Instructions come next: at 24 an element (norm, weights and rotation as
// run-time choices inside the element loop, 64-bit token arithmetic) the kernel
// was issue bound, 4.3 TB/s at 1 x 75600 x 40 x 128; hence the scope and the
// pairing as template arguments, one form (x - mu) * r * w for both norms in packed
// pairs, and one block per token with no division: 547 to 581 us (0.82 to 0.87 of a copy).
#include <cuda_bf16.h>
#include <cstdint>

#include "../../include/sage_sparse.h"
#include "internal.h"
#include "sm100.cuh"

namespace sage {

namespace {

constexpr int kNrThreads = 128;

struct NrTensor {
  const uint4* x;        // row n of batch b at (b * N + n) * stride8
  long long stride8;     // row stride in 8-channel vectors
  uint4* y;
  const void* w;         // [d] or [H * d], bf16 or fp32, or null
  const void* b;
};

struct NrParams {
  NrTensor t[2];
  const float4* cos4;
  const float4* sin4;
  int B, N, H, norm, w_f32, begin, len, ranks;   // len 0: no rotation
  uint32_t rank_mul;     // ceil(2^16 / heads of a rank): h * rank_mul >> 16 = h / heads of a rank for h < 256
  double inv_width;      // 1 / (H * d)
  float inv_width_f32, eps;
};

__device__ __forceinline__ void nr_unpack(const uint4& u, float2 (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

// eight consecutive weights at vector index i
__device__ __forceinline__ void nr_weights(const void* w, int w_f32, int i, float2 (&x)[4]) {
  if (w_f32) {
    const float4 a = __ldg(static_cast<const float4*>(w) + 2 * i), b = __ldg(static_cast<const float4*>(w) + 2 * i + 1);
    x[0] = make_float2(a.x, a.y);
    x[1] = make_float2(a.z, a.w);
    x[2] = make_float2(b.x, b.y);
    x[3] = make_float2(b.z, b.w);
  } else {
    nr_unpack(__ldg(static_cast<const uint4*>(w) + i), x);
  }
}

// Sum over the threads that share one token (a warp, or the whole block).
template <int TPT>
__device__ __forceinline__ float token_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPT > 32) {
    const int w = threadIdx.x >> 5;
    __syncthreads();                       // red may still be read from the previous sum
    if ((threadIdx.x & 31) == 0) red[w] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < TPT / 32; ++i) v += red[i];
  }
  return v;
}

// Sum over the L consecutive lanes that hold one head of one token.
template <int L>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float inv_root(float v) { return v == 0.f ? 0.f : rsqrtf(v); }

// grid (ceil(N / TOKENS), tensors, B), TOKENS = kNrThreads / TPT.  Registers are left to the
// compiler: 78 to 96 at 5120 channels, no spills.  Held to six blocks per SM (over all heads) or five
// (per head), 1 x 75600 x 40 x 128 takes as long over all heads (548 us) and longer with half-split
// pairs, which then spill (754 us, so: 659), and per head (594, so: 541).
template <int D, int TPT, int CH, bool ALL, bool HALF>
__global__ void __launch_bounds__(kNrThreads) qk_norm_rope_kernel(const NrParams p, int first) {
  constexpr int L = D / 8;                 // lanes of one head
  constexpr int TOKENS = kNrThreads / TPT;
  constexpr int F = HALF ? 2 : 1;          // float4 of factors a thread needs: 8 pairs (halves) or 4
  static_assert(TPT % L == 0 && kNrThreads % TPT == 0, "a thread must see the same channels in every chunk");
  __shared__ float red[kNrThreads / 32];
  const int b = blockIdx.z, n = blockIdx.x * TOKENS + threadIdx.x / TPT;
  if (n >= p.N) return;                    // whole warps leave together, and at TPT == 128 the whole block
  const NrTensor t = p.t[first + blockIdx.y];
  const int lane = threadIdx.x % TPT;
  const int l = lane % L;
  const int nvec = p.H * L;
  const long long tokens = (long long)p.B * p.N, tok = (long long)b * p.N + n;
  (void)tokens;

  float2 x[CH][4];
  const uint4* row = t.x + tok * t.stride8 + lane;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (i * TPT + lane < nvec && SAGE_DCHECK(tok * t.stride8 + i * TPT + lane, (tokens - 1) * t.stride8 + nvec, kSiteNormIn))
      u = row[i * TPT];
    nr_unpack(u, x[i]);
  }
  // this thread's rotation factors
  const int at = n - p.begin;
  const bool turn = at >= 0 && at < p.len;
  float cs[4 * F], sn[4 * F];
  if (turn) {
    const long long base = (long long)at * (D / 8) + (HALF ? 2 * (l % (L / 2)) : l);   // in float4: d / 2 floats a row
#pragma unroll
    for (int f = 0; f < F; ++f)
      if (SAGE_DCHECK(base + f, (long long)p.len * (D / 8), kSiteNormTable)) {
        const float4 c4 = __ldg(p.cos4 + base + f), s4 = __ldg(p.sin4 + base + f);
        cs[4 * f] = c4.x; cs[4 * f + 1] = c4.y; cs[4 * f + 2] = c4.z; cs[4 * f + 3] = c4.w;
        sn[4 * f] = s4.x; sn[4 * f + 1] = s4.y; sn[4 * f + 2] = s4.z; sn[4 * f + 3] = s4.w;
      }
  }
  float2 wv[4], bv[4];
  if (!ALL) {
    if (t.w) nr_weights(t.w, p.w_f32, l, wv);
    if (t.b) nr_weights(t.b, p.w_f32, l, bv);
  }

  // x becomes x - mu, and y = (x - mu) * r before the weights: a vector without variance is
  // exactly 0, which x * r - mu * r, with mu * r rounded, is not.
  float r = 1.f;
  if (ALL && p.norm != SAGE_NORM_NONE) {
    float2 s = make_float2(0.f, 0.f);
    if (p.norm == SAGE_NORM_LAYER) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) s = fadd2(s, x[i][u]);
      // In fp64: for equal channels every partial sum is exact (at most 2^14 times a value of 8
      // bits) and the mean must be that value; times fp32's 1 / width it may be its neighbour.
      const float mu = __double2float_rn((double)token_sum<TPT>(s.x + s.y, red) * p.inv_width);
      const float2 m2 = make_float2(mu, mu);
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) x[i][u] = fsub2(x[i][u], m2);
      s = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (i * TPT + lane < nvec)
#pragma unroll
        for (int u = 0; u < 4; ++u) s = ffma2v(x[i][u], x[i][u], s);
    r = inv_root(token_sum<TPT>(s.x + s.y, red) * p.inv_width_f32 + p.eps);
  }

  // the first chunk's output vector; in the plain layout a chunk is TPT / L heads further
  const int h0 = lane / L;
  const int Hl = p.ranks > 0 ? p.H / p.ranks : p.H;
  const long long step = (long long)(TPT / L) * p.N * L;
  long long out = (((long long)b * p.H + h0) * p.N + n) * L + l;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = i * TPT + lane;
    if (!ALL && p.norm != SAGE_NORM_NONE) {
      float mu = 0.f;
      if (p.norm == SAGE_NORM_LAYER) {
        float2 s = fadd2(fadd2(x[i][0], x[i][1]), fadd2(x[i][2], x[i][3]));
        mu = head_sum<L>(s.x + s.y) * (1.f / (float)D);
      }
      const float2 m2 = make_float2(mu, mu);
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        x[i][u] = fsub2(x[i][u], m2);
        s = ffma2v(x[i][u], x[i][u], s);
      }
      r = inv_root(head_sum<L>(s.x + s.y) * (1.f / (float)D) + p.eps);
    }
    if (p.norm != SAGE_NORM_NONE) {
      if (ALL && c < nvec) {
        if (t.w) nr_weights(t.w, p.w_f32, c, wv);
        if (t.b) nr_weights(t.b, p.w_f32, c, bv);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) x[i][u] = fmul2(x[i][u], r);
      if (t.w)
#pragma unroll
        for (int u = 0; u < 4; ++u) x[i][u] = fmul2v(x[i][u], wv[u]);
      if (t.b)
#pragma unroll
        for (int u = 0; u < 4; ++u) x[i][u] = fadd2(x[i][u], bv[u]);
    }
    if constexpr (HALF) {
      // the partner channel c +- d/2 sits L/2 lanes away; every lane of the warp takes part
      const float sign = l < L / 2 ? -1.f : 1.f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float ox = __shfl_xor_sync(0xffffffffu, x[i][u].x, L / 2), oy = __shfl_xor_sync(0xffffffffu, x[i][u].y, L / 2);
        if (turn)
          x[i][u] = make_float2(x[i][u].x * cs[2 * u] + sign * ox * sn[2 * u],
                                x[i][u].y * cs[2 * u + 1] + sign * oy * sn[2 * u + 1]);
      }
    } else {
      if (turn)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          x[i][u] = make_float2(x[i][u].x * cs[u] - x[i][u].y * sn[u], x[i][u].x * sn[u] + x[i][u].y * cs[u]);
    }
    if (c < nvec) {
      if (p.ranks > 0) {
        const int h = h0 + i * (TPT / L), rk = (int)((uint32_t)h * p.rank_mul >> 16);
        out = ((((long long)rk * p.B + b) * p.N + n) * Hl + (h - rk * Hl)) * L + l;
      }
      if (SAGE_DCHECK(out, tokens * nvec, kSiteNormOut))
        t.y[out] = make_uint4(pack_bf16x2(x[i][0].x, x[i][0].y), pack_bf16x2(x[i][1].x, x[i][1].y),
                                      pack_bf16x2(x[i][2].x, x[i][2].y), pack_bf16x2(x[i][3].x, x[i][3].y));
    }
    out += step;
  }
}

template <int D, int TPT, int CH>
cudaError_t nr_launch(const NrParams& p, bool all, bool half, int first, int tensors, cudaStream_t stream) {
  constexpr int TOKENS = kNrThreads / TPT;
  const dim3 grid((unsigned)((p.N + TOKENS - 1) / TOKENS), (unsigned)tensors, (unsigned)p.B);
  if (all && half)
    qk_norm_rope_kernel<D, TPT, CH, true, true><<<grid, kNrThreads, 0, stream>>>(p, first);
  else if (all)
    qk_norm_rope_kernel<D, TPT, CH, true, false><<<grid, kNrThreads, 0, stream>>>(p, first);
  else if (half)
    qk_norm_rope_kernel<D, TPT, CH, false, true><<<grid, kNrThreads, 0, stream>>>(p, first);
  else
    qk_norm_rope_kernel<D, TPT, CH, false, false><<<grid, kNrThreads, 0, stream>>>(p, first);
  return cudaGetLastError();
}

// Threads per token by the width: up to 512 channels a warp (no block-wide sum), above
// that a block of four (a warp with eight chunks a thread took 146 us where the block
// with two takes 128: 2 x 17776 x 30 x 64, LAYER per head).
template <int D>
cudaError_t nr_dispatch(const NrParams& p, bool all, bool half, int first, int tensors, cudaStream_t stream) {
  const int nvec = p.H * (D / 8);
  if (nvec <= 2 * 32) return nr_launch<D, 32, 2>(p, all, half, first, tensors, stream);
  if (nvec <= 2 * 128) return nr_launch<D, 128, 2>(p, all, half, first, tensors, stream);
  if (nvec <= 5 * 128) return nr_launch<D, 128, 5>(p, all, half, first, tensors, stream);
  if (nvec <= 8 * 128) return nr_launch<D, 128, 8>(p, all, half, first, tensors, stream);
  return nr_launch<D, 128, 16>(p, all, half, first, tensors, stream);
}

}  // namespace

unsigned debug_take_norm_rope(unsigned long long* first) {
#ifdef SAGE_DEBUG
  return debug_take_tu(first);
#else
  (void)first;
  return 0;
#endif
}

cudaError_t launch_qk_norm_rope(const void* q, const void* k, long long q_stride, long long k_stride, const void* wq,
                                const void* bq, const void* wk, const void* bk, int w_f32, const float* cos_t,
                                const float* sin_t, int B, int N, int H, int d, int norm, int all_heads, float eps,
                                int rope, int rope_begin, int rope_len, void* q_out, void* k_out, int ranks,
                                cudaStream_t stream) {
  NrParams p;
  p.t[0] = NrTensor{static_cast<const uint4*>(q), q_stride / 8, static_cast<uint4*>(q_out), wq, bq};
  p.t[1] = NrTensor{static_cast<const uint4*>(k), k_stride / 8, static_cast<uint4*>(k_out), wk, bk};
  p.cos4 = reinterpret_cast<const float4*>(cos_t);
  p.sin4 = reinterpret_cast<const float4*>(sin_t);
  p.B = B;
  p.N = N;
  p.H = H;
  p.norm = norm;
  p.w_f32 = w_f32;
  p.begin = rope_begin;
  p.len = rope == SAGE_ROPE_NONE ? 0 : rope_len;
  p.ranks = ranks;
  const int Hl = ranks > 0 ? H / ranks : H;
  p.rank_mul = (65536u + Hl - 1) / Hl;
  p.inv_width = 1.0 / (H * d);
  p.inv_width_f32 = 1.f / (float)(H * d);
  p.eps = eps;
  const bool half = rope == SAGE_ROPE_HALF;
  const int first = q ? 0 : 1, tensors = (q ? 1 : 0) + (k ? 1 : 0);
  return d == 128 ? nr_dispatch<128>(p, all_heads, half, first, tensors, stream)
                  : nr_dispatch<64>(p, all_heads, half, first, tensors, stream);
}

}  // namespace sage
