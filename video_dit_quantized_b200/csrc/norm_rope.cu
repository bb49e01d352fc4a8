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
  long long tokens;      // B * N
  int N, B, H, norm, all_heads, w_f32, rope, begin, len, ranks;
  float eps;
};

__device__ __forceinline__ void nr_unpack(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// eight consecutive weights at vector index i
__device__ __forceinline__ void nr_weights(const void* w, int w_f32, int i, float (&x)[8]) {
  if (w_f32) {
    const float4 a = static_cast<const float4*>(w)[2 * i], b = static_cast<const float4*>(w)[2 * i + 1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    nr_unpack(static_cast<const uint4*>(w)[i], x);
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

// grid (ceil(tokens / (kNrThreads / TPT)), 2): y selects the tensor.
template <int D, int TPT, int CH>
__global__ void __launch_bounds__(kNrThreads) qk_norm_rope_kernel(const NrParams p, int first) {
  constexpr int L = D / 8;                 // lanes of one head
  static_assert(TPT % L == 0 && kNrThreads % TPT == 0, "a thread must see the same channels in every chunk");
  __shared__ float red[kNrThreads / 32];
  const long long tok = (long long)blockIdx.x * (kNrThreads / TPT) + threadIdx.x / TPT;
  if (tok >= p.tokens) return;             // whole warps leave together, and at TPT == 128 the whole block
  const NrTensor t = p.t[first + blockIdx.y];
  const int lane = threadIdx.x % TPT;
  const int nvec = p.H * L;
  const int b = (int)(tok / p.N), n = (int)(tok - (long long)b * p.N);
  const uint4* row = t.x + tok * t.stride8;

  uint4 raw[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = i * TPT + lane;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (c < nvec && SAGE_DCHECK(tok * t.stride8 + c, (p.tokens - 1) * t.stride8 + nvec, kSiteNormIn)) raw[i] = row[c];
  }

  // this thread's rotation factors: 4 pairs (interleaved) or 8 (halves)
  const int l = lane % L;
  const bool turn = p.rope != SAGE_ROPE_NONE && n >= p.begin && n - p.begin < p.len;
  float cs[8], sn[8];
  if (turn) {
    const long long base = (long long)(n - p.begin) * (D / 8);   // in float4: d / 2 floats a row
    if (SAGE_DCHECK(base + D / 8 - 1, (long long)p.len * (D / 8), kSiteNormTable)) {
      const int i0 = p.rope == SAGE_ROPE_INTERLEAVED ? l : 2 * (l % (L / 2));
      const float4 c0 = p.cos4[base + i0], s0 = p.sin4[base + i0];
      cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w;
      sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
      if (p.rope == SAGE_ROPE_HALF) {
        const float4 c1 = p.cos4[base + i0 + 1], s1 = p.sin4[base + i0 + 1];
        cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
        sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
      }
    }
  }

  float mu = 0.f, r = 1.f;                 // statistics over all heads
  if (p.norm != SAGE_NORM_NONE && p.all_heads) {
    const float cnt = (float)(p.H * D);
    if (p.norm == SAGE_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float x[8];
        nr_unpack(raw[i], x);
#pragma unroll
        for (int u = 0; u < 8; ++u) s += x[u];
      }
      mu = token_sum<TPT>(s, red) / cnt;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float x[8];
      nr_unpack(raw[i], x);
      if (i * TPT + lane < nvec)
#pragma unroll
        for (int u = 0; u < 8; ++u) s += (x[u] - mu) * (x[u] - mu);
    }
    r = inv_root(token_sum<TPT>(s, red) / cnt + p.eps);
  }

  float wv[8], bv[8];
  const bool has_w = t.w != nullptr, has_b = t.b != nullptr;
  if (!p.all_heads) {
    if (has_w) nr_weights(t.w, p.w_f32, l, wv);
    if (has_b) nr_weights(t.b, p.w_f32, l, bv);
  }
  const int Hl = p.ranks > 0 ? p.H / p.ranks : p.H;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = i * TPT + lane;
    float x[8];
    nr_unpack(raw[i], x);
    if (p.norm != SAGE_NORM_NONE && !p.all_heads) {
      mu = 0.f;
      if (p.norm == SAGE_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) s += x[u];
        mu = head_sum<L>(s) / (float)D;
      }
      float s = 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += (x[u] - mu) * (x[u] - mu);
      r = inv_root(head_sum<L>(s) / (float)D + p.eps);
    }
    if (p.norm != SAGE_NORM_NONE) {
      if (p.all_heads && c < nvec) {
        if (has_w) nr_weights(t.w, p.w_f32, c, wv);
        if (has_b) nr_weights(t.b, p.w_f32, c, bv);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        x[u] = (x[u] - mu) * r;
        if (has_w) x[u] *= wv[u];
        if (has_b) x[u] += bv[u];
      }
    }
    if (p.rope == SAGE_ROPE_INTERLEAVED) {
      if (turn)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float a0 = x[2 * u], a1 = x[2 * u + 1];
          x[2 * u] = a0 * cs[u] - a1 * sn[u];
          x[2 * u + 1] = a0 * sn[u] + a1 * cs[u];
        }
    } else if (p.rope == SAGE_ROPE_HALF) {
      // the partner channel c +- d/2 sits L/2 lanes away; every lane of the warp takes part
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float o = __shfl_xor_sync(0xffffffffu, x[u], L / 2);
        if (turn) x[u] = l < L / 2 ? x[u] * cs[u] - o * sn[u] : o * sn[u] + x[u] * cs[u];
      }
    }
    if (c < nvec) {
      const int h = c / L;
      long long out;                       // row of d channels
      if (p.ranks == 0) {
        out = ((long long)b * p.H + h) * p.N + n;
      } else {
        const int rk = h / Hl;
        out = (((long long)rk * p.B + b) * p.N + n) * Hl + (h - rk * Hl);
      }
      if (SAGE_DCHECK(out * L + l, p.tokens * nvec, kSiteNormOut))
        t.y[out * L + l] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                      pack_bf16x2(x[6], x[7]));
    }
  }
}

template <int D, int TPT, int CH>
cudaError_t nr_launch(const NrParams& p, int first, int tensors, cudaStream_t stream) {
  const long long per = kNrThreads / TPT;
  const dim3 grid((unsigned)((p.tokens + per - 1) / per), (unsigned)tensors);
  qk_norm_rope_kernel<D, TPT, CH><<<grid, kNrThreads, 0, stream>>>(p, first);
  return cudaGetLastError();
}

// Threads per token by the width: up to 2048 channels one warp holds the row
// (no block-wide sum), above that a block of four warps.
template <int D>
cudaError_t nr_dispatch(const NrParams& p, int first, int tensors, cudaStream_t stream) {
  const int nvec = p.H * (D / 8);
  if (nvec <= 2 * 32) return nr_launch<D, 32, 2>(p, first, tensors, stream);
  if (nvec <= 8 * 32) return nr_launch<D, 32, 8>(p, first, tensors, stream);
  if (nvec <= 5 * 128) return nr_launch<D, 128, 5>(p, first, tensors, stream);
  if (nvec <= 8 * 128) return nr_launch<D, 128, 8>(p, first, tensors, stream);
  return nr_launch<D, 128, 16>(p, first, tensors, stream);
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
  p.tokens = (long long)B * N;
  p.N = N;
  p.B = B;
  p.H = H;
  p.norm = norm;
  p.all_heads = all_heads;
  p.w_f32 = w_f32;
  p.rope = rope;
  p.begin = rope_begin;
  p.len = rope_len;
  p.ranks = ranks;
  p.eps = eps;
  const int first = q ? 0 : 1, tensors = (q ? 1 : 0) + (k ? 1 : 0);
  return d == 128 ? nr_dispatch<128>(p, first, tensors, stream) : nr_dispatch<64>(p, first, tensors, stream);
}

}  // namespace sage
