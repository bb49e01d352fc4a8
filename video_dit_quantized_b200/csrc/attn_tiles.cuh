// attn_tiles.cuh -- what the dense and the block-sparse attention kernels share:
// the CTA shape, the shared-memory tile formats and the tcgen05 issue loops of
// S = Q K^T and O += P V for one 128-key tile.
#pragma once
#include <cstdint>

#include "internal.h"
#include "sm100.cuh"

namespace sage {

namespace {

constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kTmemCols = 512;
// Register split: the kernel is compiled for kLaunchRegs per thread (384 threads,
// one CTA per SM); warpgroup 0 (producer, MMA, idle warps) drops to Cfg::REGS_LOW
// and the two softmax warpgroups rise to Cfg::REGS_HIGH, within 384 * 168.
constexpr int kLaunchRegs = 168;

// log2(e) / sqrt(d), formed in double and rounded once to fp32
__host__ __device__ constexpr float softmax_c(int d) {
  return d == 128 ? (float)(1.4426950408889634073599246810019 / 11.313708498984760390413509793678)
                  : (float)(1.4426950408889634073599246810019 / 8.0);
}

template <int D, bool QUANT>
struct Cfg {
  static constexpr int ELEM = QUANT ? 1 : 2;
  static constexpr int TILE_BYTES = 128 * D * ELEM;               // one Q, K or V tile
  static constexpr int P_BYTES = QUANT ? 128 * 128 : 0;           // one e4m3 P tile in smem
  static constexpr int STAGES = QUANT ? (D == 128 ? 4 : 8) : (D == 128 ? 2 : 3);
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + STAGES * TILE_BYTES;
  static constexpr int OFF_P = OFF_V + STAGES * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_P + 2 * P_BYTES;
  static constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;          // barriers + 1 KB alignment slack
  // Q/K operand rows in shared memory (bytes) and their swizzle
  static constexpr int QK_ROW = QUANT ? D : 128;                   // bf16: one 64-element atom
  static constexpr uint32_t QK_LAYOUT = (QUANT && D == 64) ? kLayoutSW64 : kLayoutSW128;
  static constexpr uint32_t QK_SBO = 8 * QK_ROW;
  static constexpr int QK_KSTEPS = QUANT ? D / 32 : D / 16;
  static constexpr int PV_KSTEPS = QUANT ? 128 / 32 : 128 / 16;
  static constexpr uint32_t IDESC_QK =
      QUANT ? make_idesc(kFmtS32Acc, kFmtS8, kFmtS8, 0, 128, 128) : make_idesc(kFmtF32Acc, kFmtBF16, kFmtBF16, 0, 128, 128);
  static constexpr uint32_t IDESC_PV =
      QUANT ? make_idesc(kFmtF32Acc, kFmtE4M3, kFmtE4M3, 0, 128, D) : make_idesc(kFmtF32Acc, kFmtBF16, kFmtBF16, 1, 128, D);
  static constexpr int KIND_QK = QUANT ? kKindI8 : kKindF16;
  static constexpr int REGS_LOW = QUANT ? 96 : 80;
  static constexpr int REGS_HIGH = QUANT ? 200 : 208;
  static_assert(128 * REGS_LOW + 256 * REGS_HIGH <= kThreads * kLaunchRegs, "register split exceeds the launch budget");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// S[tmem] = Q[smem] K[smem]^T for one 128x128 tile (K-major operands).
template <int D, bool QUANT>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t q_smem, uint32_t k_smem) {
  using C = Cfg<D, QUANT>;
#pragma unroll
  for (int s = 0; s < C::QK_KSTEPS; ++s) {
    // 32-byte K step; bf16 tiles hold 64-element (128-byte) atoms of 16 KB each
    const uint32_t off = QUANT ? s * 32 : (s / 4) * 16384 + (s % 4) * 32;
    const uint64_t a = make_sdesc(q_smem + off, 16, C::QK_SBO, C::QK_LAYOUT);
    const uint64_t b = make_sdesc(k_smem + off, 16, C::QK_SBO, C::QK_LAYOUT);
    mma_ss<C::KIND_QK>(d_tmem, a, b, C::IDESC_QK, s > 0 ? 1u : 0u);
  }
}

// QUANT: O[tmem] (+)= P8[smem] V8[smem] for one 128-key tile.  P tile [128 rows]
// [128 keys] e4m3 and V^T tile [D rows][128 keys] e4m3, both K-major with the
// 128-byte swizzle; 32-byte K steps.
template <int D>
__device__ __forceinline__ void issue_pv_quant(uint32_t d_tmem, uint32_t p_smem, uint32_t v_smem, uint32_t accumulate) {
  using C = Cfg<D, true>;
#pragma unroll
  for (int s = 0; s < C::PV_KSTEPS; ++s) {
    const uint64_t a = make_sdesc(p_smem + s * 32, 16, 1024, kLayoutSW128);
    const uint64_t b = make_sdesc(v_smem + s * 32, 16, 1024, kLayoutSW128);
    mma_ss<kKindF8F6F4>(d_tmem, a, b, C::IDESC_PV, (s > 0 || accumulate) ? 1u : 0u);
  }
}

// BF16: O[tmem] (+)= P[tmem] V[smem]; V tile [128 keys][D] stored as 64-channel
// atoms (16 KB each), MN-major; P bf16 in TMEM (64 columns).
template <int D>
__device__ __forceinline__ void issue_pv_bf16(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_smem, uint32_t accumulate) {
  using C = Cfg<D, false>;
#pragma unroll
  for (int s = 0; s < C::PV_KSTEPS; ++s) {
    const uint64_t b = make_sdesc(v_smem + s * 2048, 16384, 1024, kLayoutSW128);
    mma_ts<kKindF16>(d_tmem, p_tmem + s * 8, b, C::IDESC_PV, (s > 0 || accumulate) ? 1u : 0u);
  }
}

// One thread's 128-byte P row into a [128 x 128 B] tile with the 128-byte
// swizzle (16-byte chunk c of row r sits at chunk position c ^ (r % 8)); the
// tile base is 1024-byte aligned.
__device__ __forceinline__ void store_p_row(uint8_t* tile, int row, const uint32_t (&pk)[32]) {
  uint8_t* rp = tile + row * 128;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(rp + ((c ^ (row & 7)) << 4)) = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
}

}  // namespace

}  // namespace sage
