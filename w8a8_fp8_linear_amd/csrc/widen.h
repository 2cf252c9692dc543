// Weights of the default maths widened to BF16 in registers, and the
// weight-streaming dot product that the few-token kernels share.
//
// Without the fast-math flag the pages' runtime widens the 8-bit and 4-bit
// weights to 16 bits as it multiplies (Lernex/Metis-1.6-Logos-FP8, "What
// --fast-math does"; Lernex/Metis-1.6-Praxis-NVFP4, "What --fast-math does").
// Every format's scaled or unscaled value is exact in BF16:
//   FP8    dec(E4M3): 4 significant bits. The row's float32 scale stays in
//          the epilogue.
//   MXFP4  dec(E2M1) * 2^(e - 127): 2 significant bits, the block exponent
//          applied by the conversion instruction itself.
//   NVFP4  dec(E2M1) * dec(E4M3 block scale): 2 + 4 = 6 significant bits at
//          most, magnitudes 2^-10 .. 2688. The matrix's float32 scale stays
//          in the epilogue.
// So products with BF16 activations are exact in float32, and the BF16
// matrix cores sum them in float32.
#pragma once

#include "device.h"

namespace w8a8 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

enum { kFmtFp8 = 0, kFmtMxfp4 = 1, kFmtNvfp4 = 2 };

__device__ inline v4f mfma_16x16x32_bf16(v4i a, v4i b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

// Two float32 values that are exact in BF16 -> their BF16 halves packed (a in the low half).
__device__ inline uint32_t pack_bf16(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// 8 E4M3 codes (bytes of w0 then w1, value 0 in the low byte) -> 8 BF16 values.
// The hardware conversion decodes E4M3 exactly into float32 (checked on gfx950
// against the format's definition for all 256 codes).
__device__ inline v4i widen8(uint32_t w0, uint32_t w1) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w0, false);
  const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w0, true);
  const auto c = __builtin_amdgcn_cvt_pk_f32_fp8((int)w1, false);
  const auto d = __builtin_amdgcn_cvt_pk_f32_fp8((int)w1, true);
  return v4i{(int)pack_bf16(a[0], a[1]), (int)pack_bf16(b[0], b[1]), (int)pack_bf16(c[0], c[1]),
             (int)pack_bf16(d[0], d[1])};
}

// 8 E2M1 codes (nibbles of w, value 0 in the low nibble) times 2^(e - 127),
// `scale` the float32 whose exponent field is e -> 8 BF16 values. The
// conversion multiplies by the power of two in its scale operand's exponent
// field (the mantissa is ignored), one instruction per two values.
__device__ inline v4i widen8_mx(uint32_t w, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return v4i{__builtin_bit_cast(int, a), __builtin_bit_cast(int, b), __builtin_bit_cast(int, c),
             __builtin_bit_cast(int, d)};
}

// 8 E2M1 codes times the float32 block scale s -> 8 BF16 values (exact).
__device__ inline v4i widen8_nv(uint32_t w, float s) {
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  return v4i{(int)pack_bf16(a[0] * s, a[1] * s), (int)pack_bf16(b[0] * s, b[1] * s),
             (int)pack_bf16(c[0] * s, c[1] * s), (int)pack_bf16(d[0] * s, d[1] * s)};
}

__device__ inline float mx_scale_value(uint32_t e) { return __uint_as_float(e << 23); }

// Geometry of one streamed step of a weight row: every lane of a wave loads
// 16 code bytes (lane = 16 g + r: row r, K values kLaneK * g .. of the step)
// and feeds kMfma 16x16x32 MFMAs, each with 8 of them.
template <int F>
struct WideFmt {
  static constexpr int kLaneK = F == kFmtFp8 ? 16 : 32;
  static constexpr int kStepK = 4 * kLaneK;
  static constexpr int kMfma = kLaneK / 8;
  static constexpr int kBlock = F == kFmtMxfp4 ? 32 : 16;      // K values per block scale
  __host__ __device__ static constexpr int64_t row_bytes(int64_t K) { return F == kFmtFp8 ? K : K / 2; }
  __host__ __device__ static constexpr int64_t row_scales(int64_t K) { return F == kFmtFp8 ? 0 : K / kBlock; }
};

// The lane's block scales of one step (K values k .. k + 31 of a row whose
// scale bytes start at srow): one E8M0 byte or two E4M3 bytes.
template <int F>
__device__ inline uint32_t load_block_scales(__amdgpu_buffer_rsrc_t r, uint32_t srow, int k, bool live) {
  if constexpr (F == kFmtMxfp4)
    return __builtin_amdgcn_raw_buffer_load_b8(r, live ? srow + (uint32_t)(k >> 5) : kOutOfRange, 0, 0);
  else if constexpr (F == kFmtNvfp4)
    return __builtin_amdgcn_raw_buffer_load_b16(r, live ? srow + (uint32_t)(k >> 4) : kOutOfRange, 0, 0);
  else
    return 0;
}

// The MFMA operand i (8 BF16 values) of a lane's 16 code bytes.
template <int F>
__device__ inline v4i widen_part(v4i w, uint32_t sc, int i) {
  const uint32_t d[4] = {(uint32_t)w.x, (uint32_t)w.y, (uint32_t)w.z, (uint32_t)w.w};
  if constexpr (F == kFmtFp8) {
    return widen8(d[2 * i], d[2 * i + 1]);
  } else if constexpr (F == kFmtMxfp4) {
    return widen8_mx(d[i], mx_scale_value(sc));
  } else {
    const auto s = __builtin_amdgcn_cvt_pk_f32_fp8((int)sc, false);  // the two blocks' E4M3 scales
    return widen8_nv(d[i], i < 2 ? s[0] : s[1]);
  }
}

// acc[a][t] += W[16 rows of set a][K] . X[16 rows of tile t][K]^T over the K
// steps first, first + stride, ... of ceil(K / kStepK). wrow / srow: byte
// offsets of this lane's row (lane % 16) of each set in rW / rS; xrow: of its
// X row (kOutOfRange for an empty column; any offset from there on reads
// zeros). U steps' loads are issued together ahead of their MFMAs: bytes in
// flight are what a weight stream needs.
template <int F, int NR, int NT, int U>
__device__ inline void stream_dot(__amdgpu_buffer_rsrc_t rW, __amdgpu_buffer_rsrc_t rS, const uint32_t (&wrow)[NR],
                                  const uint32_t (&srow)[NR], __amdgpu_buffer_rsrc_t rX, const uint32_t (&xrow)[NT],
                                  int K, int first, int stride, v4f (&acc)[NR][NT]) {
  using W = WideFmt<F>;
  const int g = (threadIdx.x & 63) >> 4;
  const int nk = (K + W::kStepK - 1) / W::kStepK;
  for (int kt = first; kt < nk; kt += stride * U) {
    v4i w[U][NR], x[U][NT][W::kMfma];
    uint32_t sc[U][NR];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (kt + stride * u) * W::kStepK + W::kLaneK * g;  // K is a multiple of kLaneK: all in or all out
      const bool live = kt + stride * u < nk && k < K;
#pragma unroll
      for (int a = 0; a < NR; ++a) {
        w[u][a] = buffer_load16(rW, live ? wrow[a] + (uint32_t)W::row_bytes(k) : kOutOfRange);
        sc[u][a] = load_block_scales<F>(rS, srow[a], k, live);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < W::kMfma; ++i)
          x[u][t][i] = buffer_load16(rX, live ? xrow[t] + (uint32_t)(2 * k + 16 * i) : kOutOfRange);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < W::kMfma; ++i)
#pragma unroll
        for (int a = 0; a < NR; ++a) {
          const v4i b = widen_part<F>(w[u][a], sc[u][a], i);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[a][t] = mfma_16x16x32_bf16(b, x[u][t][i], acc[a][t]);
        }
  }
}

}  // namespace w8a8
