// Weights of the default maths widened to BF16 in registers, and the
// weight-streaming dot product that the products of few rows share.
//
// Without the fast-math flag the pages' runtime widens the 8-bit and 4-bit
// weights to 16 bits as it multiplies (Lernex/Metis-1.6-Logos-FP8, "What
// --fast-math does"; Lernex/Metis-1.6-Praxis-NVFP4, "What --fast-math does").
// Every format's scaled or unscaled value is exact in BF16:
//   FP8    dec(E4M3): 4 significant bits. The row's float32 scale stays in
//          the epilogue.
//   MXFP4  dec(E2M1) * 2^(e - 127): 2 significant bits, the block exponent
//          applied by the conversion instruction itself. Exact for e = 0 .. 252
//          (2^-128 is a subnormal BF16; the quantiser writes no larger e); at
//          253 and 254 a value of 2^128 or more is infinite, as in float32.
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

// LDS written and read by the lanes of one wave: the hardware keeps a wave's
// LDS accesses in order, this keeps the compiler to it.
__device__ inline void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A mask of the lowest n bytes of a dword: none for n <= 0, all for n >= 4.
__device__ inline uint32_t low_bytes(int n) { return n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u; }

// The block scales of U consecutive steps of NR sets of 16 weight rows. Read
// where they are used they would be one or two bytes a lane, 16 cache lines
// per load for 64 or 128 bytes; instead lane 16 g + r loads 16 bytes of row r
// of set g / kPieces at once, and hands them out through 1 KB of LDS that the
// wave keeps for itself. Scale rows start at any byte: the dwords around the
// piece are loaded and shifted (a dword that holds a byte of the tensor can
// always be read).
template <int F, int NR, int U>
struct BlockScales {
  static constexpr bool kAny = F != kFmtFp8;
  static constexpr int kStepBytes = kAny ? WideFmt<F>::kStepK / WideFmt<F>::kBlock : 0;
  static constexpr int kPieces = U * kStepBytes > 16 ? U * kStepBytes / 16 : 1;
  static constexpr int kLds = kAny ? 1024 : 16;  // bytes of LDS a wave needs
  static_assert(NR * kPieces <= 4, "a wave's 64 lanes load all pieces at once");
  v4i q;
  uint32_t top, shift;

  // off(a): byte offset in r of set a's first scale of these steps, for this
  // lane's row; r begins at a multiple of 16.
  template <class OFF>
  __device__ inline void load(__amdgpu_buffer_rsrc_t r, const OFF& off) {
    if constexpr (kAny) {
      const int g = (threadIdx.x & 63) >> 4;
      uint32_t at = kOutOfRange;
#pragma unroll
      for (int a = 0; a < NR; ++a)
        if (g / kPieces == a) at = off(a) + (uint32_t)(g % kPieces) * 16u;
      shift = at & 3u;
      q = buffer_load16(r, at & ~3u);
      top = __builtin_amdgcn_raw_buffer_load_b32(r, (at & ~3u) + 16u, 0, 0);
    }
  }

  // To the wave's LDS; the scales of step u, set a are then at get(). `bytes`:
  // what is left of the row; past its end a scale is 0, not the next row's,
  // whose NaN would be one here too although the codes there count as 0.
  __device__ inline void spread(uint8_t* lds, int bytes) const {
    if constexpr (kAny) {
      const uint32_t d[5] = {(uint32_t)q.x, (uint32_t)q.y, (uint32_t)q.z, (uint32_t)q.w, top};
      v4i o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = (int)__builtin_amdgcn_alignbyte(d[i + 1], d[i], shift);
      const int left = bytes - ((threadIdx.x & 63) >> 4) % kPieces * 16;
      if (left < 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] &= (int)low_bytes(left - 4 * i);
      }
      wave_lds_order();
      *reinterpret_cast<v4i*>(lds + (threadIdx.x & 63) * 16) = o;
      wave_lds_order();
    }
  }

  static __device__ inline uint32_t get(const uint8_t* lds, int u, int a) {
    if constexpr (kAny) {
      const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
      const int at = u * kStepBytes;  // g's bytes follow: never past a 16-byte piece
      const uint8_t* s = lds + (r16 + 16 * (a * kPieces + at / 16)) * 16 + at % 16;
      if constexpr (F == kFmtMxfp4)
        return s[g];
      else
        return reinterpret_cast<const uint16_t*>(s)[g];
    }
    return 0;
  }
};

// A resource over the scale rows of one matrix that begins at any byte:
// `skew` is where the matrix begins in it.
__device__ inline __amdgpu_buffer_rsrc_t scale_rsrc(const void* base, int64_t bytes, uint32_t* skew) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(base);
  *skew = (uint32_t)(b & 15u);
  return make_rsrc(reinterpret_cast<const void*>(b & ~(uintptr_t)15), (bytes + *skew + 3) & ~(int64_t)3);
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

// acc[a][t] += W[16 rows of set a][K] . X[16 rows of tile t][K]^T over `steps`
// K steps from this lane's kbase on. wrow / srow: byte offsets of this lane's
// row of each set in rW / rS; xrow: of its X row (kOutOfRange for an empty
// column; any offset from there on reads zeros). U steps' loads are issued
// together ahead of their MFMAs: bytes in flight are what a weight stream
// needs. lds: BlockScales::kLds bytes of this wave.
template <int F, int NR, int NT, int U>
__device__ inline void stream_dot(__amdgpu_buffer_rsrc_t rW, __amdgpu_buffer_rsrc_t rS, const uint32_t (&wrow)[NR],
                                  const uint32_t (&srow)[NR], __amdgpu_buffer_rsrc_t rX, const uint32_t (&xrow)[NT],
                                  int K, int kbase, int steps, uint8_t* lds, v4f (&acc)[NR][NT]) {
  using W = WideFmt<F>;
  using S = BlockScales<F, NR, U>;
  const int g = (threadIdx.x & 63) >> 4;
  for (int kt = 0; kt < steps; kt += U) {
    v4i w[U][NR], x[U][NT][W::kMfma];
    S sc;
    const int k0 = kbase + kt * W::kStepK;
    sc.load(rS, [&](int a) { return k0 < K ? srow[a] + (uint32_t)(k0 / W::kBlock) : kOutOfRange; });
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ku = k0 + u * W::kStepK;
      const int kw = ku + W::kLaneK * g;  // K is a multiple of kLaneK: a lane is all in or all out
      const bool live = kt + u < steps && kw < K;
#pragma unroll
      for (int a = 0; a < NR; ++a) w[u][a] = buffer_load16(rW, live ? wrow[a] + (uint32_t)W::row_bytes(kw) : kOutOfRange);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < W::kMfma; ++i)
          x[u][t][i] = buffer_load16(rX, live ? xrow[t] + 2u * (uint32_t)kw + 16u * i : kOutOfRange);
    }
    __builtin_amdgcn_sched_barrier(0);
    sc.spread(lds, (K - k0) / W::kBlock);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t s[NR];
#pragma unroll
      for (int a = 0; a < NR; ++a) s[a] = S::get(lds, u, a);
#pragma unroll
      for (int i = 0; i < W::kMfma; ++i)
#pragma unroll
        for (int a = 0; a < NR; ++a) {
          const v4i b = widen_part<F>(w[u][a], s[a], i);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[a][t] = mfma_16x16x32_bf16(b, x[u][t][i], acc[a][t]);
        }
    }
  }
}

}  // namespace w8a8
