// NVFP4: E2M1 values with one E4M3 scale per 16 consecutive inputs and one
// float32 scale per matrix (the pages' 4-bit checkpoint keeps one per expert;
// Lernex/Metis-1.6-Praxis-NVFP4, "What is in NVFP4"). Quantisation of a
// group [R, K] of BF16 values, every step rounded once:
//   g    = max(fl32(max|x| / 2688), 2^-96), 1 for an all-zero group
//          (2688 = 6 * 448: the largest block scale times the largest code)
//   s[b] = E4M3(min(fl32(fl32(max|x_b| / 6) / g), 448))
//   d    = fl32(dec(s[b]) * g)
//   q    = E2M1(fl32(x / d)), round to nearest, ties to even, saturating at
//          6; +-0 where d = 0
// and back: y = bf16(fl32(dec(q) * d)).
//
// The quantiser is bound by HBM: the group's maximum is needed before its
// first code, so x is read twice. nvfp4_amax leaves a maximum per chunk of a
// group (no atomics, nothing to clear), nvfp4_quant reduces the few chunk
// maxima of its group and quantises; it walks the chunks in the opposite
// order, so that what was read last is still in the 256 MB last-level cache.
#include "device.h"
#include "launch.h"

namespace w8a8 {
namespace {

constexpr int kChunk = 32768;  // values a workgroup reads
constexpr float kGscaleMin = 0x1p-96f;

__device__ inline float group_scale(uint32_t amax_bits) {
  if (amax_bits == 0) return 1.0f;
  return fmaxf(__uint_as_float(amax_bits << 16) / 2688.0f, kGscaleMin);
}

// fl32(x / d) for r = fl32(1 / d), both correctly rounded: one residual
// correction of x * r (Markstein's method). Exact where the quotient matters:
// d >= 2^-105 (g >= 2^-96, s >= 2^-9), so the residual of any quotient that
// does not round to code 0 is a normal number.
__device__ inline float quotient(float x, float d, float r) {
  const float q0 = x * r;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q0, d, x), r, q0), x);
}

__device__ inline uint32_t block_max(uint32_t v, int mask) {
#pragma unroll
  for (int m = 1; m <= mask; m <<= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, m, 64);
    v = v > o ? v : o;
  }
  return v;
}

// part[g * parts + c] = the largest |x| (BF16 bits) of chunk c of group g
__global__ __launch_bounds__(256) void nvfp4_amax(const uint16_t* __restrict__ x, int64_t n, int parts,
                                                  uint32_t* __restrict__ part) {
  __shared__ uint32_t red[4];
  const int64_t grp = blockIdx.x / parts;
  const int64_t c0 = (int64_t)(blockIdx.x % parts) * kChunk;
  const int64_t len = min((int64_t)kChunk, n - c0);
  const v4i* p = reinterpret_cast<const v4i*>(x + grp * n + c0);
  uint32_t m = 0;
  for (int i = threadIdx.x; i < (int)(len >> 3); i += 256) {
    const v4i t = p[i];
    const uint32_t a = absmax8(make_uint4((uint32_t)t.x, (uint32_t)t.y, (uint32_t)t.z, (uint32_t)t.w));
    m = m > a ? m : a;
  }
  m = wave_max_u32(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = max(max(red[0], red[1]), max(red[2], red[3]));
}

// Two lanes hold a 16-value block, 8 values each.
__global__ __launch_bounds__(256) void nvfp4_quant(const uint16_t* __restrict__ x, int64_t n, int parts,
                                                   const uint32_t* __restrict__ part, uint8_t* __restrict__ q,
                                                   uint8_t* __restrict__ s, float* __restrict__ gscale) {
  __shared__ uint32_t red[4];
  const int64_t b = (int64_t)gridDim.x - 1 - blockIdx.x;
  const int64_t grp = b / parts, c0 = (b % parts) * kChunk;
  float g;
  if (part) {
    uint32_t m = 0;
    for (int i = threadIdx.x; i < parts; i += 256) m = max(m, part[grp * parts + i]);
    m = wave_max_u32(m);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    g = group_scale(max(max(red[0], red[1]), max(red[2], red[3])));
    if (c0 == 0 && threadIdx.x == 0) gscale[grp] = g;
  } else {
    g = gscale[grp];
  }
  const int64_t len = min((int64_t)kChunk, n - c0);
  const int64_t base = grp * n + c0;
  const v4i* p = reinterpret_cast<const v4i*>(x + base);
  for (int i = threadIdx.x; i < (int)(len >> 3); i += 256) {
    const v4i t = p[i];
    const uint32_t w[4] = {(uint32_t)t.x, (uint32_t)t.y, (uint32_t)t.z, (uint32_t)t.w};
    const uint32_t m = block_max(absmax8(make_uint4(w[0], w[1], w[2], w[3])), 1);
    const float f = fminf((__uint_as_float(m << 16) / 6.0f) / g, 448.0f);
    const uint32_t code = e4m3x4(f, 0.f, 0.f, 0.f) & 0xFFu;
    const float d = __builtin_amdgcn_cvt_f32_fp8((int)code, 0) * g;
    const float r = d > 0.f ? 1.0f / d : 0.f;
    uint32_t c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v0 = bf16_lo(w[k]), v1 = bf16_hi(w[k]);
      v0 = fminf(fmaxf(quotient(v0, d, r), -6.0f), 6.0f);
      v1 = fminf(fmaxf(quotient(v1, d, r), -6.0f), 6.0f);
      c |= (__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v0, v1, 1.0f, 0) & 0xFFu) << (8 * k);
    }
    reinterpret_cast<uint32_t*>(q + (base >> 1))[i] = c;
    if ((i & 1) == 0) s[(base >> 4) + (i >> 1)] = (uint8_t)code;
  }
}

// 32 values (16 code bytes, two scales) per thread.
__global__ __launch_bounds__(256) void nvfp4_dequant(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                     const float* __restrict__ gscale, int64_t n, int64_t total,
                                                     uint16_t* __restrict__ y) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // a run of 8 values
  if (i * 8 >= total) return;
  const float g = gscale[i * 8 / n];
  const uint32_t w = reinterpret_cast<const uint32_t*>(q)[i];
  const float d = __builtin_amdgcn_cvt_f32_fp8((int)s[i >> 1], 0) * g;
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const auto e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  reinterpret_cast<uint4*>(y)[i] = make_uint4(bf16x2_rne(a[0] * d, a[1] * d), bf16x2_rne(b[0] * d, b[1] * d),
                                              bf16x2_rne(c[0] * d, c[1] * d), bf16x2_rne(e[0] * d, e[1] * d));
}

}  // namespace

int64_t nvfp4_parts(int64_t n) { return (n + kChunk - 1) / kChunk; }

hipError_t launch_nvfp4_quantize(const uint16_t* x, int64_t G, int64_t n, uint8_t* q, uint8_t* s, float* gscale,
                                 bool given, uint32_t* part, hipStream_t stream) {
  const int parts = (int)nvfp4_parts(n);
  const dim3 grid((unsigned)(G * parts));
  if (!given) {
    hipLaunchKernelGGL(nvfp4_amax, grid, dim3(256), 0, stream, x, n, parts, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(nvfp4_quant, grid, dim3(256), 0, stream, x, n, parts, given ? nullptr : part, q, s, gscale);
  return hipGetLastError();
}

hipError_t launch_nvfp4_dequantize(const uint8_t* q, const uint8_t* s, const float* gscale, int64_t G, int64_t n,
                                   uint16_t* y, hipStream_t stream) {
  const int64_t total = G * n;
  hipLaunchKernelGGL(nvfp4_dequant, dim3((unsigned)((total / 8 + 255) / 256)), dim3(256), 0, stream, q, s, gscale, n,
                     total, y);
  return hipGetLastError();
}

}  // namespace w8a8
