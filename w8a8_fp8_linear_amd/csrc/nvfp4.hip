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
// maxima of its group and quantises. 128 x 1024 x 1024 values: 69 + 76
// us, and 62 us back, 954 MB in all at 4.6 TB/s, where a large copy reaches
// 5.1. The second read of x gains
// nothing from the last-level cache: neither the opposite order of the chunks
// nor batches of 16 to 128 MB (maxima, then codes of each) made it faster.
#include "device.h"
#include "launch.h"

namespace w8a8 {
namespace {

constexpr int kMaxParts = 1024;  // chunks of a group: every quantising workgroup reads their maxima

// Values per chunk, what a workgroup takes the maximum of: two loads a thread,
// more where a group has more than kMaxParts such chunks.
constexpr int64_t kChunk = 4096;

int64_t chunk_of(int64_t n) {
  const int64_t c = (n + kMaxParts - 1) / kMaxParts;
  return c <= kChunk ? kChunk : (c + kChunk - 1) / kChunk * kChunk;
}

// Values a workgroup quantises. Small tensors need every workgroup they can
// get (1024 x 1024 values: 3.9 us by chunks of 4096, 9.8 us by 32768); large
// ones gain from fewer that keep four loads a thread under way and reduce the
// group's maxima less often (128 x 1024 x 1024: 76 us by 32768, 88 us by 4096).
constexpr int64_t kLargeChunk = 32768, kLargeTotal = int64_t(1) << 24;

constexpr float kGscaleMin = 0x1p-96f;

__device__ inline float group_scale(uint32_t amax_bits) {
  if (amax_bits == 0) return 1.0f;
  return fmaxf(__uint_as_float(amax_bits << 16) / 2688.0f, kGscaleMin);
}

// fl32(x / d) held to +-6, for r = fl32(1 / d), both correctly rounded, and
// lim = fl32(6 d). x is held before the division: where the scale is given,
// x / d may pass the largest float32, and infinity would leave NaN. (What is
// held at lim comes out within a step of 6 and is code 7 or 15.) One residual
// correction of x * r (Markstein's method), exact where the residual x - q0 d is
// a float32: its last bit is worth ulp(q0) ulp(d), 2^-49 d at least for a
// quotient from 2^-3 on (a smaller one is code 0 either way), so d >= 2^-100.
// g >= 2^-91 gives that, s being 2^-9 at least; below it a division is made.
constexpr float kQuotientMinGscale = 0x1p-91f;

__device__ inline float quotient(float x, float d, float r, float lim) {
  const float v = __builtin_amdgcn_fmed3f(x, -lim, lim);
  const float q0 = v * r;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q0, d, v), r, q0), x);
}

// part[g * parts + c] = the largest |x| (BF16 bits) of chunk c of group g
__global__ __launch_bounds__(256) void nvfp4_amax(const uint16_t* __restrict__ x, int64_t n, int64_t chunk, int parts,
                                                  uint32_t* __restrict__ part) {
  __shared__ uint32_t red[4];
  const int64_t grp = blockIdx.x / parts, c0 = (int64_t)(blockIdx.x % parts) * chunk;
  const int64_t len = (min(chunk, n - c0)) >> 3;
  const v4i* p = reinterpret_cast<const v4i*>(x + grp * n + c0);
  uint32_t m = 0;
  for (int64_t i = threadIdx.x; i < len; i += 512) {
    const v4i a = p[i], b = i + 256 < len ? p[i + 256] : v4i{0, 0, 0, 0};
    m = max(m, absmax8(make_uint4((uint32_t)a.x, (uint32_t)a.y, (uint32_t)a.z, (uint32_t)a.w)));
    m = max(m, absmax8(make_uint4((uint32_t)b.x, (uint32_t)b.y, (uint32_t)b.z, (uint32_t)b.w)));
  }
  m = wave_max_u32(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = max(max(red[0], red[1]), max(red[2], red[3]));
}

// 8 values; two lanes (an even one and the next) hold a 16-value block.
__device__ inline void quant8_nv(v4i t, float g, uint32_t* q, uint8_t* s, int64_t i) {
  const uint32_t w[4] = {(uint32_t)t.x, (uint32_t)t.y, (uint32_t)t.z, (uint32_t)t.w};
  uint32_t m = absmax8(make_uint4(w[0], w[1], w[2], w[3]));
  m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
  const float f = fminf((__uint_as_float(m << 16) / 6.0f) / g, 448.0f);
  const uint32_t code = e4m3x4(f, 0.f, 0.f, 0.f) & 0xFFu;
  const float d = __builtin_amdgcn_cvt_f32_fp8((int)code, 0) * g;
  const float r = d > 0.f ? 1.0f / d : 0.f, lim = 6.0f * d;
  uint32_t c = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float v0 = bf16_lo(w[k]), v1 = bf16_hi(w[k]);
    if (__builtin_expect(g >= kQuotientMinGscale, 1)) {
      v0 = quotient(v0, d, r, lim);
      v1 = quotient(v1, d, r, lim);
    } else {
      v0 = d > 0.f ? __builtin_amdgcn_fmed3f(v0, -lim, lim) / d : __builtin_copysignf(0.f, v0);
      v1 = d > 0.f ? __builtin_amdgcn_fmed3f(v1, -lim, lim) / d : __builtin_copysignf(0.f, v1);
    }
    c |= (__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v0, v1, 1.0f, 0) & 0xFFu) << (8 * k);
  }
  q[i] = c;
  if ((i & 1) == 0) s[i >> 1] = (uint8_t)code;
}

// V 16-byte pieces a thread are loaded together
template <int V>
__global__ __launch_bounds__(256) void nvfp4_quant(const uint16_t* __restrict__ x, int64_t n, int64_t chunk, int chunks,
                                                   int parts, const uint32_t* __restrict__ part,
                                                   uint8_t* __restrict__ q, uint8_t* __restrict__ s,
                                                   float* __restrict__ gscale) {
  __shared__ uint32_t red[4];
  const int64_t grp = blockIdx.x / chunks, c0 = (int64_t)(blockIdx.x % chunks) * chunk;
  const int64_t base = grp * n + c0, len = (min(chunk, n - c0)) >> 3;
  const v4i* p = reinterpret_cast<const v4i*>(x + base);
  uint32_t* qc = reinterpret_cast<uint32_t*>(q + (base >> 1));
  uint8_t* sc = s + (base >> 4);
  v4i a[V];
  auto load = [&](int64_t i) {
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = i + 256 * v < len ? p[i + 256 * v] : v4i{0, 0, 0, 0};
  };
  load(threadIdx.x);  // the first values, on their way while the group's maximum is put together
  float g;
  if (part) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kMaxParts / 256; ++k) {
      const int j = threadIdx.x + 256 * k;
      m = max(m, j < parts ? part[grp * parts + j] : 0u);
    }
    m = wave_max_u32(m);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    g = group_scale(max(max(red[0], red[1]), max(red[2], red[3])));
    if (c0 == 0 && threadIdx.x == 0) gscale[grp] = g;
  } else {
    g = gscale[grp];
  }
  for (int64_t i = threadIdx.x; i < len; i += 256 * V) {
    v4i cur[V];
#pragma unroll
    for (int v = 0; v < V; ++v) cur[v] = a[v];
    load(i + 256 * V);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (i + 256 * v < len) quant8_nv(cur[v], g, qc, sc, i + 256 * v);
  }
}

// 8 values (4 code bytes) per thread.
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

int64_t nvfp4_parts(int64_t n) { return (n + chunk_of(n) - 1) / chunk_of(n); }

hipError_t launch_nvfp4_quantize(const uint16_t* x, int64_t G, int64_t n, uint8_t* q, uint8_t* s, float* gscale,
                                 bool given, uint32_t* part, hipStream_t stream) {
  const int64_t chunk = chunk_of(n);
  const int parts = (int)nvfp4_parts(n);
  if (!given) {
    hipLaunchKernelGGL(nvfp4_amax, dim3((unsigned)(G * parts)), dim3(256), 0, stream, x, n, chunk, parts, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  uint32_t* const maxima = given ? nullptr : part;
  if (G * n >= kLargeTotal) {
    const int64_t big = chunk < kLargeChunk ? kLargeChunk : chunk;
    const int chunks = (int)((n + big - 1) / big);
    hipLaunchKernelGGL(nvfp4_quant<4>, dim3((unsigned)(G * chunks)), dim3(256), 0, stream, x, n, big, chunks, parts,
                       maxima, q, s, gscale);
  } else {
    hipLaunchKernelGGL(nvfp4_quant<2>, dim3((unsigned)(G * parts)), dim3(256), 0, stream, x, n, chunk, parts, parts,
                       maxima, q, s, gscale);
  }
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
