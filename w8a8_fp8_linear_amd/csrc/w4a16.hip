// Products with 4-bit weights in the default maths:
//   Y[m, n] = bf16( g * sum_k x[m, k] * s[n, k / block] * dec(W[n, k]) )
// NVFP4: E2M1 codes, an E4M3 scale per 16 inputs and one float32 scale g (the
// format of the pages' 4-bit checkpoint, Lernex/Metis-1.6-Praxis-NVFP4, "What
// is in NVFP4"). MXFP4: E2M1 codes and a power of two per 32 inputs, g = 1.
//
// Without the fast-math flag the weights are widened to 16 bits as they are
// multiplied and the activations stay BF16 (same page, "What --fast-math
// does"). A code times its block scale is exact in BF16 (widen.h), products
// are exact in float32, sums are float32, g is applied once in float32 and
// the result is rounded to nearest even.
//
//  * w4a16_skinny: at most 32 rows, set by the weight stream. 16 weight rows
//    per workgroup, the 4 waves split K, every lane widens the 32 codes of
//    its 16-byte load in registers.
//  * w4a16_tiled: more rows. BM x BN tiles, 64-deep K steps double buffered
//    in LDS by direct loads (128 bytes of activations, 32 bytes of codes a
//    row); a lane's block scale of the step comes by a byte load one step
//    ahead, since scale rows need not start on a dword.
#include "device.h"
#include "launch.h"
#include "widen.h"

namespace w8a8 {
namespace {

struct W4Args {
  const uint16_t* x;   // [M, K]
  const uint8_t* w;    // [N, K/2]
  const uint8_t* s;    // [N, K/block]
  const float* g;      // NVFP4: [1]
  uint16_t* y;         // [M, N]
  int M, N, K;
};

template <int F>
__device__ inline float w4_scale(const W4Args& p) {
  return F == kFmtNvfp4 ? *p.g : 1.0f;
}

// MT = number of 16-row activation tiles, U = steps in flight.
template <int F, int MT, int U>
__global__ __launch_bounds__(256) void w4a16_skinny(const W4Args p) {
  using W = WideFmt<F>;
  __shared__ v4f red[3][MT][64];
  __shared__ __attribute__((aligned(16))) uint8_t slds[4][BlockScales<F, 1, U>::kLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16;
  const int64_t rb = W::row_bytes(p.K), rs = W::row_scales(p.K);
  const auto rW = make_rsrc(p.w + n0 * rb, (p.N - n0) * rb);
  uint32_t skew;
  const auto rS = scale_rsrc(p.s + n0 * rs, (p.N - n0) * rs, &skew);
  const auto rX = make_rsrc(p.x, (int64_t)p.M * p.K * 2);
  const int r16 = lane & 15, g = lane >> 4;
  const uint32_t wrow[1] = {(uint32_t)(r16 * rb)}, srow[1] = {skew + (uint32_t)(r16 * rs)};
  uint32_t xrow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) xrow[t] = t * 16 + r16 < p.M ? (uint32_t)(t * 16 + r16) * (uint32_t)p.K * 2u : kOutOfRange;
  const float gs = w4_scale<F>(p);
  v4f acc[1][MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[0][t] = v4f{0.f, 0.f, 0.f, 0.f};
  const int steps = ((p.K + W::kStepK - 1) / W::kStepK + 3) / 4;  // of a wave's quarter of K
  stream_dot<F, 1, MT, U>(rW, rS, wrow, srow, rX, xrow, p.K, wave * steps * W::kStepK, steps, slds[wave], acc);
  if (wave > 0) {
#pragma unroll
    for (int t = 0; t < MT; ++t) red[wave - 1][t][lane] = acc[0][t];
  }
  __syncthreads();
  if (wave != 0) return;
  const int n = n0 + 4 * g;
  if (n >= p.N) return;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const v4f a = acc[0][t] + red[0][t][lane] + red[1][t][lane] + red[2][t][lane];
    const int m = t * 16 + r16;
    if (m < p.M)
      *reinterpret_cast<uint2*>(p.y + (int64_t)m * p.N + n) =
          make_uint2(bf16x2_rne(a[0] * gs, a[1] * gs), bf16x2_rne(a[2] * gs, a[3] * gs));
  }
}

// Some rows, too few for the tiled kernel to fill the GPU: 64 x 64 results a
// workgroup, K split over its 4 waves, operands straight from global memory
// (the activations from L2); a wave's K fits a few rounds of loads.
template <int F>
__global__ __launch_bounds__(256) void w4a16_mid(const W4Args p) {
  using W = WideFmt<F>;
  constexpr int TN = 4, TM = 4;
  __shared__ v4f red[2][TN * TM][64];
  __shared__ __attribute__((aligned(16))) uint8_t slds[4][BlockScales<F, TN, 1>::kLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_n = (p.N + 63) / 64;
  const int n0 = blockIdx.x % tiles_n * 64, m0 = blockIdx.x / tiles_n * 64;
  const int64_t rb = W::row_bytes(p.K), rs = W::row_scales(p.K);
  const auto rW = make_rsrc(p.w + n0 * rb, (p.N - n0) * rb);
  uint32_t skew;
  const auto rS = scale_rsrc(p.s + n0 * rs, (p.N - n0) * rs, &skew);
  const auto rX = make_rsrc(p.x + (int64_t)m0 * p.K, (int64_t)(p.M - m0) * p.K * 2);
  const int r16 = lane & 15, g = lane >> 4;
  uint32_t wrow[TN], srow[TN], xrow[TM];
#pragma unroll
  for (int a = 0; a < TN; ++a) {
    wrow[a] = (uint32_t)((a * 16 + r16) * rb);
    srow[a] = skew + (uint32_t)((a * 16 + r16) * rs);
  }
#pragma unroll
  for (int t = 0; t < TM; ++t) xrow[t] = (uint32_t)(t * 16 + r16) * (uint32_t)p.K * 2u;
  const float gs = w4_scale<F>(p);
  v4f acc[TN][TM];
#pragma unroll
  for (int a = 0; a < TN; ++a)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[a][t] = v4f{0.f, 0.f, 0.f, 0.f};
  const int steps = ((p.K + W::kStepK - 1) / W::kStepK + 3) / 4;  // of a wave's quarter of K
  stream_dot<F, TN, TM, 1>(rW, rS, wrow, srow, rX, xrow, p.K, wave * steps * W::kStepK, steps, slds[wave], acc);
  // waves 2, 3 add to 0, 1, then wave 1 to 0: each in half of the tiles at the end
  if (wave >= 2) {
#pragma unroll
    for (int i = 0; i < TN * TM; ++i) red[wave - 2][i][lane] = acc[i / TM][i % TM];
  }
  __syncthreads();
  if (wave < 2) {
#pragma unroll
    for (int i = 0; i < TN * TM; ++i) acc[i / TM][i % TM] += red[wave][i][lane];
  }
  __syncthreads();
  if (wave < 2) {  // wave 0 keeps the first half of the tiles, wave 1 the second
#pragma unroll
    for (int i = 0; i < TN * TM / 2; ++i) {
      red[wave][i][lane] = wave == 0 ? acc[(i + TN * TM / 2) / TM][i % TM] : acc[i / TM][i % TM];
    }
  }
  __syncthreads();
  if (wave >= 2) return;
#pragma unroll
  for (int i = 0; i < TN * TM / 2; ++i) {
    const int a = wave == 0 ? i / TM : (i + TN * TM / 2) / TM, t = i % TM;
    const v4f v = (wave == 0 ? acc[i / TM][t] : acc[(i + TN * TM / 2) / TM][t]) + red[1 - wave][i][lane];
    const int n = n0 + a * 16 + 4 * g, m = m0 + t * 16 + r16;
    if (n < p.N && m < p.M)
      *reinterpret_cast<uint2*>(p.y + (int64_t)m * p.N + n) =
          make_uint2(bf16x2_rne(v[0] * gs, v[1] * gs), bf16x2_rne(v[2] * gs, v[3] * gs));
  }
}

template <int BM, int BN, int WGM, int WGN>
struct Tiled4 {
  static constexpr int kThreads = 64 * WGM * WGN;
  static constexpr int WM = BM / WGM, WN = BN / WGN;
  static constexpr int SM = WM / 16, SN = WN / 16;
  static constexpr int kWBytes = BN * 32;               // code part of a stage
  static constexpr int kStage = kWBytes + BM * 128;     // + BF16 activation part
  static constexpr int kSlotsW = BN * 2, kSlots = kSlotsW + BM * 8;  // 16-byte LDS slots
  static constexpr int kLoads = (kSlots + kThreads - 1) / kThreads;
  static constexpr int kEpiStride = BN * 2 + 16;
  static constexpr int kEpi = BM * kEpiStride;
  static constexpr int kLds = (2 * kStage > kEpi) ? 2 * kStage : kEpi;
  static_assert(kSlotsW % 64 == 0 && kSlots % 64 == 0, "every load instruction must stay in one part");
  static_assert(WM % 16 == 0 && WN % 16 == 0, "wave tile must be a multiple of 16");
};

template <int F, int BM, int BN, int WGM, int WGN>
__global__ __launch_bounds__(64 * WGM * WGN) __attribute__((amdgpu_waves_per_eu(1, 2)))
void w4a16_tiled(const W4Args p, int tiles_m, int tiles_n) {
  using C = Tiled4<BM, BN, WGM, WGN>;
  using W = WideFmt<F>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int M = p.M, N = p.N, K = p.K;
  int tm, tn;
  map_tile<4>(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int64_t rb = W::row_bytes(K), rs = W::row_scales(K);
  const auto rW = make_rsrc(p.w + n0 * rb, (N - n0) * rb);
  const auto rS = make_rsrc(p.s + n0 * rs, (N - n0) * rs);
  const auto rX = make_rsrc(p.x + (int64_t)m0 * K, (int64_t)(M - m0) * K * 2);

  // Loader: slot s = tid + kThreads * i. Slots [0, kSlotsW) are weight row
  // s / 2, chunk s % 2 (32 codes); the rest are activation row s' / 8,
  // physical chunk s' % 8 (s' = s - kSlotsW), stored swizzled (stage_off). A
  // wave's 64 slots never straddle the two parts.
  uint32_t off[C::kLoads];  // byte offset of the slot's chunk in the first K step
  int kc[C::kLoads];        // first K index of that chunk inside a step
  bool isw[C::kLoads], live[C::kLoads];
#pragma unroll
  for (int i = 0; i < C::kLoads; ++i) {
    const int s = tid + C::kThreads * i;
    live[i] = s < C::kSlots;
    isw[i] = s < C::kSlotsW;
    if (isw[i]) {
      kc[i] = (s & 1) << 5;
      off[i] = (uint32_t)((s >> 1) * rb) + (uint32_t)(kc[i] >> 1);
    } else {
      const int s2 = s - C::kSlotsW, row = s2 >> 3, c = (s2 & 7) ^ (row & 7);
      kc[i] = c << 3;
      off[i] = (uint32_t)row * (uint32_t)K * 2u + (uint32_t)(c << 4);
    }
  }
  auto issue = [&](int stage, int k0) {  // k0: first K index of the step
    uint8_t* base = smem + stage * C::kStage;
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
      if (!live[i]) continue;
      const int s0 = wave * 64 + C::kThreads * i;
      const bool kin = k0 + kc[i] < K;  // K is a multiple of 32: a chunk is all in or all out
      if (isw[i]) {
        buffer_load16_lds(rW, base + s0 * 16, kin ? off[i] + (uint32_t)(k0 >> 1) : kOutOfRange);
      } else {
        buffer_load16_lds(rX, base + C::kWBytes + (s0 - C::kSlotsW) * 16, kin ? off[i] + (uint32_t)k0 * 2u : kOutOfRange);
      }
    }
  };

  const int wm = wave % WGM, wn = wave / WGM;
  const int r16 = lane & 15, g = lane >> 4;
  // this lane's weight rows: their scale of a step is the byte of K 16 g ..
  uint32_t srow[C::SN];
#pragma unroll
  for (int i = 0; i < C::SN; ++i) srow[i] = (uint32_t)((wn * C::WN + i * 16 + r16) * rs);
  auto load_scales = [&](uint32_t (&sc)[C::SN], int k0) {
    const int k = k0 + 16 * g;
#pragma unroll
    for (int i = 0; i < C::SN; ++i)
      sc[i] = __builtin_amdgcn_raw_buffer_load_b8(rS, k < K ? srow[i] + (uint32_t)(k / W::kBlock) : kOutOfRange, 0, 0);
  };
  v4f acc[C::SN][C::SM];
#pragma unroll
  for (int i = 0; i < C::SN; ++i)
#pragma unroll
    for (int j = 0; j < C::SM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const float gs = w4_scale<F>(p);

  const int nk = (K + 63) >> 6;
  uint32_t sc[C::SN], sc_next[C::SN];
  load_scales(sc_next, 0);
  issue(0, 0);
  for (int kt = 0; kt < nk; ++kt) {
    wait_vmem_all();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C::SN; ++i) sc[i] = sc_next[i];
    if (kt + 1 < nk) {
      load_scales(sc_next, (kt + 1) << 6);
      issue((kt + 1) & 1, (kt + 1) << 6);
    }
    const uint8_t* st = smem + (kt & 1) * C::kStage;
    const uint8_t* sx = st + C::kWBytes;
    v4i xlo[C::SM], xhi[C::SM];
#pragma unroll
    for (int j = 0; j < C::SM; ++j) {
      const int row = wm * C::WM + j * 16 + r16;
      xlo[j] = *reinterpret_cast<const v4i*>(sx + stage_off(row, 2 * g));
      xhi[j] = *reinterpret_cast<const v4i*>(sx + stage_off(row, 2 * g + 1));
    }
#pragma unroll
    for (int i = 0; i < C::SN; ++i) {
      const int row = wn * C::WN + i * 16 + r16;
      const uint2 w = *reinterpret_cast<const uint2*>(st + row * 32 + g * 8);
      v4i wlo, whi;
      if constexpr (F == kFmtMxfp4) {
        const float s = mx_scale_value(sc[i]);
        wlo = widen8_mx(w.x, s);
        whi = widen8_mx(w.y, s);
      } else {
        const float s = __builtin_amdgcn_cvt_f32_fp8((int)sc[i], 0);
        wlo = widen8_nv(w.x, s);
        whi = widen8_nv(w.y, s);
      }
#pragma unroll
      for (int j = 0; j < C::SM; ++j) {
        acc[i][j] = mfma_16x16x32_bf16(wlo, xlo[j], acc[i][j]);
        acc[i][j] = mfma_16x16x32_bf16(whi, xhi[j], acc[i][j]);
      }
    }
  }

  // Epilogue: acc[i][j][r] = Y[m][n], m = m-tile j row lane % 16, n = n-tile i,
  // 4 * (lane / 16) + r. Scale, round to BF16, stage in LDS, store row segments.
  __syncthreads();
#pragma unroll
  for (int i = 0; i < C::SN; ++i) {
    const int nl = wn * C::WN + i * 16 + 4 * g;
#pragma unroll
    for (int j = 0; j < C::SM; ++j) {
      const int ml = wm * C::WM + j * 16 + r16;
      const v4f a = acc[i][j];
      *reinterpret_cast<uint2*>(smem + ml * C::kEpiStride + nl * 2) =
          make_uint2(bf16x2_rne(a[0] * gs, a[1] * gs), bf16x2_rne(a[2] * gs, a[3] * gs));
    }
  }
  __syncthreads();
  constexpr int kRowChunks = BN / 8;
  for (int c = tid; c < BM * kRowChunks; c += C::kThreads) {
    const int row = c / kRowChunks, col = (c % kRowChunks) * 8;
    const int m = m0 + row, n = n0 + col;
    if (m < M && n < N)
      *reinterpret_cast<uint4*>(p.y + (int64_t)m * N + n) =
          *reinterpret_cast<const uint4*>(smem + row * C::kEpiStride + col * 2);
  }
}

template <int F, int BM, int BN, int WGM, int WGN>
hipError_t launch_tiled(const W4Args& a, hipStream_t stream) {
  const int tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN;
  hipLaunchKernelGGL((w4a16_tiled<F, BM, BN, WGM, WGN>), dim3(tiles_m * tiles_n), dim3(64 * WGM * WGN), 0, stream, a,
                     tiles_m, tiles_n);
  return hipGetLastError();
}

template <int F>
hipError_t launch_w4(const W4Args& a, hipStream_t stream) {
  const dim3 skinny_grid((unsigned)((a.N + 15) / 16));
  if (a.M <= 16) {
    hipLaunchKernelGGL((w4a16_skinny<F, 1, 4>), skinny_grid, dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  if (a.M <= 32) {
    hipLaunchKernelGGL((w4a16_skinny<F, 2, 2>), skinny_grid, dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  const int64_t big = (int64_t)((a.M + 255) / 256) * ((a.N + 191) / 192);
  if (big < 128) {
    hipLaunchKernelGGL(w4a16_mid<F>, dim3((unsigned)((a.M + 63) / 64 * ((a.N + 63) / 64))), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  return launch_tiled<F, 256, 192, 2, 4>(a, stream);
}

}  // namespace

hipError_t launch_w4a16_gemm(int format, const uint16_t* x, const uint8_t* w, const uint8_t* s, const float* g,
                             uint16_t* y, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  const W4Args a{x, w, s, g, y, (int)M, (int)N, (int)K};
  return format == kFmtMxfp4 ? launch_w4<kFmtMxfp4>(a, stream) : launch_w4<kFmtNvfp4>(a, stream);
}

}  // namespace w8a8
