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
//  * w4a16_skinny: at most 32 rows, bound by the weight stream's latency and
//    the activations' L2 traffic. 16 or 32 weight rows per workgroup, the 4
//    waves split K, every lane widens the 32 codes of its 16-byte load in
//    registers (nvfp4 1 x 8192 x 2048: 4.8 us for 9.4 MB; mxfp4 24 x 6160 x
//    2048: 6.7 us).
//  * w4a16_mid: 32 x 64 or 64 x 64 results a workgroup, bound by a few rounds of
//    load latency and L1's rate (mxfp4 301 x 1040 x 1056: 5.9 us).
//  * w4a16_tiled: BM x BN tiles, 64-deep K steps in three LDS stages by direct
//    loads (128 bytes of activations, 32 bytes of codes a row). The tile's
//    block scales come 16 steps at a time, through registers (scale rows need
//    not start on a dword), and are read from LDS; a byte load per lane and
//    step instead was more than half of all requests to L2. A SIMD's MFMAs,
//    widening and LDS reads share its time (nvfp4, 4096 x 6144 x 2048: 101 us
//    back to back, 1016 TFLOP/s; mxfp4 95 us).
#include "device.h"
#include "launch.h"
#include "widen.h"

namespace w8a8 {
namespace {

constexpr int kCUs = 256;

typedef int v2i __attribute__((ext_vector_type(2)));

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

// NR x 16 weight rows a workgroup, MT tiles of 16 activation rows, U steps in
// flight, WAVES split K.
template <int F, int NR, int MT, int U, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void w4a16_skinny(const W4Args p) {
  using W = WideFmt<F>;
  __shared__ v4f red[WAVES][NR * MT][64];
  __shared__ __attribute__((aligned(16))) uint8_t slds[WAVES][BlockScales<F, NR, U>::kLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16 * NR;
  const int64_t rb = W::row_bytes(p.K), rs = W::row_scales(p.K);
  const auto rW = make_rsrc(p.w + n0 * rb, (p.N - n0) * rb);
  uint32_t skew;
  const auto rS = scale_rsrc(p.s + n0 * rs, (p.N - n0) * rs, &skew);
  const auto rX = make_rsrc(p.x, (int64_t)p.M * p.K * 2);
  const int r16 = lane & 15, g = lane >> 4;
  uint32_t wrow[NR], srow[NR], xrow[MT];
#pragma unroll
  for (int a = 0; a < NR; ++a) {
    wrow[a] = (uint32_t)((a * 16 + r16) * rb);
    srow[a] = skew + (uint32_t)((a * 16 + r16) * rs);
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) xrow[t] = t * 16 + r16 < p.M ? (uint32_t)(t * 16 + r16) * (uint32_t)p.K * 2u : kOutOfRange;
  const float gs = w4_scale<F>(p);
  v4f acc[NR][MT];
#pragma unroll
  for (int a = 0; a < NR; ++a)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[a][t] = v4f{0.f, 0.f, 0.f, 0.f};
  const int steps = ((p.K + W::kStepK - 1) / W::kStepK + WAVES - 1) / WAVES;  // of a wave's part of K
  stream_dot<F, NR, MT, U>(rW, rS, wrow, srow, rX, xrow, p.K, wave * steps * W::kStepK, steps, slds[wave], acc);
#pragma unroll
  for (int i = 0; i < NR * MT; ++i) red[wave][i][lane] = acc[i / MT][i % MT];
  __syncthreads();
  for (int i = wave; i < NR * MT; i += WAVES) {  // a tile a wave
    v4f v = red[0][i][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += red[w][i][lane];
    const int n = n0 + i / MT * 16 + 4 * g, m = i % MT * 16 + r16;
    if (n < p.N && m < p.M)
      *reinterpret_cast<uint2*>(p.y + (int64_t)m * p.N + n) =
          make_uint2(bf16x2_rne(v[0] * gs, v[1] * gs), bf16x2_rne(v[2] * gs, v[3] * gs));
  }
}

// Some rows, too few for the tiled kernel to fill the GPU: 16 TM x 64 results a
// workgroup, K split over its 4 waves, operands straight from global memory
// (the activations from L2); a wave's K fits a few rounds of loads.
template <int F, int TM>
__global__ __launch_bounds__(256) void w4a16_mid(const W4Args p) {
  using W = WideFmt<F>;
  constexpr int TN = 4;
  __shared__ v4f red[2][TN * TM][64];
  __shared__ __attribute__((aligned(16))) uint8_t slds[4][BlockScales<F, TN, 1>::kLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_n = (p.N + 63) / 64;
  const int n0 = blockIdx.x % tiles_n * 64, m0 = blockIdx.x / tiles_n * 16 * TM;
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
  // two waves leave their sums, the other two add theirs, then every wave
  // finishes the tiles of one column tile
#pragma unroll
  for (int turn = 0; turn < 2; ++turn) {
    if (wave >> 1 == turn) {
#pragma unroll
      for (int i = 0; i < TN * TM; ++i) {
        v4f& r = red[wave & 1][i][lane];
        r = turn ? r + acc[i / TM][i % TM] : acc[i / TM][i % TM];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const v4f v = red[0][wave * TM + t][lane] + red[1][wave * TM + t][lane];
    const int n = n0 + wave * 16 + 4 * g, m = m0 + t * 16 + r16;
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
  static constexpr int kStages = 3 * kStage > kEpi ? 3 * kStage : kEpi;
  static constexpr int kMinLoads = kSlots / kThreads;  // loads a wave issues for a stage, at least
  // a chunk of block scales: 16 steps, at most 64 bytes of every weight row, padded against bank conflicts
  static constexpr int kScaleStride = 68, kScaleChunk = BN * kScaleStride;
  static constexpr int kLds = kStages + 2 * kScaleChunk;
  static_assert(kSlotsW % 64 == 0 && kSlots % 64 == 0, "every load instruction must stay in one part");
  static_assert(WM % 16 == 0 && WN % 16 == 0, "wave tile must be a multiple of 16");
};

template <int F, int BM, int BN, int WGM, int WGN, int PER_EU>
__global__ __launch_bounds__(64 * WGM * WGN) __attribute__((amdgpu_waves_per_eu(1, PER_EU)))
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
  uint32_t skew;
  const auto rS = scale_rsrc(p.s + n0 * rs, (N - n0) * rs, &skew);
  const auto rX = make_rsrc(p.x + (int64_t)m0 * K, (int64_t)(M - m0) * K * 2);

  // Loader: slot s = tid + kThreads * i. Slots [0, kSlotsW) are weight row
  // s / 2, chunk s % 2 (32 codes); the rest are activation row s' / 8,
  // physical chunk s' % 8 (s' = s - kSlotsW), stored swizzled (stage_off). A
  // wave's 64 slots never straddle the two parts.
  // Which part a load fills is a scalar per wave: as a lane's condition it
  // would pick the buffer resource per lane, which the compiler turns into a
  // loop over the distinct ones.
  uint32_t off[C::kLoads];  // byte offset of the slot's chunk in the first K step
  int kc[C::kLoads];        // first K index of that chunk inside a step
#pragma unroll
  for (int i = 0; i < C::kLoads; ++i) {
    const int s0 = wave * 64 + C::kThreads * i, s = s0 + lane;
    if (s0 < C::kSlotsW) {
      kc[i] = (s & 1) << 5;
      off[i] = (uint32_t)((s >> 1) * rb) + (uint32_t)(kc[i] >> 1);
    } else {
      const int s2 = s - C::kSlotsW, row = s2 >> 3, c = (s2 & 7) ^ (row & 7);
      kc[i] = c << 3;
      off[i] = (uint32_t)row * (uint32_t)K * 2u + (uint32_t)(c << 4);
    }
  }
  auto issue = [&](uint8_t* base, int k0) {  // k0: first K index of the step
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
      const int s0 = wave * 64 + C::kThreads * i;
      const bool kin = k0 + kc[i] < K;  // K is a multiple of 32: a chunk is all in or all out
      if (s0 < C::kSlotsW) {
        buffer_load16_lds(rW, base + s0 * 16, kin ? off[i] + (uint32_t)(k0 >> 1) : kOutOfRange);
      } else if (s0 < C::kSlots) {
        buffer_load16_lds(rX, base + s0 * 16, kin ? off[i] + (uint32_t)k0 * 2u : kOutOfRange);
      }
    }
  };

  const int wm = wave % WGM, wn = wave / WGM;
  const int r16 = lane & 15, g = lane >> 4;
  // Scale chunks: thread t loads 16-byte pieces t, t + kThreads, ... (piece =
  // row, 16 bytes of the chunk) and shifts them to their place.
  constexpr int kRowPieces = 1024 / W::kBlock / 16;  // of a row's chunk: 1024 inputs
  constexpr int kPieces = (BN * kRowPieces + C::kThreads - 1) / C::kThreads;
  v4i sq[kPieces];
  uint32_t stop[kPieces];
  auto load_scales = [&](int chunk) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int piece = tid + C::kThreads * i, k = chunk * 1024 + piece % kRowPieces * (16 * W::kBlock);
      const uint32_t at = skew + (uint32_t)(piece / kRowPieces * rs) + (uint32_t)(k / W::kBlock);
      const uint32_t from = piece < BN * kRowPieces && k < K ? at & ~3u : kOutOfRange;
      sq[i] = buffer_load16(rS, from);
      stop[i] = __builtin_amdgcn_raw_buffer_load_b32(rS, from + 16u, 0, 0);
    }
  };
  auto store_scales = [&](int chunk) {
    uint8_t* dst = smem + C::kStages + (chunk & 1) * C::kScaleChunk;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int piece = tid + C::kThreads * i;
      if (piece >= BN * kRowPieces) break;
      const int k = chunk * 1024 + piece % kRowPieces * (16 * W::kBlock);
      const uint32_t shift = (skew + (uint32_t)(piece / kRowPieces * rs) + (uint32_t)(k / W::kBlock)) & 3u;
      const uint32_t d[5] = {(uint32_t)sq[i].x, (uint32_t)sq[i].y, (uint32_t)sq[i].z, (uint32_t)sq[i].w, stop[i]};
      uint32_t* o = reinterpret_cast<uint32_t*>(dst + piece / kRowPieces * C::kScaleStride + piece % kRowPieces * 16);
      const int left = (K - k) / W::kBlock;  // past the row's end 0, not the next row's
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __builtin_amdgcn_alignbyte(d[j + 1], d[j], shift) & low_bytes(left - 4 * j);
    }
  };
  v4f acc[C::SN][C::SM];
#pragma unroll
  for (int i = 0; i < C::SN; ++i)
#pragma unroll
    for (int j = 0; j < C::SM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const float gs = w4_scale<F>(p);

  // A step's MFMAs come in two halves (a lane's first and second 8 inputs).
  // While one half's run, the other half's activations are on their way from
  // LDS: half 1 of this step during half 0, half 0 of the next step during
  // half 1. The one barrier of a step stands between the halves. There every
  // wave has read all of this step's stage, which the loads of the third step
  // from here may then overwrite, and the next step's stage is complete: the
  // loads of the step after next, at least kMinLoads a wave, may still be out.
  const int nk = (K + 63) >> 6;
  uint32_t sc[C::SN], sc_next[C::SN];
  v4i xa[C::SM], xb[C::SM];
  // the lane's scale of a step: the byte of K 16 g .. of its rows
  auto read_scales = [&](uint32_t (&s)[C::SN], int kt) {
    const int at = ((kt & 15) * 64 + 16 * g) / W::kBlock;
    const uint8_t* src = smem + C::kStages + ((kt >> 4) & 1) * C::kScaleChunk + (at & ~3);
#pragma unroll
    for (int i = 0; i < C::SN; ++i)
      s[i] = (*reinterpret_cast<const uint32_t*>(src + (wn * C::WN + i * 16 + r16) * C::kScaleStride) >> (8 * (at & 3))) & 0xFFu;
  };
  v2i wc[C::SN], wc_next[C::SN];
  auto read_x = [&](v4i (&x)[C::SM], const uint8_t* st, int half) {
#pragma unroll
    for (int j = 0; j < C::SM; ++j)
      x[j] = *reinterpret_cast<const v4i*>(st + C::kWBytes + stage_off(wm * C::WM + j * 16 + r16, 2 * g + half));
  };
  auto read_w = [&](v2i (&w)[C::SN], const uint8_t* st) {
#pragma unroll
    for (int i = 0; i < C::SN; ++i)
      w[i] = *reinterpret_cast<const v2i*>(st + (wn * C::WN + i * 16 + r16) * 32 + g * 8);
  };
  auto multiply = [&](const v4i (&x)[C::SM], int half) {
#pragma unroll
    for (int i = 0; i < C::SN; ++i) {
      const uint32_t w = (uint32_t)(half ? wc[i].y : wc[i].x);
      v4i a;
      if constexpr (F == kFmtMxfp4)
        a = widen8_mx(w, mx_scale_value(sc[i]));
      else
        a = widen8_nv(w, __builtin_amdgcn_cvt_f32_fp8((int)sc[i], 0));
#pragma unroll
      for (int j = 0; j < C::SM; ++j) acc[i][j] = mfma_16x16x32_bf16(a, x[j], acc[i][j]);
    }
    // the first weight fragment's widening, then the others' between the MFMAs
    // of the one before (nvfp4, 4096 x 6144 x 2048: 120 us against 128 us without)
    constexpr int kWiden = F == kFmtMxfp4 ? 5 : 17;  // vector instructions of one fragment
    __builtin_amdgcn_sched_group_barrier(0x002, kWiden, 0);
#pragma unroll
    for (int i = 0; i < C::SN * C::SM; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, (kWiden + C::SM - 1) / C::SM, 0);
    }
  };
  uint8_t *st = smem, *st1 = smem + C::kStage, *st2 = smem + 2 * C::kStage;
  load_scales(0);
  issue(st, 0);
  store_scales(0);
  issue(st1, 64);
  issue(st2, 128);  // past the end: out of range, which reads zeros
  wait_vmcnt<2 * C::kMinLoads>();
  lds_barrier();
  read_x(xa, st, 0);
  read_w(wc, st);
  read_scales(sc, 0);
  for (int kt = 0; kt < nk; ++kt) {
    read_x(xb, st, 1);
    // the next chunk of scales: on its way during a chunk's first steps, in
    // LDS half a chunk later, in the place of the chunk before
    if ((kt & 15) == 0) load_scales((kt >> 4) + 1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(xa, 0);
    if ((kt & 15) == 8) store_scales((kt >> 4) + 1);
    wait_vmcnt<C::kMinLoads>();
    lds_barrier();
    issue(st, (kt + 3) << 6);
    read_x(xa, st1, 0);
    read_w(wc_next, st1);
    read_scales(sc_next, kt + 1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(xb, 1);
#pragma unroll
    for (int i = 0; i < C::SN; ++i) {
      sc[i] = sc_next[i];
      wc[i] = wc_next[i];
    }
    uint8_t* const free = st;
    st = st1;
    st1 = st2;
    st2 = free;
  }
  wait_vmem_all();  // the loads past the end write zeros to the stages, which the epilogue reuses

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

template <int F, int BM, int BN, int WGM, int WGN, int PER_EU>
hipError_t launch_tiled(const W4Args& a, hipStream_t stream) {
  const int tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN;
  hipLaunchKernelGGL((w4a16_tiled<F, BM, BN, WGM, WGN, PER_EU>), dim3(tiles_m * tiles_n), dim3(64 * WGM * WGN), 0, stream, a,
                     tiles_m, tiles_n);
  return hipGetLastError();
}

template <int F>
hipError_t launch_w4(const W4Args& a, hipStream_t stream) {
  // Every workgroup reads all activations, from L2: with 32 weight rows each
  // that is half the traffic of 16 (24 x 6160 x 2048: 6.6 us against 9.5 us,
  // 1 x 8192 x 2048: 4.6 against 4.8 us), as long as they fill half the GPU.
  const bool wide = a.N >= 4096;
  const dim3 grid((unsigned)(wide ? (a.N + 31) / 32 : (a.N + 15) / 16));
  if (a.M <= 16) {
    if (wide)
      hipLaunchKernelGGL((w4a16_skinny<F, 2, 1, 2, 4>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((w4a16_skinny<F, 1, 1, 4, 4>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  if (a.M <= 32) {
    if (wide)
      hipLaunchKernelGGL((w4a16_skinny<F, 2, 2, 2, 4>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((w4a16_skinny<F, 1, 2, 2, 4>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  // The tile grows with the work, so that each kernel starts with at most one
  // workgroup a CU: 32 x 64 with K split (64 x 6144 x 2048: 10.6 us against
  // 15.0 us in 64 x 64; but 128 x 6144 x 2048: 16.4 against 15.1 us), 64 x 64
  // (64 x 16384 x 2048: 15.9 us against 20.8 us in 64 x 128 tiles), 64 x 128 (256 x 6144 x 2048: 21.6 us against
  // 25.2 us in 64 x 64 and 27.0 us in 128 x 128), 128 x 128 (512 x 6144 x 2048:
  // 27.3 us against 35.3 us in 64 x 64 and 49.8 us in 256 x 192).
  const auto tiles = [&](int bm, int bn) { return (int64_t)((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
  if (tiles(32, 64) <= kCUs) {
    hipLaunchKernelGGL((w4a16_mid<F, 2>), dim3((unsigned)tiles(32, 64)), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  if (tiles(64, 64) <= kCUs) {
    hipLaunchKernelGGL((w4a16_mid<F, 4>), dim3((unsigned)tiles(64, 64)), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  if (tiles(64, 128) <= kCUs) return launch_tiled<F, 64, 128, 1, 4, 2>(a, stream);
  // From there on by rounds of 256 tiles: one of 128 x 128 costs two fifths of
  // one of 256 x 192 (K 2048: 20 us and 49 us; measured 60 against 53 us at 1536 x
  // 6144, 89 against 103 us at 2304, 124 against 103 us at 4096).
  const auto rounds = [](int64_t n) { return (n + kCUs - 1) / kCUs; };
  if (2 * rounds(tiles(128, 128)) < 5 * rounds(tiles(256, 192))) return launch_tiled<F, 128, 128, 2, 4, 4>(a, stream);
  return launch_tiled<F, 256, 192, 2, 4, 2>(a, stream);
}

}  // namespace

hipError_t launch_w4a16_gemm(int format, const uint16_t* x, const uint8_t* w, const uint8_t* s, const float* g,
                             uint16_t* y, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  const W4Args a{x, w, s, g, y, (int)M, (int)N, (int)K};
  return format == kFmtMxfp4 ? launch_w4<kFmtMxfp4>(a, stream) : launch_w4<kFmtNvfp4>(a, stream);
}

}  // namespace w8a8
