// A whole routed-expert layer for a few tokens in the default maths: router,
// gate/up + SwiGLU, down + weighted sum, three launches.
//
// A step with few tokens is set by how fast the expert weights are read, and
// the pages' runtime uses the default maths there: BF16 activations, weights
// widened to 16 bits as they are multiplied (Lernex/Metis-1.6-Logos-FP8,
// "What --fast-math does"). So each picked expert's weights are read once,
// whatever the number of tokens that picked it, and nothing is sorted,
// quantised or written in between but h:
//
//  * router: l[t, e] = sum_k x[t, k] wr[e, k] in float64, the score
//    softmax(l) or sigmoid(l), the top-k experts by score + bias, and their
//    weights. The products of two BF16 values are exact in float32 and the
//    sums are float64, so the experts a token gets do not depend on how many
//    tokens run with it or on how the sum is split.
//  * few_gate_up: one workgroup per (expert, 16 columns of h): the 16 gate
//    and 16 up rows of that expert, K split over the waves, for every token
//    that picked it (the MFMA's column side). h = silu(g) * u is written as a
//    pair of BF16 values, h = hi + lo: 16 significant bits, so that the down
//    product of an h kept in float32 (the reading of the grouped calls) is
//    met to 2^-17 while it runs on the BF16 matrix cores.
//  * few_down: one workgroup per 16 output columns: it walks all picked
//    experts, each wave taking its share of (expert, part of K) units, adds
//    the router-weighted results per token in float32 and rounds once to
//    BF16. No partial result leaves the workgroup, and the order of the sum
//    is fixed by the ids alone.
//
// A token that names an expert twice is one column whose router weights add.
#include "device.h"
#include "launch.h"
#include "widen.h"

namespace w8a8 {
namespace {

// ---- router ------------------------------------------------------------------

constexpr int kRouterThreads = 1024;
constexpr int kRouterMaxE = 1024;

__device__ inline double shfl_xor_f64(double v, int m) { return __shfl_xor(v, m, 64); }

// 8 BF16 values -> float64 (exact).
__device__ inline void bf16x8_to_f64(v4i v, double* d) {
  const uint32_t w[4] = {(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d[2 * i] = (double)bf16_lo(w[i]);
    d[2 * i + 1] = (double)bf16_hi(w[i]);
  }
}

struct RouterArgs {
  const uint16_t* x;   // [T, H]
  const uint16_t* wr;  // [E, H]
  const float* bias;   // [E] or NULL
  int32_t* ids;        // [T, k]
  float* tw;           // [T, k]
  int T, H, E, k, sigmoid, renorm;
  float scale;
};

template <int TT>
__global__ __launch_bounds__(kRouterThreads) void router(const RouterArgs p) {
  __shared__ double val[TT][kRouterMaxE];  // logits, then scores
  __shared__ double sel[TT][kRouterMaxE];  // what the experts are ordered by
  __shared__ double picked[TT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.x * TT;
  const int nt = min(TT, p.T - t0);
  const auto rX = make_rsrc(p.x + (int64_t)t0 * p.H, (int64_t)nt * p.H * 2);
  const auto rW = make_rsrc(p.wr, (int64_t)p.E * p.H * 2);

  constexpr int NE = 4;  // experts a wave takes together
  for (int e0 = wave * NE; e0 < p.E; e0 += (kRouterThreads / 64) * NE) {
    double acc[NE][TT];
#pragma unroll
    for (int e = 0; e < NE; ++e)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[e][t] = 0.0;
    for (int k = lane * 8; k < p.H; k += 512) {
      v4i xv[TT], wv[NE];
#pragma unroll
      for (int t = 0; t < TT; ++t) xv[t] = buffer_load16(rX, (uint32_t)(t * p.H + k) * 2u);
#pragma unroll
      for (int e = 0; e < NE; ++e) wv[e] = buffer_load16(rW, (uint32_t)((e0 + e) * p.H + k) * 2u);
      double x[TT][8];
#pragma unroll
      for (int t = 0; t < TT; ++t) bf16x8_to_f64(xv[t], x[t]);
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        double w[8];
        bf16x8_to_f64(wv[e], w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int t = 0; t < TT; ++t) acc[e][t] = __builtin_fma(w[i], x[t][i], acc[e][t]);
      }
    }
#pragma unroll
    for (int e = 0; e < NE; ++e)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        double a = acc[e][t];
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) a += shfl_xor_f64(a, m);
        if (lane == 0 && e0 + e < p.E) val[t][e0 + e] = a;
      }
  }
  __syncthreads();

  // Scores. The threads are split over the tokens; each wave finds its
  // token's maximum and sum by itself.
  constexpr int G = kRouterThreads / TT;  // threads per token
  const int t = tid / G, i = tid % G;
  double mx = -INFINITY;
  for (int e = lane; e < p.E; e += 64) mx = fmax(mx, val[t][e]);
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) mx = fmax(mx, shfl_xor_f64(mx, m));
  __syncthreads();
  for (int e = i; e < p.E; e += G) {
    const double l = val[t][e];
    val[t][e] = p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - mx);
  }
  __syncthreads();
  if (!p.sigmoid) {
    double sum = 0.0;
    for (int e = lane; e < p.E; e += 64) sum += val[t][e];
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) sum += shfl_xor_f64(sum, m);
    __syncthreads();
    for (int e = i; e < p.E; e += G) val[t][e] /= sum;
    __syncthreads();
  }
  for (int e = i; e < p.E; e += G) {
    const double s = val[t][e] + (p.bias ? (double)p.bias[e] : 0.0);
    sel[t][e] = s == s ? s : -INFINITY;  // a NaN score comes last: every rank below is taken once
  }
  __syncthreads();
  // rank[e] = how many experts go before e: a larger score, or the same and a
  // lower index. The experts with rank < k are the choice, in order.
  int parts = 1;
  while (parts < 64 && 2 * parts * p.E <= G) parts *= 2;
  for (int e0 = 0; e0 < p.E; e0 += G / parts) {
    const int e = e0 + i / parts;
    int rank = 0;
    if (e < p.E) {
      const double s = sel[t][e];
      for (int o = i % parts; o < p.E; o += parts) {
        const double v = sel[t][o];
        rank += (v > s || (v == s && o < e)) ? 1 : 0;
      }
    }
    for (int m = 1; m < parts; m <<= 1) rank += __shfl_xor(rank, m, 64);
    if (e < p.E && i % parts == 0 && rank < p.k) {
      picked[t][rank] = val[t][e];
      if (t < nt) p.ids[(int64_t)(t0 + t) * p.k + rank] = e;
    }
  }
  __syncthreads();
  if (i < p.k && t < nt) {
    double w = picked[t][i];
    if (p.renorm) {
      double sum = 0.0;
      for (int j = 0; j < p.k; ++j) sum += picked[t][j];
      w /= sum;
    }
    p.tw[(int64_t)(t0 + t) * p.k + i] = (float)(w * (double)p.scale);
  }
}

// ---- experts -----------------------------------------------------------------

struct FewArgs {
  const uint16_t* x;      // [T, H]
  const int32_t* ids;     // [T, k]
  const float* tw;        // [T, k]
  const uint8_t* w13;     // [E, 2I, H] codes
  const void* s13;        // FP8: float [E, 2I]; else block scale bytes [E, 2I, H / block]
  const float* g13;       // NVFP4: float [E]
  const uint8_t* w2;      // [E, H, I] codes
  const void* s2;
  const float* g2;
  uint16_t* h;            // [T * k, 2, I]: hi and lo of every routed copy's h
  uint16_t* out;          // [T, H]
  int T, H, I, E, k;
};

constexpr int kFewMaxE = 1024;

// Which tokens picked expert e: lane t < T looks through its token's ids.
// Returns the mask over tokens; *slot (of lane t) is the first of the token's
// slots that names e.
__device__ inline uint64_t tokens_of(const FewArgs& p, int e, int lane, int* slot) {
  int first = -1;
  if (lane < p.T) {
    for (int j = p.k - 1; j >= 0; --j)
      if (p.ids[lane * p.k + j] == e) first = lane * p.k + j;
  }
  *slot = first;
  return __ballot(first >= 0);
}

__device__ inline int rank_in(uint64_t mask, int lane) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

template <int F, int NT, int U>
__device__ inline void gate_up_tile(const FewArgs& p, int e, int row0, int n, const int* cols, v4f* red, int wave,
                                    int lane) {
  using W = WideFmt<F>;
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t rb = W::row_bytes(p.H), rs = W::row_scales(p.H);
  const auto rW = make_rsrc(p.w13 + (int64_t)e * 2 * p.I * rb, 2 * (int64_t)p.I * rb);
  const auto rS = make_rsrc(static_cast<const uint8_t*>(p.s13) + (int64_t)e * 2 * p.I * rs, 2 * (int64_t)p.I * rs);
  const auto rX = make_rsrc(p.x, (int64_t)p.T * p.H * 2);
  const uint32_t wrow[2] = {(uint32_t)((row0 + r16) * rb), (uint32_t)((p.I + row0 + r16) * rb)};
  const uint32_t srow[2] = {(uint32_t)((row0 + r16) * rs), (uint32_t)((p.I + row0 + r16) * rs)};
  uint32_t xrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 16 + r16;
    xrow[t] = c < n ? (uint32_t)(cols[c] / p.k) * (uint32_t)p.H * 2u : kOutOfRange;
  }
  v4f acc[2][NT];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[a][t] = v4f{0.f, 0.f, 0.f, 0.f};
  stream_dot<F, 2, NT, U>(rW, rS, wrow, srow, rX, xrow, p.H, wave, 4, acc);
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t) red[((wave * 2 + a) * NT + t) * 64 + lane] = acc[a][t];
  __syncthreads();
  // wave t finishes column tile t: lane (r16, g) holds column r16, h columns row0 + 4 g ..
  const int t = wave;
  const int c = t * 16 + r16;
  if (t >= NT || c >= n) return;
  v4f gu[2];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    gu[a] = red[(a * NT + t) * 64 + lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) gu[a] += red[((w * 2 + a) * NT + t) * 64 + lane];
    if constexpr (F == kFmtFp8) {
      const float4 s = *reinterpret_cast<const float4*>(static_cast<const float*>(p.s13) + (int64_t)e * 2 * p.I +
                                                        a * p.I + row0 + 4 * g);
      gu[a] *= v4f{s.x, s.y, s.z, s.w};
    } else if constexpr (F == kFmtNvfp4) {
      const float s = p.g13[e];
      gu[a] *= v4f{s, s, s, s};
    }
  }
  float h[4], lo[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) h[r] = silu_f32(gu[0][r]) * gu[1][r];
  const uint32_t h0 = bf16x2_rne(h[0], h[1]), h1 = bf16x2_rne(h[2], h[3]);
  lo[0] = h[0] - bf16_lo(h0);
  lo[1] = h[1] - bf16_hi(h0);
  lo[2] = h[2] - bf16_lo(h1);
  lo[3] = h[3] - bf16_hi(h1);
  uint16_t* dst = p.h + (int64_t)cols[c] * 2 * p.I + row0 + 4 * g;
  *reinterpret_cast<uint2*>(dst) = make_uint2(h0, h1);
  *reinterpret_cast<uint2*>(dst + p.I) = make_uint2(bf16x2_rne(lo[0], lo[1]), bf16x2_rne(lo[2], lo[3]));
}

// Workgroups (group, tile of 16 h columns). With no more routed copies than
// experts a group is a copy (slot), and the first copy of an expert works for
// all of them; otherwise a group is an expert. Either way a group that has
// nothing to do leaves after reading the ids.
template <int F, int NTMAX>
__global__ __launch_bounds__(256) void few_gate_up(const FewArgs p, int tiles, int by_slot) {
  __shared__ int cols[16 * NTMAX];
  __shared__ v4f red[4 * 2 * NTMAX * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = blockIdx.x / tiles, row0 = (blockIdx.x % tiles) * 16;
  const int e = by_slot ? p.ids[group] : group;
  if (e < 0 || e >= p.E) return;
  int slot;
  const uint64_t mask = tokens_of(p, e, lane, &slot);
  if (mask == 0) return;
  if (by_slot && __shfl(slot, __builtin_ctzll(mask), 64) != group) return;
  const int n = __builtin_popcountll(mask);
  if (slot >= 0 && wave == 0) cols[rank_in(mask, lane)] = slot;
  __syncthreads();
  if (NTMAX == 1 || n <= 16)
    gate_up_tile<F, 1, 4>(p, e, row0, n, cols, red, wave, lane);
  else if (NTMAX == 2 || n <= 32)
    gate_up_tile<F, (NTMAX >= 2 ? 2 : 1), 2>(p, e, row0, n, cols, red, wave, lane);
  else
    gate_up_tile<F, (NTMAX >= 4 ? 4 : 1), 1>(p, e, row0, n, cols, red, wave, lane);
}

constexpr int kDownWaves = 16;

// LDS written and read by the lanes of one wave: the hardware keeps a wave's
// LDS accesses in order, this keeps the compiler to it.
__device__ inline void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// One unit of the down projection: part `part` of `parts` of expert e's K
// range, for all its tokens, added into this wave's accumulators.
template <int F, int NT, int U>
__device__ inline void down_unit(const FewArgs& p, int e, int part, int parts, int row0, int n, const int* col_slot,
                                 const float* col_w, float* acc_w, int lane) {
  using W = WideFmt<F>;
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t rb = W::row_bytes(p.I), rs = W::row_scales(p.I);
  const auto rW = make_rsrc(p.w2 + ((int64_t)e * p.H + row0) * rb, 16 * rb);
  const auto rS = make_rsrc(static_cast<const uint8_t*>(p.s2) + ((int64_t)e * p.H + row0) * rs, 16 * rs);
  const auto rX = make_rsrc(p.h, (int64_t)p.T * p.k * p.I * 4);
  const uint32_t wrow[1] = {(uint32_t)(r16 * rb)}, srow[1] = {(uint32_t)(r16 * rs)};
  uint32_t xrow[2 * NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 16 + r16;
    xrow[t] = c < n ? (uint32_t)col_slot[c] * (uint32_t)p.I * 4u : kOutOfRange;
    xrow[NT + t] = c < n ? xrow[t] + (uint32_t)p.I * 2u : kOutOfRange;
  }
  v4f s = v4f{1.f, 1.f, 1.f, 1.f};
  if constexpr (F == kFmtFp8) {
    const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p.s2) + (int64_t)e * p.H + row0 + 4 * g);
    s = v4f{f.x, f.y, f.z, f.w};
  } else if constexpr (F == kFmtNvfp4) {
    const float f = p.g2[e];
    s = v4f{f, f, f, f};
  }
  v4f acc[1][2 * NT];
#pragma unroll
  for (int t = 0; t < 2 * NT; ++t) acc[0][t] = v4f{0.f, 0.f, 0.f, 0.f};
  stream_dot<F, 1, 2 * NT, U>(rW, rS, wrow, srow, rX, xrow, p.I, part, parts, acc);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 16 + r16;
    if (c < n) {
      const float w = col_w[c];
      v4f* a = reinterpret_cast<v4f*>(acc_w + (col_slot[c] / p.k) * 16 + 4 * g);
      *a += (acc[0][t] + acc[0][NT + t]) * s * v4f{w, w, w, w};
    }
  }
}

template <int F, int NTMAX>
__global__ __launch_bounds__(64 * kDownWaves) void few_down(const FewArgs p) {
  constexpr int TMAX = 16 * NTMAX;
  __shared__ unsigned long long mask[kFewMaxE];      // tokens of each expert
  __shared__ uint16_t active[kFewMaxE];              // experts with tokens, ascending
  __shared__ int s_ids[kFewMaxSlots];
  __shared__ float s_tw[kFewMaxSlots];
  __shared__ int s_active;
  __shared__ int col_slot[kDownWaves][TMAX];
  __shared__ float col_w[kDownWaves][TMAX];
  __shared__ v4f acc[kDownWaves][TMAX * 4];          // [wave][token][16 output columns]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row0 = blockIdx.x * 16;
  for (int i = tid; i < p.E; i += 64 * kDownWaves) mask[i] = 0;
  for (int i = lane; i < p.T * 4; i += 64) acc[wave][i] = v4f{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  for (int i = tid; i < p.T * p.k; i += 64 * kDownWaves) {
    const int e = p.ids[i];
    s_ids[i] = e;
    s_tw[i] = p.tw[i];
    if (e >= 0 && e < p.E) atomicOr(&mask[e], 1ull << (i / p.k));
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const bool on = e0 + lane < p.E && mask[e0 + lane] != 0;
      const uint64_t m = __ballot(on);
      if (on) active[n + rank_in(m, lane)] = (uint16_t)(e0 + lane);
      n += __builtin_popcountll(m);
    }
    if (lane == 0) s_active = n;
  }
  __syncthreads();
  const int na = s_active;
  // Few experts are cut into parts of K, so that every wave has a unit.
  const int nk = (p.I + WideFmt<F>::kStepK - 1) / WideFmt<F>::kStepK;
  int parts = 1;
  while (parts < nk && parts * na < kDownWaves) parts *= 2;
  for (int u = wave; u < na * parts; u += kDownWaves) {
    const int e = active[u / parts];
    const uint64_t m = mask[e];
    const int n = __builtin_popcountll(m);
    if ((m >> lane) & 1) {
      float w = 0.f;
      int first = -1;
      for (int j = p.k - 1; j >= 0; --j)
        if (s_ids[lane * p.k + j] == e) {
          first = lane * p.k + j;
          w += s_tw[first];
        }
      const int c = rank_in(m, lane);
      col_slot[wave][c] = first;
      col_w[wave][c] = w;
    }
    wave_lds_order();
    const int part = u % parts;
    if (NTMAX == 1 || n <= 16)
      down_unit<F, 1, 4>(p, e, part, parts, row0, n, col_slot[wave], col_w[wave], (float*)acc[wave], lane);
    else if (NTMAX == 2 || n <= 32)
      down_unit<F, (NTMAX >= 2 ? 2 : 1), 1>(p, e, part, parts, row0, n, col_slot[wave], col_w[wave], (float*)acc[wave], lane);
    else
      down_unit<F, (NTMAX >= 4 ? 4 : 1), 1>(p, e, part, parts, row0, n, col_slot[wave], col_w[wave], (float*)acc[wave], lane);
    wave_lds_order();
  }
  __syncthreads();
  for (int i = tid; i < p.T * 4; i += 64 * kDownWaves) {
    v4f s = acc[0][i];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) s += acc[w][i];
    *reinterpret_cast<uint2*>(p.out + (int64_t)(i >> 2) * p.H + row0 + 4 * (i & 3)) =
        make_uint2(bf16x2_rne(s[0], s[1]), bf16x2_rne(s[2], s[3]));
  }
}

template <int F, int NTMAX>
hipError_t launch_few_nt(const FewArgs& a, hipStream_t stream) {
  const int tiles = a.I / 16;
  const int by_slot = a.T * a.k <= a.E ? 1 : 0;
  const int groups = by_slot ? a.T * a.k : a.E;
  hipLaunchKernelGGL((few_gate_up<F, NTMAX>), dim3(groups * tiles), dim3(256), 0, stream, a, tiles, by_slot);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((few_down<F, NTMAX>), dim3(a.H / 16), dim3(64 * kDownWaves), 0, stream, a);
  return hipGetLastError();
}

template <int F>
hipError_t launch_few_fmt(const FewArgs& a, hipStream_t stream) {
  if (a.T <= 16) return launch_few_nt<F, 1>(a, stream);
  if (a.T <= 32) return launch_few_nt<F, 2>(a, stream);
  return launch_few_nt<F, 4>(a, stream);
}

}  // namespace

hipError_t launch_router(const uint16_t* x, const uint16_t* wr, const float* bias, int32_t* ids, float* tw, int64_t T,
                         int64_t H, int64_t E, int64_t topk, int sigmoid, int renorm, float scale,
                         hipStream_t stream) {
  const RouterArgs a{x, wr, bias, ids, tw, (int)T, (int)H, (int)E, (int)topk, sigmoid, renorm, scale};
  if (T <= 256)
    hipLaunchKernelGGL(router<1>, dim3((unsigned)T), dim3(kRouterThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(router<4>, dim3((unsigned)((T + 3) / 4)), dim3(kRouterThreads), 0, stream, a);
  return hipGetLastError();
}

size_t few_workspace_bytes(int64_t T, int64_t I, int64_t topk) { return (size_t)(T * topk * I * 4); }

hipError_t launch_few(int format, const uint16_t* x, const int32_t* ids, const float* tw, const uint8_t* w13,
                      const void* s13, const float* g13, const uint8_t* w2, const void* s2, const float* g2,
                      uint16_t* out, int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk, void* ws,
                      hipStream_t stream) {
  const FewArgs a{x,   ids, tw,     w13,    s13,    g13,    w2,        s2, g2, static_cast<uint16_t*>(ws),
                  out, (int)T, (int)H, (int)I, (int)E, (int)topk};
  if (format == kFmtFp8) return launch_few_fmt<kFmtFp8>(a, stream);
  if (format == kFmtMxfp4) return launch_few_fmt<kFmtMxfp4>(a, stream);
  return launch_few_fmt<kFmtNvfp4>(a, stream);
}

}  // namespace w8a8
