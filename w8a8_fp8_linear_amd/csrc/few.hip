// A whole routed-expert layer for a few tokens in the default maths: router
// (logits, choice), gate/up + SwiGLU, down, weighted sum.
//
// A step with few tokens is set by how fast the expert weights are read, and
// the pages' runtime uses the default maths there: BF16 activations, weights
// widened to 16 bits as they are multiplied (Lernex/Metis-1.6-Logos-FP8,
// "What --fast-math does"). So each picked expert's weights are read once,
// whatever the number of tokens that picked it, and nothing is sorted or
// quantised in between:
//
//  * router_logits_*: l[t, e] = sum_k x[t, k] wr[e, k] in float64. The
//    products of two BF16 values are exact in float32, the sums are float64:
//    two experts change places only where their logits agree to 2^-45 or so.
//  * router_select: the score softmax(l) or sigmoid(l), the top-k experts by
//    score + bias, and their weights.
//  * few_rows (gate/up): tiles of 16 columns of h: the 16 gate and 16 up rows
//    of an expert, for every token that picked it (the MFMA's column side).
//    h = silu(g) * u is kept in float32 (the reading of the grouped calls).
//  * few_down_small (at most 8 tokens and 64 routed copies): one workgroup per
//    8 output columns walks all picked experts, a wave an expert, and
//    adds the router-weighted results per token in registers, by float32 FMAs.
//  * few_rows (down) + few_combine (more): tiles of 32 rows of an expert's W2
//    leave its tokens' weighted float32 rows, and the rows of a token are
//    added in the order of its slots. The BF16 matrix cores take h as three
//    BF16 values, h = hi + mid + lo: 3 x 8 significant bits are float32's 24.
// The output is rounded to BF16 once. Every sum's order is fixed by the ids
// and the sizes alone.
//
// A token that names an expert twice is one column whose router weights add.
#include "device.h"
#include "launch.h"
#include "widen.h"

#include <float.h>

#include <type_traits>

namespace w8a8 {
namespace {

// ---- router ------------------------------------------------------------------

typedef double v4d __attribute__((ext_vector_type(4)));

// Wave-wide reductions by DPP: row shifts by 1, 2, 4, 8, then the row
// broadcasts leave the result in lane 63. A DPP move takes a few cycles where
// a shuffle through LDS takes a hundred.
template <int CTRL, int ROWS = 0xF>
__device__ inline uint32_t dpp_u32(uint32_t old, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xF, false);
}

template <int CTRL, int ROWS = 0xF>
__device__ inline double dpp_f64(double old, double v) {
  const uint2 u = __builtin_bit_cast(uint2, v), o = __builtin_bit_cast(uint2, old);
  return __builtin_bit_cast(double, make_uint2(dpp_u32<CTRL, ROWS>(o.x, u.x), dpp_u32<CTRL, ROWS>(o.y, u.y)));
}

__device__ inline double readlane_f64(double v, int lane) {
  const uint2 u = __builtin_bit_cast(uint2, v);
  return __builtin_bit_cast(double, make_uint2((uint32_t)__builtin_amdgcn_readlane((int)u.x, lane),
                                               (uint32_t)__builtin_amdgcn_readlane((int)u.y, lane)));
}

__device__ inline uint32_t wave_max(uint32_t v) {
  v = max(v, dpp_u32<0x111>(0, v));
  v = max(v, dpp_u32<0x112>(0, v));
  v = max(v, dpp_u32<0x114>(0, v));
  v = max(v, dpp_u32<0x118>(0, v));
  v = max(v, dpp_u32<0x142>(0, v));
  v = max(v, dpp_u32<0x143>(0, v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ inline double wave_max(double v) {
  v = fmax(v, dpp_f64<0x111>(v, v));
  v = fmax(v, dpp_f64<0x112>(v, v));
  v = fmax(v, dpp_f64<0x114>(v, v));
  v = fmax(v, dpp_f64<0x118>(v, v));
  v = fmax(v, dpp_f64<0x142>(v, v));
  v = fmax(v, dpp_f64<0x143>(v, v));
  return readlane_f64(v, 63);
}

__device__ inline double wave_sum(double v) {  // the same order of additions whatever the values
  v += dpp_f64<0x111>(0.0, v);
  v += dpp_f64<0x112>(0.0, v);
  v += dpp_f64<0x114>(0.0, v);
  v += dpp_f64<0x118>(0.0, v);
  v += dpp_f64<0x142, 0xA>(0.0, v);
  v += dpp_f64<0x143, 0xC>(0.0, v);
  return readlane_f64(v, 63);
}

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
  double* logits;      // [T, E]
  int32_t* ids;        // [T, k]
  float* tw;           // [T, k]
  int T, H, E, k, sigmoid, renorm;
  float scale;
  float* logits32;     // [T, E] or NULL
};

// Few tokens: a wave per expert, lanes along K, TT tokens. One round of load
// latency (1 token, 192 experts, H 1024: 2.8 us; 64 tokens, 64 experts, H
// 2048: 4.7 us), so up to two tokens get workgroups of their own; more share
// a read of the expert's row.
template <int TT>
__global__ __launch_bounds__(256) void router_logits_few(const RouterArgs p) {
  constexpr int U = TT <= 2 ? 4 : 2;  // 512-value pieces of the rows loaded together
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.y * TT;
  if (e >= p.E) return;
  const auto rX = make_rsrc(p.x + (int64_t)t0 * p.H, (int64_t)min(TT, p.T - t0) * p.H * 2);
  const auto rW = make_rsrc(p.wr + (int64_t)e * p.H, (int64_t)p.H * 2);
  double acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.0;
  for (int k0 = lane * 8; k0 < p.H; k0 += 512 * U) {
    v4i wv[U], xv[U][TT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 512 * u;
      wv[u] = buffer_load16(rW, k < p.H ? (uint32_t)k * 2u : kOutOfRange);
#pragma unroll
      for (int t = 0; t < TT; ++t) xv[u][t] = buffer_load16(rX, k < p.H ? (uint32_t)(t * p.H + k) * 2u : kOutOfRange);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      double w[8], x[8];
      bf16x8_to_f64(wv[u], w);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        bf16x8_to_f64(xv[u][t], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[t] = __builtin_fma(w[i], x[i], acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const double s = wave_sum(acc[t]);
    if (lane == 0 && t0 + t < p.T) p.logits[(int64_t)(t0 + t) * p.E + e] = s;
  }
}

// More tokens: 16 tokens x 16 experts a workgroup on the float64 matrix
// cores, K split over the 8 waves in 32-deep steps. A lane loads 8
// consecutive values of its token's and of its expert's row (K 8 g .. of the
// step); MFMA i takes value i of each, so the step's K order is permuted alike
// on both sides. Bound by the float64 matrix units (4096 tokens x 64 experts x
// 2048: 25.0 us, 14.5 us at their full rate; four expert tiles a workgroup with
// loads a step ahead: 24.0 us, not worth a second variant for fewer tokens).
__global__ __launch_bounds__(512) void router_logits_mfma(const RouterArgs p) {
  __shared__ double red[8][256];
  constexpr int U = 4;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int tiles_e = (p.E + 15) / 16;
  const int t0 = blockIdx.x / tiles_e * 16, e0 = blockIdx.x % tiles_e * 16;
  const auto rX = make_rsrc(p.x + (int64_t)t0 * p.H, (int64_t)(p.T - t0) * p.H * 2);
  const auto rW = make_rsrc(p.wr + (int64_t)e0 * p.H, (int64_t)(p.E - e0) * p.H * 2);
  const uint32_t row = (uint32_t)r16 * (uint32_t)p.H * 2u;
  v4d acc[2] = {v4d{0, 0, 0, 0}, v4d{0, 0, 0, 0}};
  const int nk = (p.H + 31) >> 5;
  for (int kt = wave; kt < nk; kt += 8 * U) {
    v4i xv[U], wv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = ((kt + 8 * u) << 5) + 8 * g;
      const uint32_t off = kt + 8 * u < nk && k < p.H ? row + (uint32_t)k * 2u : kOutOfRange;
      xv[u] = buffer_load16(rX, off);
      wv[u] = buffer_load16(rW, off);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      double x[8], w[8];
      bf16x8_to_f64(xv[u], x);
      bf16x8_to_f64(wv[u], w);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        acc[i & 1] = __builtin_amdgcn_mfma_f64_16x16x4f64(x[i], w[i], acc[i & 1], 0, 0, 0);
    }
  }
  // acc[r] of lane (r16, g): token 4 r + g, expert r16
#pragma unroll
  for (int r = 0; r < 4; ++r) red[wave][(4 * r + g) * 16 + r16] = acc[0][r] + acc[1][r];
  __syncthreads();
  const int i = threadIdx.x;
  if (i < 256) {
    double s = red[0][i];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += red[w][i];
    const int t = t0 + (i >> 4), e = e0 + (i & 15);
    if (t < p.T && e < p.E) p.logits[(int64_t)t * p.E + e] = s;
  }
}

// The choice: a wave per token, lane l holding the NV experts from NV * l on.
// k times the largest of what is left: the lanes' largest, the wave's, and
// the first lane that has it, so that equal scores go by index. Lane j < k
// returns the j-th expert and its weight. A chain of dependent steps: 2.8 us
// for one token's 4 of 192, 4.8 us for 4096 tokens' 8 of 64.
template <int NV>
__device__ inline void select_token(const RouterArgs& p, int t, int lane, int* id, float* tw) {
  const double* l = p.logits + (int64_t)t * p.E;
  double val[NV], sel[NV];
  float bias[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane * NV + i;
    val[i] = e < p.E ? l[e] : -INFINITY;
    bias[i] = p.bias && e < p.E ? p.bias[e] : 0.f;
  }
  double inv = 1.0;
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < NV; ++i) val[i] = 1.0 / (1.0 + exp(-val[i]));
  } else {
    double mx = val[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) mx = fmax(mx, val[i]);
    mx = wave_max(mx);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      val[i] = exp(val[i] - mx);
      sum += val[i];
    }
    inv = 1.0 / wave_sum(sum);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    // -infinity (a bias that bars an expert) and NaN come after every number,
    // what is no expert or already chosen after all
    const double s = val[i] * inv + (double)bias[i];
    sel[i] = lane * NV + i >= p.E ? -INFINITY : s > -DBL_MAX ? s : -DBL_MAX;
  }
  double mine = 0.0, all = 0.0;  // lane j: the j-th chosen score; the sum of the chosen
  int mine_e = 0;
  for (int j = 0; j < p.k; ++j) {
    double best = sel[0], v = val[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < NV; ++i) {
      const bool up = sel[i] > best;
      best = up ? sel[i] : best;
      v = up ? val[i] : v;
      at = up ? i : at;
    }
    // the largest, by the bits of the float64 made to order as unsigned
    // numbers: the upper halves decide unless they are equal
    const uint2 bits = __builtin_bit_cast(uint2, best);
    const uint32_t neg = (uint32_t)((int)bits.y >> 31);
    const uint32_t hi = bits.y ^ (neg | 0x80000000u), lo = bits.x ^ neg;
    const bool top = hi == wave_max(hi);
    uint64_t who = __ballot(top);
    if (who & (who - 1)) {
      const uint32_t low = wave_max(top ? lo : 0u);  // by all lanes
      who = __ballot(top && lo == low);
    }
    const int from = __builtin_ctzll(who);
    const double score = readlane_f64(v, from) * inv;
    const int e = from * NV + __builtin_amdgcn_readlane(at, from);
    all += score;
    if (lane == j) {
      mine = score;
      mine_e = e;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane == from && i == at) sel[i] = -INFINITY;
  }
  *id = mine_e;
  *tw = (float)((p.renorm ? mine / all : mine) * (double)p.scale);
}

template <int NV>
__global__ __launch_bounds__(64) void router_select(const RouterArgs p) {
  const int lane = threadIdx.x, t = blockIdx.x;
  int id;
  float tw;
  select_token<NV>(p, t, lane, &id, &tw);
  if (lane < p.k) {
    p.ids[(int64_t)t * p.k + lane] = id;
    p.tw[(int64_t)t * p.k + lane] = tw;
  }
  if (p.logits32 != nullptr)
    for (int e = lane; e < p.E; e += 64) p.logits32[(int64_t)t * p.E + e] = (float)p.logits[(int64_t)t * p.E + e];
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
  float* h;               // [T * k, I]: every routed copy's h
  float* y;               // [T * k, H]: weighted float32 rows of the larger steps
  uint16_t* out;          // [T, H]
  int T, H, I, E, k, by_slot;
};

__device__ inline int rank_in(uint64_t mask, int lane) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// The work of a group: an expert and the tokens that picked it.
struct Group {
  int e;   // -1: nothing to do
  int n;   // tokens
};

// With no more routed copies than experts a group is a copy (slot), and the
// first copy of an expert works for all of them; otherwise a group is an
// expert. Lane t < T looks through its token's ids, eight loads at a time.
// cols[c] and (if asked) colw[c]: the first slot and the summed router weight
// of the group's c-th token, written by wave 0; the caller's barrier follows.
// `early` is called with the expert once it is known, when the ids are on their
// way: the first weights' loads go out there. (A copy that turns out not to be
// its expert's first has then read what the first one reads too; an expert
// without tokens, one round of loads for nothing.)
template <bool WEIGHTS, class EARLY>
__device__ inline Group find_group(const FewArgs& p, const int32_t* ids, int group, int* cols, float* colw,
                                   const EARLY& early) {
  const int lane = threadIdx.x & 63;
  const int own = p.by_slot ? ids[group] : 0;
  int slot = -1, e = -1;
  float w = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    int id[8];
    float tw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = lane < p.T && j0 + j < p.k;
      const int s = lane * p.k + j0 + j;
      id[j] = in ? ids[s] : -1;
      tw[j] = WEIGHTS && in ? p.tw[s] : 0.f;
    }
    if (j0 == 0) {
      e = __builtin_amdgcn_readfirstlane(p.by_slot ? own : group);
      if (e < 0 || e >= p.E) return {-1, 0};
      early(e);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (id[j] == e) {
        slot = slot < 0 ? lane * p.k + j0 + j : slot;
        w += tw[j];
      }
    }
  }
  const uint64_t mask = __ballot(slot >= 0);
  if (mask == 0) return {-1, 0};
  if (p.by_slot && __builtin_amdgcn_readlane(slot, __builtin_ctzll(mask)) != group) return {-1, 0};
  if (slot >= 0 && threadIdx.x < 64) {
    const int c = rank_in(mask, lane);
    cols[c] = slot;
    if (WEIGHTS) colw[c] = w;
  }
  return {e, __builtin_popcountll(mask)};
}

constexpr int kFewWaves = 4;
constexpr int kFewMaxE = 1024;

template <int F>
__device__ inline v4f row_scales(const void* s, const float* g, int64_t row, int e) {
  if constexpr (F == kFmtFp8) {
    const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(s) + row);
    return v4f{f.x, f.y, f.z, f.w};
  } else if constexpr (F == kFmtNvfp4) {
    const float f = g[e];
    return v4f{f, f, f, f};
  } else {
    return v4f{1.f, 1.f, 1.f, 1.f};
  }
}

// Steps of a round of few_rows: fewer for a short K split over waves, and where
// four waves' rounds would not leave the staged h (three values) in LDS.
template <int F, bool DOWN, int NT, int KS>
constexpr int kRowsU = (F == kFmtFp8 || (KS == 1 && !DOWN) ? 4 : 2) / (DOWN && KS == 4 ? 2 : 1);

// LDS for the staged rows, so that two workgroups share a CU.
constexpr int kRowsLds = 65536;

// 8 float32 values -> three BF16 operands whose sum is the values: each is the
// upper half of what the ones before leave, 8 significant bits. The
// subtractions are exact; infinity and NaN are the first operand's alone (their
// difference with themselves is NaN). A quiet NaN keeps its upper half's bits.
__device__ inline void split3(const float (&h)[8], v4i (&part)[3]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = h[i];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) part[q][i] = (int)pack_bf16(r[2 * i], r[2 * i + 1]);
    if (q == 2) break;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float left = r[i] - __uint_as_float(__float_as_uint(r[i]) & 0xFFFF0000u);
      r[i] = q == 0 && !__builtin_isfinite(r[i]) ? 0.f : left;
    }
  }
}

// One projection of one group of tokens. A tile is two sets of 16 weight rows
// (gate/up: 16 gate rows and their up rows; down: 32 rows); KS waves split a
// tile's K, so a workgroup holds kFewWaves / KS tiles at a time and takes
// `rounds` such sets of tiles one after another.
//
// The group's input rows (gate/up: x; down: the three parts of h, taken apart on
// the way) are staged in LDS once, in pieces of KC inputs if they do not fit
// whole, and every wave reads its MFMA columns from there. The weights go straight to registers, U steps
// of 2 x 16 rows x 64 bytes at a time, with the next U steps' loads issued
// before the current ones are used: nothing but the start waits for the
// weight stream, and with two workgroups per CU 128 KB of it are in flight.
//
// FP8, 64 tokens of 64 experts, 2048 x 512: gate/up 134 MB in 30 us (4.5
// TB/s), down 67 MB in 22 us (nvfp4 21 us), of which the third part of h is 1.2
// us and taking h apart 1 us. 8 tokens, nvfp4: gate/up about 50 MB in 17.5 us, of
// which some 4 us are the start (ids, then inputs and weights).
//
// ROUTE (at most kFewWaves tokens, few workgroups): the choice is made here
// from the logits, a wave per token, by every workgroup for itself, and
// written out by the first. That is 1 us of latency more, and a launch less.
template <int F, bool DOWN, int NT, int KS, bool ROUTE>
__global__ __launch_bounds__(64 * kFewWaves) __attribute__((amdgpu_waves_per_eu(2, 4)))
void few_rows(const FewArgs p, const RouterArgs route, int wgs_per_group, int rounds, int lds_bytes) {
  using W = WideFmt<F>;
  constexpr int U = kRowsU<F, DOWN, NT, KS>;
  using S = BlockScales<F, 2, U>;
  constexpr int P = DOWN ? 3 : 1;                 // parts of the input: h = hi + mid + lo
  constexpr int kRound = U * KS * W::kStepK;      // K values a round of loads covers
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ int cols[64];
  __shared__ float colw[64];
  __shared__ v4f red[KS > 1 ? kFewWaves * 2 * NT * 64 : 1];
  __shared__ __attribute__((aligned(16))) uint8_t slds[kFewWaves][S::kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int ks = wave % KS;
  const int K = DOWN ? p.I : p.H, rows = DOWN ? p.H : 2 * p.I;
  const int tile_rows = DOWN ? 32 : 16;           // output rows (down) or h columns (gate/up) of a tile
  const int out_rows = DOWN ? p.H : p.I;
  const int set_rows = DOWN ? 16 : p.I;           // distance of the two row sets
  const int64_t rb = W::row_bytes(K), rs = W::row_scales(K);
  __shared__ int32_t chosen[ROUTE ? kFewWaves * 64 : 1];
  const int32_t* ids = p.ids;
  if constexpr (ROUTE) {
    if (wave < p.T) {
      int id;
      float tw;
      if (route.E <= 64)
        select_token<1>(route, wave, lane, &id, &tw);
      else
        select_token<4>(route, wave, lane, &id, &tw);
      if (lane < p.k) {
        chosen[wave * p.k + lane] = id;
        if (blockIdx.x == 0) {
          route.ids[wave * p.k + lane] = id;
          route.tw[wave * p.k + lane] = tw;
        }
      }
    }
    lds_barrier();
    ids = chosen;
  }
  // this wave's tiles: row0, row0 + tile_step, ...
  const int tile_step = tile_rows * (kFewWaves / KS);
  const int row_first = (blockIdx.x % wgs_per_group) * rounds * tile_step + (wave / KS) * tile_rows;
  const int k_wave = ks * U * W::kStepK;          // this wave's part of a round

  // The loads of one round of the expert's weights. They are issued whether or
  // not there is one (then out of range, which reads nothing): behind a branch
  // the compiler would have to wait for all of them before the first use of
  // the round before.
  struct Buf {
    v4i w[U][2];
    S sc;
  } buf[2];
  __amdgpu_buffer_rsrc_t rW, rS;
  uint32_t skew;
  auto load = [&](Buf& b, int k, int row_at, bool there) {
    const int row = row_at + r16;
    const bool in = there && row_at < out_rows;
    const uint32_t w0 = (uint32_t)(row * rb), w1 = (uint32_t)((row + set_rows) * rb);
    const int kw = k + k_wave;
    b.sc.load(rS, [&](int a) {
      return in && kw < K ? skew + (uint32_t)((row + a * set_rows) * rs) + (uint32_t)(kw / W::kBlock) : kOutOfRange;
    });
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ku = kw + u * W::kStepK + W::kLaneK * g;
      const bool live = in && ku < K;
      b.w[u][0] = buffer_load16(rW, live ? w0 + (uint32_t)W::row_bytes(ku) : kOutOfRange);
      b.w[u][1] = buffer_load16(rW, live ? w1 + (uint32_t)W::row_bytes(ku) : kOutOfRange);
    }
  };
  const Group grp = find_group<DOWN>(p, ids, blockIdx.x / wgs_per_group, cols, colw, [&](int e) {
    rW = make_rsrc((DOWN ? p.w2 : p.w13) + (int64_t)e * rows * rb, (int64_t)rows * rb);
    rS = scale_rsrc(static_cast<const uint8_t*>(DOWN ? p.s2 : p.s13) + (int64_t)e * rows * rs, (int64_t)rows * rs, &skew);
    if (!DOWN) {
      load(buf[0], 0, row_first, true);
      __builtin_amdgcn_sched_barrier(0);
    }
  });
  if (grp.e < 0) return;
  const int e = grp.e;
  const auto rX = DOWN ? make_rsrc(p.h, (int64_t)p.T * p.k * p.I * 4) : make_rsrc(p.x, (int64_t)p.T * p.H * 2);
  lds_barrier();  // cols, colw

  // The pass over the weights for the group's n tokens in TT column tiles: a
  // copy of the code for each TT, so that none has a branch on the number of
  // tiles inside.
  const int n = grp.n;
  auto pass = [&](auto tt) {
  constexpr int TT = decltype(tt)::value;
  // KC: all of K if the n rows fit, else whole rounds; half a round where the
  // most rows that TT has would not fit otherwise
  constexpr int SUB = 16 * TT * 2 * P * kRound > kRowsLds ? 2 : 1;
  static_assert(16 * TT * 2 * P * kRound / SUB <= kRowsLds && (SUB == 1 || KS == 1), "a piece of all rows must fit");
  const int k_all = (K + kRound - 1) / kRound * kRound;
  const int fit = lds_bytes / (n * 2 * P) / kRound * kRound;
  const int KC = fit == 0 ? kRound / SUB : fit < k_all ? fit : k_all;
  const int k_pad = (k_all + KC - 1) / KC * KC;
  const int cpr = KC >> 3;                        // 16-byte chunks of a staged row

  int row0 = row_first;
  int load_k = 0, load_row = row0;  // the next round to load
  auto load_next = [&](Buf& b, bool there) {
    load(b, load_k, load_row, there);
    load_k += kRound;
    if (load_k >= k_pad) {
      load_k = 0;
      load_row += tile_step;
    }
  };
  if (!DOWN) {  // loaded while the group was found
    load_k = kRound < k_pad ? kRound : 0;
    load_row += load_k ? 0 : tile_step;
  } else {
    load_next(buf[0], true);
  }

  // A staged row holds its parts one after another; the 16-byte chunks of row
  // r are stored with their index XORed with r % 8, so that the 8 rows that 8
  // lanes read at one K lie in different banks. `loads` is called once the first
  // rows' loads are on their way.
  auto stage = [&](int k0, auto loads) {
    if constexpr (DOWN) {
      // four runs of 8 values a thread at a time
      const int runs = n * cpr;
      const float per_row = 1.0f / (float)cpr;
      auto batch = [&](int i0, auto between) {
        v4i v[4][2];
        uint32_t dst[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + 64 * kFewWaves * j;
          const int row = i < runs ? (int)(((float)i + 0.5f) * per_row) : 0;  // i / cpr: i is below 2^12
          const int c = i - row * cpr, k = k0 + 8 * c;
          const uint32_t at = i < runs && k < K ? ((uint32_t)cols[row] * (uint32_t)p.I + (uint32_t)k) * 4u : kOutOfRange;
          v[j][0] = buffer_load16(rX, at);
          v[j][1] = buffer_load16(rX, at + 16u);
          dst[j] = (uint32_t)(row * KC * (2 * P) + ((c ^ (row & 7)) << 4));
        }
        between();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (i0 + 64 * kFewWaves * j >= runs) break;
          float h[8];
          v4i part[P];
#pragma unroll
          for (int e8 = 0; e8 < 8; ++e8) h[e8] = __int_as_float(v[j][e8 >> 2][e8 & 3]);
          split3(h, part);
#pragma unroll
          for (int q = 0; q < P; ++q) *reinterpret_cast<v4i*>(smem + dst[j] + q * (KC * 2)) = part[q];
        }
      };
      batch(tid, loads);
      for (int i0 = tid + 64 * kFewWaves * 4; i0 < runs; i0 += 64 * kFewWaves * 4) batch(i0, [] {});
    } else {
      for (int row = wave; row < n; row += kFewWaves) {  // in 1 KB pieces of 64 chunks
        const uint32_t base = (uint32_t)(cols[row] / p.k) * (uint32_t)p.H * 2u;
        uint8_t* dst = smem + row * (KC * 2);
        for (int c0 = 0; c0 < cpr; c0 += 64) {
          const int k = k0 + 8 * ((c0 + lane) ^ (row & 7));
          if (c0 + lane < cpr) buffer_load16_lds(rX, dst + c0 * 16, k < K ? base + 2u * (uint32_t)k : kOutOfRange);
        }
      }
      loads();
      wait_vmem_all();
    }
  };
  uint32_t xrow[TT], xswz[TT];  // this lane's staged rows (columns past the last one read it again)
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const uint32_t row = (uint32_t)min(t * 16 + r16, n - 1);
    xrow[t] = row * (uint32_t)(KC * 2 * P);
    xswz[t] = (row & 7u) << 4;
  }
  v4f scale[2];  // the current tile's row scales
  auto load_scales = [&]() {
#pragma unroll
    for (int a = 0; a < 2; ++a)
      scale[a] = row0 < out_rows ? row_scales<F>(DOWN ? p.s2 : p.s13, DOWN ? p.g2 : p.g13,
                                                 (int64_t)e * rows + row0 + a * set_rows + 4 * g, e)
                                 : v4f{0.f, 0.f, 0.f, 0.f};
  };
  load_scales();

  v4f acc[2][TT];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[a][t] = v4f{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](const Buf& b, int sub, int kk) {  // part of the round, its first K inside the staged piece
#pragma unroll
    for (int u = sub * (U / SUB); u < (sub + 1) * (U / SUB); ++u) {
      const uint32_t at = 2u * (uint32_t)(kk + k_wave + (u - sub * (U / SUB)) * W::kStepK + W::kLaneK * g);
      const uint32_t s0 = S::get(slds[wave], u, 0), s1 = S::get(slds[wave], u, 1);
#pragma unroll
      for (int i = 0; i < W::kMfma; ++i) {
        const v4i w0 = widen_part<F>(b.w[u][0], s0, i), w1 = widen_part<F>(b.w[u][1], s1, i);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int q = 0; q < P; ++q) {
            const v4i x = *reinterpret_cast<const v4i*>(smem + xrow[t] + q * (KC * 2) + ((at + 16u * i) ^ xswz[t]));
            acc[0][t] = mfma_16x16x32_bf16(w0, x, acc[0][t]);
            acc[1][t] = mfma_16x16x32_bf16(w1, x, acc[1][t]);
          }
      }
    }
  };

  auto finish = [&]() {  // the sums of tile row0: lane (r16, g) holds rows 4 g .. of both sets, column 16 t + r16
    if constexpr (KS > 1) {
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int t = 0; t < TT; ++t) red[((wave * 2 + a) * TT + t) * 64 + lane] = acc[a][t];
      lds_barrier();
      if (ks == 0) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int w = 1; w < KS; ++w) acc[a][t] += red[(((wave + w) * 2 + a) * TT + t) * 64 + lane];
      }
      lds_barrier();
    }
    if (ks == 0 && row0 < out_rows) {
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const int c = t * 16 + r16;
        if (c < n) {
          const v4f v0 = acc[0][t] * scale[0], v1 = acc[1][t] * scale[1];
          if constexpr (DOWN) {
            const float w = colw[c];
            float* dst = p.y + (int64_t)cols[c] * p.H + row0 + 4 * g;
            *reinterpret_cast<v4f*>(dst) = v0 * v4f{w, w, w, w};
            *reinterpret_cast<v4f*>(dst + 16) = v1 * v4f{w, w, w, w};
          } else {
            v4f h;
#pragma unroll
            for (int r = 0; r < 4; ++r) h[r] = silu_f32(v0[r]) * v1[r];
            *reinterpret_cast<v4f*>(p.h + (int64_t)cols[c] * p.I + row0 + 4 * g) = h;
          }
        }
      }
    }
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[a][t] = v4f{0.f, 0.f, 0.f, 0.f};
    row0 += tile_step;
  };

  const int total = rounds * (k_pad / kRound);
  int k0 = 0, kk = 0;  // first K of the current round inside its tile, inside the staged piece
  auto step = [&](int r, const Buf& cur, Buf& next) {
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub) {
      const bool fresh = kk == 0 && (KC < k_pad || r == 0);  // a new piece of the input rows
      auto loads = [&]() {
        if (sub == 0) load_next(next, r + 1 < total);
      };
      if (fresh) {
        if (r || sub) lds_barrier();  // every wave is done with the piece before
        stage(k0 + sub * (kRound / SUB), loads);
        lds_barrier();
      } else {
        loads();
      }
      __builtin_amdgcn_sched_barrier(0);
      if (sub == 0) cur.sc.spread(slds[wave], (K - k0 - k_wave) / W::kBlock);
      compute(cur, sub, kk);
      kk = kk + kRound / SUB < KC ? kk + kRound / SUB : 0;
    }
    k0 += kRound;
    if (k0 >= k_pad) {
      k0 = 0;
      finish();
      if (r + 1 < total) load_scales();
    }
  };
  for (int r = 0; r < total; r += 2) {
    step(r, buf[0], buf[1]);
    if (r + 1 < total) step(r + 1, buf[1], buf[0]);
  }
  };
  // n <= 16 NT
  if (NT == 1 || n <= 16)
    pass(std::integral_constant<int, 1>{});
  else if (n <= 32)
    pass(std::integral_constant<int, NT == 1 ? 1 : 2>{});
  else
    pass(std::integral_constant<int, NT>{});
}

// out[t] = bf16(sum of the token's rows, in the order of its slots). A slot
// counts if its id is valid and no earlier slot of the token names it. 4.7 us
// for 64 tokens' 8 rows of 2048: the ids, then eight rows' loads at once.
__global__ __launch_bounds__(256) void few_combine(const FewArgs p) {
  const int t = blockIdx.y, lane = threadIdx.x & 63;
  const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
  uint64_t rows = 0;
  for (int j = 0; j < p.k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    if (e >= 0 && e < p.E && __builtin_ctzll(__ballot(id == e)) == j) rows |= 1ull << j;
  }
  if (c >= p.H) return;
  const float* y = p.y + (int64_t)t * p.k * p.H + c;
  v4f s = v4f{0.f, 0.f, 0.f, 0.f};
  while (rows) {
    v4f v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = v4f{0.f, 0.f, 0.f, 0.f};
      if (rows) v[i] = *reinterpret_cast<const v4f*>(y + (int64_t)__builtin_ctzll(rows) * p.H);
      rows &= rows - 1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.H + c) = make_uint2(bf16x2_rne(s[0], s[1]), bf16x2_rne(s[2], s[3]));
}

// 16 codes (FP8) or 32 (4-bit) of a lane's 16 bytes -> float32, MXFP4's times their block's scale (in its exponent).
template <int F>
__device__ inline void codes_f32(v4i w, float scale, float* f) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t c = (uint32_t)w[d];
    if constexpr (F == kFmtFp8) {
      const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
      f[4 * d] = a[0], f[4 * d + 1] = a[1], f[4 * d + 2] = b[0], f[4 * d + 3] = b[1];
    } else {
      const auto a0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0), a1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
      const auto a2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2), a3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3);
      f[8 * d] = a0[0], f[8 * d + 1] = a0[1], f[8 * d + 2] = a1[0], f[8 * d + 3] = a1[1];
      f[8 * d + 4] = a2[0], f[8 * d + 5] = a2[1], f[8 * d + 6] = a3[0], f[8 * d + 7] = a3[1];
    }
  }
}

// At most 8 tokens and 64 slots: 8 output columns a workgroup, so that a narrow
// output still fills the GPU. The picked experts, in the order of their first
// slots, times their rounds of 512 inputs are dealt to the waves in turn; lane s
// holds slot s's id and weight, so a ballot finds the expert's tokens. Lane
// (r16, g) works on row r16 % 8 in half r16 / 8 of K and loads 16 code bytes a
// step; the h rows of the expert's tokens go to LDS by direct loads, four tokens
// at a time, and a token's dot product is float32 FMAs: h keeps its 24 bits, a
// token that did not pick the expert is not touched, and most experts of so few
// tokens have one or two, where an MFMA would fill 8 columns. 8 tokens of 64
// nvfp4 experts, 2048 x 512: 11.9 us for 25 MB, the vector units busy 51% of the
// time and a wave waiting 49% of its own; one token's 4 fp8 experts, 1024 x 512:
// 4.0 us. Registers are held to 128 for four waves a SIMD; a spill costs 3 us.
template <int F, int WAVES>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(4, 4)))
void few_down_small(const FewArgs p) {
  using W = WideFmt<F>;
  constexpr int R = 8, TOK = 8;
  constexpr int B = 4;                       // tokens staged together
  constexpr int U = F == kFmtFp8 ? 4 : 2;    // steps of a round
  constexpr int kHalf = U * W::kStepK;       // inputs of a round in one half of K
  static_assert(2 * kHalf == 512, "a token's h of a round is two loads of a wave");
  using S = BlockScales<F, 1, U>;
  __shared__ uint32_t first[kFewMaxE];             // the first slot of every expert
  __shared__ __attribute__((aligned(1024))) float hbuf[WAVES][B][512];
  __shared__ __attribute__((aligned(16))) uint8_t slds[WAVES][S::kLds];
  __shared__ float sums[WAVES][TOK * R];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4, row = r16 % R, half = r16 / R;
  const int row0 = blockIdx.x * R;
  const int slots = p.T * p.k;
  const int id = lane < slots ? p.ids[lane] : -1;
  const float tw = lane < slots ? p.tw[lane] : 0.f;
  const int slot_tok = lane / p.k;
  const bool valid = id >= 0 && id < p.E;
  for (int i = threadIdx.x; i < p.E; i += 64 * WAVES) first[i] = 64;
  __syncthreads();
  if (wave == 0 && valid) atomicMin(&first[id], (uint32_t)lane);
  __syncthreads();
  uint64_t leaders = __ballot(valid && first[id] == (uint32_t)lane);
  const int64_t rb = W::row_bytes(p.I), rs = W::row_scales(p.I);
  const int steps = ((p.I + W::kStepK - 1) / W::kStepK + 1) / 2;  // of one half
  const int kbase = half * steps * W::kStepK;
  const int rounds = (steps + U - 1) / U;
  const auto rX = make_rsrc(p.h, (int64_t)slots * p.I * 4);
  const uint64_t kmask = p.k == 64 ? ~0ull : (1ull << p.k) - 1;
  float y[TOK];
#pragma unroll
  for (int t = 0; t < TOK; ++t) y[t] = 0.f;
  int round = wave;  // of the first of the experts that are left
  while (true) {
    for (; leaders && round >= rounds; round -= rounds) leaders &= leaders - 1;
    if (!leaders) break;
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(leaders));
    const uint64_t same = __ballot(id == e);
    const auto rW = make_rsrc(p.w2 + ((int64_t)e * p.H + row0) * rb, R * rb);
    uint32_t skew;
    const auto rS = scale_rsrc(static_cast<const uint8_t*>(p.s2) + ((int64_t)e * p.H + row0) * rs, R * rs, &skew);
    float scale = 1.f;
    if constexpr (F == kFmtFp8) scale = static_cast<const float*>(p.s2)[(int64_t)e * p.H + row0 + row];
    if constexpr (F == kFmtNvfp4) scale = p.g2[e];
    const int kt = round * U;
    round += WAVES;
    const int k0 = kbase + kt * W::kStepK;
    v4i w[U];
    S sc;
    sc.load(rS, [&](int) { return k0 < p.I ? skew + (uint32_t)(row * rs) + (uint32_t)(k0 / W::kBlock) : kOutOfRange; });
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * W::kStepK + W::kLaneK * g;
      w[u] = buffer_load16(rW, kt + u < steps && k < p.I ? (uint32_t)(row * rb) + (uint32_t)W::row_bytes(k) : kOutOfRange);
    }
    uint32_t hk[2];  // bytes into an h row of the 4 values that this lane brings to LDS for each half
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = 4 * lane;
      const int k = (i * steps + kt) * W::kStepK + at;
      hk[i] = kt + at / W::kStepK < steps && k < p.I ? (uint32_t)k * 4u : kOutOfRange;
    }
    float f[U][W::kLaneK], s[U][2];
    uint64_t rest = same;  // the slots of the tokens that are still to come
    auto stage = [&]() {   // the next B tokens' h
      uint64_t left = rest;
      int n = 0;
      for (; left && n < B; ++n) {
        const int slot = __builtin_ctzll(left);
        left &= ~(kmask << (__builtin_amdgcn_readlane(slot_tok, slot) * p.k));
        const uint32_t at = (uint32_t)slot * (uint32_t)p.I * 4u;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          buffer_load16_lds(rX, &hbuf[wave][n][256 * i], hk[i] == kOutOfRange ? kOutOfRange : at + hk[i]);
      }
      wait_vmem_all();
      wave_lds_order();
      return n;
    };
    int n = stage();
    sc.spread(slds[wave], (p.I - k0) / W::kBlock);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t code = S::get(slds[wave], u, 0);
      codes_f32<F>(w[u], F == kFmtMxfp4 ? mx_scale_value(code) : 1.0f, f[u]);
      if constexpr (F == kFmtNvfp4) {
        const auto two = __builtin_amdgcn_cvt_pk_f32_fp8((int)code, false);
        s[u][0] = two[0], s[u][1] = two[1];
      }
    }
    while (true) {
#pragma nounroll
      for (int b = 0; b < n; ++b) {
        const int tok = __builtin_amdgcn_readlane(slot_tok, __builtin_ctzll(rest));
        const uint64_t all = kmask << (tok * p.k);
        float weight = 0.f;
        for (uint64_t m = rest & all; m; m &= m - 1)
          weight += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(tw), __builtin_ctzll(m)));
        rest &= ~all;
        const float* h = &hbuf[wave][b][half * kHalf + W::kLaneK * g];
        float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int c0 = 0; c0 < W::kLaneK; c0 += 16) {  // 16 values: a block of NVFP4
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = c0; c < c0 + 16; c += 4) {
              const v4f x = *reinterpret_cast<const v4f*>(h + u * W::kStepK + c);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if constexpr (F == kFmtNvfp4)
                  d[i] = __builtin_fmaf(f[u][c + i], x[i], d[i]);
                else
                  a[i] = __builtin_fmaf(f[u][c + i], x[i], a[i]);
              }
            }
            if constexpr (F == kFmtNvfp4) {
#pragma unroll
              for (int i = 0; i < 4; ++i) a[i] = __builtin_fmaf(d[i], s[u][c0 / 16], a[i]);
            }
          }
        }
        const float add = ((a[0] + a[1]) + (a[2] + a[3])) * scale * weight;
#pragma unroll
        for (int t = 0; t < TOK; ++t) y[t] = tok == t ? y[t] + add : y[t];
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): what the tokens were read from is free
      wave_lds_order();
      if (!rest) break;
      n = stage();
    }
  }
  // the sum over the lanes that have the same row, in the place of the wave's h,
  // then over the waves
  float* const red = hbuf[wave][0];
  wave_lds_order();
#pragma unroll
  for (int t = 0; t < TOK; ++t) red[t * 72 + lane] = y[t];
  wave_lds_order();
  if (lane < TOK * R) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 64 / R; ++i) v += red[lane / R * 72 + i * R + lane % R];
    sums[wave][lane] = v;
  }
  __syncthreads();
  if (threadIdx.x < TOK * R) {
    const int t = threadIdx.x / R;
    if (t >= p.T) return;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += sums[w][threadIdx.x];
    p.out[(int64_t)t * p.H + row0 + threadIdx.x % R] = (uint16_t)bf16x2_rne(v, 0.f);
  }
}

// The small form takes the step's slots into one wave's lanes and its tokens
// into one operand.
bool few_small(int64_t T, int64_t topk) { return T <= 8 && T * topk <= 64; }

template <int F, bool DOWN, int NT, int KS, bool ROUTE = false>
void launch_rows_ks(const FewArgs& a, int groups, hipStream_t stream, const RouterArgs& route = {}) {
  const int K = DOWN ? a.I : a.H, P = DOWN ? 3 : 1;
  const int tiles = (DOWN ? a.H : a.I) / (DOWN ? 32 : 16), per_wg = kFewWaves / KS;
  const int sets = (tiles + per_wg - 1) / per_wg;  // sets of tiles a group has
  // two workgroups a CU run together; more tiles than they have are taken in
  // turn, with the next tile's weights on their way (down, 64 tokens of 64
  // experts: 22.4 us against 26.9 us for twice the workgroups)
  const int full = a.by_slot ? 1 : groups * sets / 512;  // by copies, many workgroups find nothing to do
  const int rounds = full < 1 ? 1 : full < 4 ? full : 4;
  const int wgs = (sets + rounds - 1) / rounds;
  const int round_k = kRowsU<F, DOWN, NT, KS> * KS * WideFmt<F>::kStepK;
  const int k_all = (K + round_k - 1) / round_k * round_k;
  const int rows = a.T < 16 * NT ? a.T : 16 * NT;
  const int64_t want = (int64_t)rows * k_all * 2 * P;
  const int lds = (int)(want < kRowsLds ? (want + 1023) / 1024 * 1024 : kRowsLds);  // a load writes 1 KB
  hipLaunchKernelGGL((few_rows<F, DOWN, NT, KS, ROUTE>), dim3((unsigned)(groups * wgs)), dim3(64 * kFewWaves), lds, stream,
                     a, route, wgs, rounds, lds);
}

int few_groups(const FewArgs& a) { return a.by_slot ? a.T * a.k : a.E; }

// Tiles up to which 4 or 2 waves share one. A 4-bit tile has more arithmetic
// to its bytes, and more waves to spread it over pay off longer (8 tokens of 64
// experts, 2048 tiles, gate/up: nvfp4 17.9 us with two waves a tile against
// 19.7 us with one, fp8 28.7 against 26.0 us).
constexpr int kSplit4 = 768;
template <int F>
constexpr int kSplit2 = F == kFmtFp8 ? 1536 : 2048;

// Whether the gate/up launch makes the choice: every workgroup does, so they
// must be few.
bool few_routes(const FewArgs& a) {
  return a.T <= kFewWaves && a.E <= 256 && few_groups(a) * (a.I / 16) <= kSplit4;
}

template <int F, bool DOWN>
hipError_t launch_rows(const FewArgs& a, const RouterArgs* route, hipStream_t stream) {
  const int groups = few_groups(a);
  const int tiles = groups * ((DOWN ? a.H : a.I) / (DOWN ? 32 : 16));
  if constexpr (!DOWN) {
    if (route) {
      launch_rows_ks<F, DOWN, 1, 4, true>(a, groups, stream, *route);
      return hipGetLastError();
    }
  }
  if (a.T > 16)
    launch_rows_ks<F, DOWN, 4, 1>(a, groups, stream);
  else if (tiles <= kSplit4)
    launch_rows_ks<F, DOWN, 1, 4>(a, groups, stream);
  else if (tiles <= kSplit2<F>)
    launch_rows_ks<F, DOWN, 1, 2>(a, groups, stream);
  else
    launch_rows_ks<F, DOWN, 1, 1>(a, groups, stream);
  return hipGetLastError();
}

template <int F>
hipError_t launch_few_fmt(const FewArgs& a, const RouterArgs* route, hipStream_t stream) {
  hipError_t e = launch_rows<F, false>(a, route, stream);
  if (e != hipSuccess) return e;
  if (few_small(a.T, a.k)) {
    // 16 waves a workgroup while each has a CU (whole layers, fp8: 8 tokens of 16
    // experts, 1024 x 2048, 27.8 us against 29.3 us with 8), two workgroups of 8 on a
    // CU for wider outputs (8192 x 512: 61.7 us against 68.5 us)
    if (a.H <= 8 * 256)
      hipLaunchKernelGGL((few_down_small<F, 16>), dim3(a.H / 8), dim3(64 * 16), 0, stream, a);
    else
      hipLaunchKernelGGL((few_down_small<F, 8>), dim3(a.H / 8), dim3(64 * 8), 0, stream, a);
    return hipGetLastError();
  }
  e = launch_rows<F, true>(a, nullptr, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(few_combine, dim3((a.H + 1023) / 1024, a.T), dim3(256), 0, stream, a);
  return hipGetLastError();
}

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

}  // namespace

size_t router_workspace_bytes(int64_t T, int64_t E) { return (size_t)(T * E * 8); }

static hipError_t launch_logits(const RouterArgs& a, hipStream_t stream) {
  const unsigned e4 = (unsigned)((a.E + 3) / 4);
  if (a.T <= 2)
    hipLaunchKernelGGL(router_logits_few<1>, dim3(e4, (unsigned)a.T), dim3(256), 0, stream, a);
  else if (a.T <= 64)
    hipLaunchKernelGGL(router_logits_few<4>, dim3(e4, (unsigned)((a.T + 3) / 4)), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(router_logits_mfma, dim3((unsigned)((a.T + 15) / 16 * ((a.E + 15) / 16))), dim3(512), 0, stream, a);
  return hipGetLastError();
}

static hipError_t launch_router(const RouterArgs& a, hipStream_t stream) {
  const hipError_t e = launch_logits(a, stream);
  if (e != hipSuccess) return e;
  if (a.E <= 64)
    hipLaunchKernelGGL(router_select<1>, dim3((unsigned)a.T), dim3(64), 0, stream, a);
  else if (a.E <= 256)
    hipLaunchKernelGGL(router_select<4>, dim3((unsigned)a.T), dim3(64), 0, stream, a);
  else
    hipLaunchKernelGGL(router_select<16>, dim3((unsigned)a.T), dim3(64), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_router(const Router& r, int64_t T, int64_t H, int64_t E, int64_t topk, void* ws, hipStream_t stream) {
  return launch_router(RouterArgs{r.x, r.wr, r.bias, static_cast<double*>(ws), r.ids, r.tw, (int)T, (int)H, (int)E,
                                  (int)topk, r.sigmoid, r.renorm, r.scale, r.logits},
                       stream);
}

// h, then the y rows; the router's logits, which are read before y is
// written, share the y rows' place.
static size_t few_h_bytes(int64_t T, int64_t I, int64_t topk) { return align256((size_t)(T * topk * I * 4)); }

size_t few_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t topk) {
  return few_h_bytes(T, I, topk) + (few_small(T, topk) ? 0 : (size_t)(T * topk * H * 4));
}

size_t few_layer_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk) {
  const size_t y = few_workspace_bytes(T, H, I, topk) - few_h_bytes(T, I, topk), l = router_workspace_bytes(T, E);
  return few_h_bytes(T, I, topk) + (y > l ? y : l);
}

hipError_t launch_few(const Few& f, const Router* r, int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk, void* ws,
                      hipStream_t stream) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  uint8_t* rest = b + few_h_bytes(T, I, topk);
  const FewArgs a{f.x, f.ids, f.tw, f.w13, f.s13, f.g13, f.w2, f.s2, f.g2, reinterpret_cast<float*>(b),
                  reinterpret_cast<float*>(rest), f.out, (int)T, (int)H, (int)I, (int)E, (int)topk, T * topk <= E ? 1 : 0};
  RouterArgs route{};
  const bool fused = r && few_routes(a);
  if (r) {
    route = RouterArgs{r->x, r->wr, r->bias, reinterpret_cast<double*>(rest), r->ids, r->tw, (int)T, (int)H, (int)E,
                       (int)topk, r->sigmoid, r->renorm, r->scale, nullptr};
    const hipError_t e = fused ? launch_logits(route, stream) : launch_router(route, stream);
    if (e != hipSuccess) return e;
  }
  const RouterArgs* choose = fused ? &route : nullptr;
  if (f.format == kFmtFp8) return launch_few_fmt<kFmtFp8>(a, choose, stream);
  if (f.format == kFmtMxfp4) return launch_few_fmt<kFmtMxfp4>(a, choose, stream);
  return launch_few_fmt<kFmtNvfp4>(a, choose, stream);
}

}  // namespace w8a8
