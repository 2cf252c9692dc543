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
//    h = silu(g) * u is written as a pair of BF16 values, h = hi + lo: 16
//    significant bits, so that the down product of an h kept in float32 (the
//    reading of the grouped calls) is met to 2^-17 while it runs on the BF16
//    matrix cores.
//  * few_down_small (at most 8 tokens and 64 routed copies): one workgroup per
//    4 or 8 output columns walks all picked experts, a wave an expert, and
//    adds the router-weighted results per token in registers.
//  * few_rows (down) + few_combine (more): tiles of 32 rows of an expert's W2
//    leave its tokens' weighted float32 rows, and the rows of a token are
//    added in the order of its slots.
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
  float* y;               // [T * k, H]: weighted float32 rows (few_down_rows)
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

// Steps of a round of few_rows. 2: a round fits 64 tokens' h in LDS, or a
// short K split over waves.
template <int F, bool DOWN, int NT, int KS>
constexpr int kRowsU = F == kFmtFp8 || (KS == 1 && !DOWN) ? 4 : 2;

// One projection of one group of tokens. A tile is two sets of 16 weight rows
// (gate/up: 16 gate rows and their up rows; down: 32 rows); KS waves split a
// tile's K, so a workgroup holds kFewWaves / KS tiles at a time and takes
// `rounds` such sets of tiles one after another.
//
// The group's input rows (gate/up: x; down: hi and lo of h) are staged in LDS
// once, in pieces of KC inputs if they do not fit whole, and every wave reads
// its MFMA columns from there. The weights go straight to registers, U steps
// of 2 x 16 rows x 64 bytes at a time, with the next U steps' loads issued
// before the current ones are used: nothing but the start waits for the
// weight stream, and with two workgroups per CU 128 KB of it are in flight.
//
// FP8, 64 tokens of 64 experts, 2048 x 512: gate/up 134 MB in 30 us (4.5
// TB/s), down 67 MB in 21 us (both parts of h are read from LDS for every
// weight). 8 tokens, nvfp4: gate/up about 50 MB in 17.5 us, of which some 4 us
// are the start (ids, then inputs and weights).
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
  constexpr int P = DOWN ? 2 : 1;                 // parts of the input: h = hi + lo
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
  // KC: whole rounds, all of K if the n rows fit
  const int k_all = (K + kRound - 1) / kRound * kRound;
  const int fit = lds_bytes / (n * 2 * P) / kRound * kRound;
  const int KC = fit < k_all ? fit : k_all;
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

  // Rows go to LDS in 1 KB pieces of 64 chunks; the 16-byte chunks of row r
  // are stored with their index XORed with r % 8, so that the 8 rows that 8
  // lanes read at one K lie in different banks.
  auto stage = [&](int k0) {
    for (int row = wave; row < P * n; row += kFewWaves) {
      const int part = row >= n ? 1 : 0;
      const int slot = cols[row - part * n];
      const uint32_t base = DOWN ? (uint32_t)slot * (uint32_t)p.I * 4u + (uint32_t)part * (uint32_t)p.I * 2u
                                 : (uint32_t)(slot / p.k) * (uint32_t)p.H * 2u;
      uint8_t* dst = smem + row * (KC * 2);
      for (int c0 = 0; c0 < cpr; c0 += 64) {
        const int k = k0 + 8 * ((c0 + lane) ^ (row & 7));
        if (c0 + lane < cpr) buffer_load16_lds(rX, dst + c0 * 16, k < K ? base + 2u * (uint32_t)k : kOutOfRange);
      }
    }
  };
  uint32_t xrow[P][TT], xswz[P][TT];  // this lane's staged rows (columns past the last one read it again)
#pragma unroll
  for (int q = 0; q < P; ++q)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const uint32_t row = (uint32_t)(q * n + min(t * 16 + r16, n - 1));
      xrow[q][t] = row * (uint32_t)(KC * 2);
      xswz[q][t] = (row & 7u) << 4;
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

  auto compute = [&](const Buf& b, int k0, int kk) {  // first K of the round, and inside the staged piece
    b.sc.spread(slds[wave], (K - k0 - k_wave) / W::kBlock);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t at = 2u * (uint32_t)(kk + k_wave + u * W::kStepK + W::kLaneK * g);
      const uint32_t s0 = S::get(slds[wave], u, 0), s1 = S::get(slds[wave], u, 1);
#pragma unroll
      for (int i = 0; i < W::kMfma; ++i) {
        const v4i w0 = widen_part<F>(b.w[u][0], s0, i), w1 = widen_part<F>(b.w[u][1], s1, i);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int q = 0; q < P; ++q) {
            const v4i x = *reinterpret_cast<const v4i*>(smem + xrow[q][t] + ((at + 16u * i) ^ xswz[q][t]));
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
            float h[4], lo[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) h[r] = silu_f32(v0[r]) * v1[r];
            const uint32_t h0 = bf16x2_rne(h[0], h[1]), h1 = bf16x2_rne(h[2], h[3]);
            lo[0] = h[0] - bf16_lo(h0);
            lo[1] = h[1] - bf16_hi(h0);
            lo[2] = h[2] - bf16_lo(h1);
            lo[3] = h[3] - bf16_hi(h1);
            uint16_t* dst = p.h + (int64_t)cols[c] * 2 * p.I + row0 + 4 * g;
            *reinterpret_cast<uint2*>(dst) = make_uint2(h0, h1);
            *reinterpret_cast<uint2*>(dst + p.I) = make_uint2(bf16x2_rne(lo[0], lo[1]), bf16x2_rne(lo[2], lo[3]));
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
    const bool fresh = kk == 0 && (KC < k_pad || r == 0);  // a new piece of the input rows
    if (fresh) {
      if (r) lds_barrier();  // every wave is done with the piece before
      stage(k0);
    }
    load_next(next, r + 1 < total);
    if (fresh) {
      wait_vmem_all();
      lds_barrier();
    }
    __builtin_amdgcn_sched_barrier(0);
    compute(cur, k0, kk);
    k0 += kRound;
    kk = kk + kRound < KC ? kk + kRound : 0;
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

// At most R tokens (R = 4 or 8) and 64 slots: R output columns a workgroup,
// so that a narrow output still fills the GPU. The 16 rows of an MFMA's
// weight operand are R weight rows at 16 / R places of K, its 16 columns R
// tokens at the same places: of the 16 x 16 results those count whose row and
// column are at the same place of K, and the places are added at the end. A
// wave takes every WAVES-th expert, in the order of their first slots; lane s
// holds slot s's id and weight, so a ballot finds the expert's tokens. 8 tokens
// of 64 nvfp4 experts, 2048 x 512: 12.0 us, 3 us and 0.23 us an expert, with
// 273 vector instructions and 20 loads per expert and wave. No single thing
// bounds it: loads a piece ahead (13.6 us), all of h in LDS and four pieces
// ahead (15.0 us) and 16 waves (12.9 us) are no faster. One token's 4 fp8
// experts, 1024 x 512: 4.3 us.
template <int F, int R, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void few_down_small(const FewArgs p) {
  using W = WideFmt<F>;
  constexpr int C = 16 / R;   // places of K
  constexpr int U = F == kFmtFp8 ? R / 2 : R / 4;  // the steps of one place of 512 inputs
  __shared__ uint32_t first[kFewMaxE];             // the first slot of every expert
  __shared__ v4f red[WAVES][64];
  __shared__ __attribute__((aligned(16))) uint8_t slds[WAVES][BlockScales<F, 1, U>::kLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int row0 = blockIdx.x * R;
  const int slots = p.T * p.k;
  const int id = lane < slots ? p.ids[lane] : -1;
  const float tw = lane < slots ? p.tw[lane] : 0.f;
  const bool valid = id >= 0 && id < p.E;
  for (int i = threadIdx.x; i < p.E; i += 64 * WAVES) first[i] = 64;
  __syncthreads();
  if (wave == 0 && valid) atomicMin(&first[id], (uint32_t)lane);
  __syncthreads();
  uint64_t leaders = __ballot(valid && first[id] == (uint32_t)lane);
  const int tok = r16 % R;
  const int64_t rb = W::row_bytes(p.I), rs = W::row_scales(p.I);
  const int steps = ((p.I + W::kStepK - 1) / W::kStepK + C - 1) / C;  // of one place
  const auto rX = make_rsrc(p.h, (int64_t)slots * p.I * 4);
  const uint32_t wrow[1] = {(uint32_t)((r16 % R) * rb)};
  v4f y = v4f{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < wave; ++i) leaders &= leaders - 1;
  while (leaders) {
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(leaders));
    const uint64_t same = __ballot(id == e);
    for (int i = 0; i < WAVES; ++i) leaders &= leaders - 1;
    const auto rW = make_rsrc(p.w2 + ((int64_t)e * p.H + row0) * rb, R * rb);
    uint32_t skew;
    const auto rS = scale_rsrc(static_cast<const uint8_t*>(p.s2) + ((int64_t)e * p.H + row0) * rs, R * rs, &skew);
    const uint32_t srow[1] = {skew + (uint32_t)((r16 % R) * rs)};
    const uint64_t kmask = p.k == 64 ? ~0ull : (1ull << p.k) - 1;
    uint64_t mine = tok < p.T ? (same >> (tok * p.k)) & kmask : 0;
    const int slot = mine ? tok * p.k + __builtin_ctzll(mine) : 0;
    const uint32_t at = (uint32_t)slot * (uint32_t)p.I * 4u;
    const uint32_t xrow[2] = {mine ? at : kOutOfRange, mine ? at + (uint32_t)p.I * 2u : kOutOfRange};
    const bool picked = mine != 0;
    float w = 0.f;
    while (__ballot(mine != 0)) {  // once, or again for a token that names the expert again
      const float v = __shfl(tw, mine ? tok * p.k + __builtin_ctzll(mine) : 0, 64);
      w += mine ? v : 0.f;
      mine &= mine - 1;
    }
    v4f acc[1][2] = {{v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}}};
    stream_dot<F, 1, 2, U>(rW, rS, wrow, srow, rX, xrow, p.I, (r16 / R) * steps * W::kStepK, steps, slds[wave], acc);
    // added for the tokens that picked the expert alone: 0 times its NaN would be NaN for the others
    const v4f add = (acc[0][0] + acc[0][1]) * row_scales<F>(p.s2, p.g2, (int64_t)e * p.H + row0 + (4 * g) % R, e) *
                    v4f{w, w, w, w};
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = picked ? y[i] + add[i] : y[i];
  }
  // lane (r16, g): rows 4 g .. 4 g + 3 of the operand, that is output columns
  // row0 + (4 g) % R .. at place 4 g / R; column r16: token r16 % R at place r16 / R
  red[wave][lane] = y;
  __syncthreads();
  if (threadIdx.x < R * R / 4) {
    const int t = threadIdx.x % R, q = threadIdx.x / R;  // token, quarter of the columns
    if (t >= p.T) return;
    v4f s = v4f{0.f, 0.f, 0.f, 0.f};
    for (int w = 0; w < WAVES; ++w)
#pragma unroll
      for (int c = 0; c < C; ++c) s += red[w][(c * (R / 4) + q) * 16 + c * R + t];
    *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.H + row0 + 4 * q) =
        make_uint2(bf16x2_rne(s[0], s[1]), bf16x2_rne(s[2], s[3]));
  }
}

// The small form takes the step's slots into one wave's lanes and its tokens
// into one operand.
bool few_small(int64_t T, int64_t topk) { return T <= 8 && T * topk <= 64; }

template <int F, bool DOWN, int NT, int KS, bool ROUTE = false>
void launch_rows_ks(const FewArgs& a, int groups, hipStream_t stream, const RouterArgs& route = {}) {
  const int K = DOWN ? a.I : a.H, P = DOWN ? 2 : 1;
  const int tiles = (DOWN ? a.H : a.I) / (DOWN ? 32 : 16), per_wg = kFewWaves / KS;
  const int sets = (tiles + per_wg - 1) / per_wg;  // sets of tiles a group has
  // two workgroups a CU run together; more tiles than they have are taken in
  // turn, with the next tile's weights on their way (down, 64 tokens of 64
  // experts: 20.6 us against 24.9 us for twice the workgroups)
  const int full = a.by_slot ? 1 : groups * sets / 512;  // by copies, many workgroups find nothing to do
  const int rounds = full < 1 ? 1 : full < 4 ? full : 4;
  const int wgs = (sets + rounds - 1) / rounds;
  const int round_k = kRowsU<F, DOWN, NT, KS> * KS * WideFmt<F>::kStepK;
  const int k_all = (K + round_k - 1) / round_k * round_k;
  const int rows = a.T < 16 * NT ? a.T : 16 * NT;
  const int64_t want = (int64_t)rows * k_all * 2 * P;
  const int lds = (int)(want < 65536 ? (want + 1023) / 1024 * 1024 : 65536);  // a load writes 1 KB
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
    // Every workgroup reads all of h: 8 columns each halve that against 4. One
    // token's h is small, and its few experts need the workgroups (1 of 128
    // experts, fp8: 4.4 us against 4.8 us; 2 of 64: 7.4 against 8.7 us).
    if (a.T == 1)
      hipLaunchKernelGGL((few_down_small<F, 4, 8>), dim3(a.H / 4), dim3(64 * 8), 0, stream, a);
    else
      hipLaunchKernelGGL((few_down_small<F, 8, 8>), dim3(a.H / 8), dim3(64 * 8), 0, stream, a);
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
                                  (int)topk, r.sigmoid, r.renorm, r.scale},
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
  const FewArgs a{f.x, f.ids, f.tw, f.w13, f.s13, f.g13, f.w2, f.s2, f.g2, reinterpret_cast<uint16_t*>(b),
                  reinterpret_cast<float*>(rest), f.out, (int)T, (int)H, (int)I, (int)E, (int)topk, T * topk <= E ? 1 : 0};
  RouterArgs route{};
  const bool fused = r && few_routes(a);
  if (r) {
    route = RouterArgs{r->x, r->wr, r->bias, reinterpret_cast<double*>(rest), r->ids, r->tw, (int)T, (int)H, (int)E,
                       (int)topk, r->sigmoid, r->renorm, r->scale};
    const hipError_t e = fused ? launch_logits(route, stream) : launch_router(route, stream);
    if (e != hipSuccess) return e;
  }
  const RouterArgs* choose = fused ? &route : nullptr;
  if (f.format == kFmtFp8) return launch_few_fmt<kFmtFp8>(a, choose, stream);
  if (f.format == kFmtMxfp4) return launch_few_fmt<kFmtMxfp4>(a, choose, stream);
  return launch_few_fmt<kFmtNvfp4>(a, choose, stream);
}

}  // namespace w8a8
