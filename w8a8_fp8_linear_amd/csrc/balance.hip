// The balance loss of a router's choice, tokens per expert, and the gradient
// of the logits.
//
// The pages' router keeps its experts balanced (Lernex/Metis-1.6-Praxis,
// "Architecture"). With c[s,e] the routed copies of sequence s that expert e
// got, n[s] its tokens that name an expert, p the token's scores made to sum
// to one, f = E c / (k n):
//   loss = coef / S * sum_s sum_e f[s,e] * mean_t p[t,e]
//        = sum_t u_t,   u_t = coef / (S n) * sum_e f[s,e] p[t,e]
// The counts are constants of the gradient, so u_t is also the term that
// softmax's backward pass subtracts,
//   dloss/dl[t,j] = p_j (1 - sigma_j or 1) (g_j - sum_e g_e p_e),  g = coef f / (S n),
// and once the counts are there loss and gradient are one pass over the
// logits: read once, the gradient written once. f - 1 takes f's place in both
// (the p sum to one), which keeps the bits that a nearly balanced choice would
// lose in g_j - sum g p; the 1 comes back in the loss.
#include <algorithm>

#include "device.h"
#include "launch.h"

namespace w8a8 {
namespace {

constexpr int kThreads = 1024;  // of a workgroup
constexpr int kMainGroups = 256;  // workgroups of the main pass over all sequences
constexpr int kTicketStride = 16;  // words
constexpr int kMaxChunks = 32;  // of a sequence: every workgroup of the main pass adds them up

struct BalanceArgs {
  const void* logits;   // [S L, E]
  const int32_t* ids;   // [S L, k]
  int32_t* part;        // [S, C, E + 1]: copies of a chunk's tokens by expert, its tokens that count
  double* sums;         // [S G]
  uint32_t* tickets;    // [1 + ceil(S G / round)] a cache line each
  float* loss;          // [1]
  int32_t* counts;      // [S, E]
  void* grad;           // [S L, E] or NULL
  int64_t L;
  int S, E, k, C, G, chunk, round;
  float coef;
};

// Sum and maximum over groups of 16, 32 or 64 lanes, in every lane, by vector
// moves alone: swaps inside quads, mirrored halves and rows, then the rows and
// halves exchanged.
template <int CTRL>
__device__ inline float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
template <int LANES, typename F>
__device__ inline float group_reduce(float v, F f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  v = f(v, dpp<0x140>(v));
  if constexpr (LANES >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (LANES >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
template <int LANES>
__device__ inline float group_sum(float v) {
  return group_reduce<LANES>(v, [](float a, float b) { return a + b; });
}
template <int LANES>
__device__ inline float group_max(float v) {
  return group_reduce<LANES>(v, [](float a, float b) { return fmaxf(a, b); });
}

// The tokens that a group of LANES lanes works on together, NC pieces of four
// values a lane. VEC: E is a multiple of 4, and a piece is one load; otherwise
// four. Loads have no condition (a lane past the end reads its row's first
// values): the compiler waits for loads where a branch ends.
template <typename TL, int LANES, int NC, bool VEC>
struct Tokens {
  static constexpr int UT = NC == 1 ? 4 : 1;  // tokens of a group in flight
  uint32_t raw[UT][NC][4];
  int id[UT];

  // Token u of the group is t0 + u * step of the sequence whose first row is row0 (L > 0).
  __device__ inline void load(const BalanceArgs& p, int64_t row0, int64_t t0, int step, int l) {
    const TL* logits = static_cast<const TL*>(p.logits);
#pragma unroll
    for (int u = 0; u < UT; ++u) {
      const int64_t t = t0 + (int64_t)u * step;
      const int64_t row = row0 + (t < p.L ? t : 0);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int e = 4 * (l + LANES * i);
        const TL* src = logits + row * p.E;
        if constexpr (VEC && sizeof(TL) == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + (e < p.E ? e : 0));
          raw[u][i][0] = v.x, raw[u][i][1] = v.y, raw[u][i][2] = v.z, raw[u][i][3] = v.w;
        } else if constexpr (VEC) {
          const uint2 v = *reinterpret_cast<const uint2*>(src + (e < p.E ? e : 0));
          raw[u][i][0] = v.x, raw[u][i][1] = v.y;
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const TL v = src[e + r < p.E ? e + r : 0];
            raw[u][i][r] = sizeof(TL) == 4 ? __builtin_bit_cast(uint32_t, (float)v) : (uint32_t)v;
          }
        }
      }
      id[u] = p.ids[row * p.k + (l < p.k ? l : 0)];
    }
    if (p.k > LANES) {  // more copies than lanes: any valid one will do
#pragma unroll
      for (int u = 0; u < UT; ++u) {
        const int64_t t = t0 + (int64_t)u * step;
        const int64_t row = row0 + (t < p.L ? t : 0);
        for (int j = l + LANES; j < p.k; j += LANES) {
          const int e = p.ids[row * p.k + j];
          if (e >= 0 && e < p.E) id[u] = e;
        }
      }
    }
  }

  __device__ inline float value(int u, int i, int r, int e, int E) const {
    const uint32_t b = sizeof(TL) == 4 ? raw[u][i][r] : !VEC ? raw[u][i][r] << 16
                       : r & 1 ? raw[u][i][r >> 1] & 0xFFFF0000u : raw[u][i][r >> 1] << 16;
    return (VEC ? e : e + r) < E ? __uint_as_float(b) : -INFINITY;
  }

  // Adds the tokens' terms of the loss to sum and writes their gradients. w:
  // this lane's (f - 1) * base.
  __device__ inline void work(const BalanceArgs& p, int64_t row0, int64_t t0, int step, int lane, int sigmoid, float base,
                              const float (&w)[NC][4], double& sum) {
    TL* grad = static_cast<TL*>(p.grad);
    const int l = lane % LANES;
    const uint64_t group = LANES == 64 ? ~0ull : ((1ull << (LANES & 63)) - 1) << (lane - l);
    float x[UT][NC][4], inv[UT], dot[UT];  // x inv: p_j times its slope
    bool here[UT];
#pragma unroll
    for (int u = 0; u < UT; ++u) {
      here[u] = (__ballot(id[u] >= 0 && id[u] < p.E) & group) != 0 && t0 + (int64_t)u * step < p.L;
      float m = sigmoid ? 0.f : -INFINITY, z = 0.f, d = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[u][i][r] = value(u, i, r, 4 * (l + LANES * i), p.E);
          if (!sigmoid) m = fmaxf(m, x[u][i][r]);
        }
      if (!sigmoid) {
        m = group_max<LANES>(m);
        m = m == -INFINITY ? 0.f : m;
      }
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float v = x[u][i][r];
          if (sigmoid) {
            // d p_j / d l_j is p_j (1 - sigmoid(l_j)) for sigmoids divided by their sum; from one
            // half on 1 - sigmoid(l) is e^-l sigmoid(l), which a subtraction would lose
            const float t = __expf(-v), y = __builtin_amdgcn_rcpf(1.0f + t);
            z += y;
            d = __builtin_fmaf(w[i][r], y, d);
            x[u][i][r] = y * (y < 0.5f ? 1.0f - y : t * y);
          } else {
            x[u][i][r] = __expf(v - m);
            z += x[u][i][r];
            d = __builtin_fmaf(w[i][r], x[u][i][r], d);
          }
        }
      z = group_sum<LANES>(z);
      // sigmoids too small for float32, where sigmoid(v) is e^v: the same p from a softmax
      if (sigmoid && z < 0x1p-60f) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) m = fmaxf(m, value(u, i, r, 4 * (l + LANES * i), p.E));
        m = group_max<LANES>(m);
        m = m == -INFINITY ? 0.f : m;
        z = d = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[u][i][r] = __expf(value(u, i, r, 4 * (l + LANES * i), p.E) - m);
            z += x[u][i][r];
            d = __builtin_fmaf(w[i][r], x[u][i][r], d);
          }
        z = group_sum<LANES>(z);
      }
      inv[u] = z > 0.f ? 1.0f / z : 0.f;
      dot[u] = group_sum<LANES>(d) * inv[u];
      if (here[u]) sum += (double)dot[u] + (z > 0.f ? (double)base : 0.0);
    }
    if (!grad) return;
#pragma unroll
    for (int u = 0; u < UT; ++u) {
      const int64_t t = t0 + (int64_t)u * step;
      if (t >= p.L) continue;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int e = 4 * (l + LANES * i);
        float d[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) d[r] = here[u] ? x[u][i][r] * inv[u] * (w[i][r] - dot[u]) : 0.f;
        TL* dst = grad + (row0 + t) * p.E + e;
        if constexpr (VEC && sizeof(TL) == 4) {
          if (e < p.E) *reinterpret_cast<float4*>(dst) = make_float4(d[0], d[1], d[2], d[3]);
        } else if constexpr (VEC) {
          if (e < p.E) *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2_rne(d[0], d[1]), bf16x2_rne(d[2], d[3]));
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (e + r < p.E) {
              if constexpr (sizeof(TL) == 4) dst[r] = d[r];
              else dst[r] = (TL)bf16x2_rne(d[r], 0.f);
            }
        }
      }
    }
  }
};

// The counts of a piece of a sequence's tokens into LDS (cleared here); h[E]:
// the tokens that count. A wave takes whole tokens, a lane a copy, and the first
// valid copy of a token counts it. Ends with a barrier.
__device__ inline void count_tokens(const BalanceArgs& p, int64_t row0, int64_t lo, int64_t hi, int* h) {
  for (int e = threadIdx.x; e <= p.E; e += kThreads) h[e] = 0;
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = 64 / p.k, t = lane / p.k, j = lane - t * p.k;  // tokens a wave, this lane's token and copy
  const uint64_t before = ((1ull << lane) - 1) & ~((1ull << (lane - j)) - 1);  // the token's earlier copies
  int here = 0;
  constexpr int U = 4;
  for (int64_t t0 = lo + (int64_t)wave * per; t0 < hi; t0 += (int64_t)U * (kThreads / 64) * per) {
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tok = t0 + (int64_t)u * (kThreads / 64) * per + t;
      const bool in = t < per && tok < hi;
      const int v = p.ids[(row0 + (in ? tok : lo)) * p.k + (in ? j : 0)];
      id[u] = in ? v : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool valid = id[u] >= 0 && id[u] < p.E;
      const uint64_t m = __ballot(valid);
      if (valid) atomicAdd(&h[id[u]], 1);
      here += __builtin_popcountll(__ballot(valid && (m & before) == 0));
    }
  }
  if (lane == 0 && here) atomicAdd(&h[p.E], here);
  __syncthreads();
}

__global__ __launch_bounds__(kThreads) void balance_count(const BalanceArgs p) {
  extern __shared__ int hist[];  // E + 1
  const int s = blockIdx.x / p.C, c = blockIdx.x % p.C;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= (p.S * p.G - 1) / p.round + 1; i += kThreads) p.tickets[i * kTicketStride] = 0u;
  count_tokens(p, (int64_t)s * p.L, (int64_t)c * p.chunk, min(p.L, (int64_t)(c + 1) * p.chunk), hist);
  int32_t* out = p.part + (int64_t)blockIdx.x * (p.E + 1);
  for (int e = threadIdx.x; e <= p.E; e += kThreads) out[e] = hist[e];
}

// A sequence is split over G workgroups; each adds up the counts of its chunks
// first, with the logits of its first tokens on their way. ONE: one workgroup
// has it all, counts included, and is the only launch.
template <typename TL, int LANES, int NC, bool VEC, bool ONE>
__global__ __launch_bounds__(kThreads) void balance_main(const BalanceArgs p, int sigmoid) {
  constexpr int kWaves = kThreads / 64;
  extern __shared__ float up[];  // [E]: (f - 1) * coef / (S n), then the counts [E + 1]
  __shared__ double part[kWaves];
  __shared__ bool last;
  using TK = Tokens<TL, LANES, NC, VEC>;
  const int s = ONE ? 0 : blockIdx.x / p.G, gi = ONE ? 0 : blockIdx.x % p.G;
  const int tid = threadIdx.x, lane = tid & 63, l = lane % LANES;
  constexpr int kGroups = kThreads / LANES, kTokens = kGroups * TK::UT;
  const int64_t row0 = (int64_t)s * p.L;
  int64_t t0 = (int64_t)gi * kTokens + tid / LANES;  // the group's tokens: t0, t0 + kGroups, ..
  // the counts' loads go out first (loads return in order), then the tokens'
  constexpr int kAhead = 4;
  const int all = ONE ? 0 : p.C * (p.E + 1);
  const int32_t* cnt = p.part + (int64_t)s * all;
  int c[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) c[i] = tid + i * kThreads < all ? cnt[tid + i * kThreads] : 0;
  TK now;
  if (p.L > 0) now.load(p, row0, t0, kGroups, l);
  int* const hist = reinterpret_cast<int*>(up + p.E);
  if constexpr (ONE) {
    count_tokens(p, row0, 0, p.L, hist);
  } else {
    for (int e = tid; e <= p.E; e += kThreads) hist[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (tid + i * kThreads < all) atomicAdd(&hist[(tid + i * kThreads) % (p.E + 1)], c[i]);
    for (int i = tid + kAhead * kThreads; i < all; i += kThreads) atomicAdd(&hist[i % (p.E + 1)], cnt[i]);
    __syncthreads();
  }
  const int n = hist[p.E];
  const float base = n > 0 ? p.coef / ((float)p.S * (float)n) : 0.f;
  for (int e = tid; e < p.E; e += kThreads) {
    // (f - 1) * base, f - 1 = (c E - k n) / (k n) from whole numbers, rounded to float32 once
    const double kn = (double)p.k * (double)n;
    up[e] = n > 0 ? base * (float)(((double)hist[e] * (double)p.E - kn) / kn) : 0.f;
    if (gi == 0) p.counts[(int64_t)s * p.E + e] = hist[e];
  }
  __syncthreads();
  float w[NC][4];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int e = 4 * (l + LANES * i) + r;
      w[i][r] = e < p.E ? up[e] : 0.f;
    }
  double sum = 0.0;
  while (t0 - tid / LANES < p.L) {
    TK next;
    const int64_t t1 = t0 + (int64_t)(ONE ? 1 : p.G) * kTokens;
    next.load(p, row0, t1, kGroups, l);
    now.work(p, row0, t0, kGroups, lane, sigmoid, base, w, sum);
    now = next;
    t0 = t1;
  }
  // the groups of a wave, its waves, then (the last workgroup) all of them, in a fixed order
  double v = l == 0 ? sum : 0.0;
  for (int o = LANES; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  if (lane == 0) part[tid >> 6] = v;
  __syncthreads();
  if (tid < 64) {
    v = lane < kWaves ? part[lane] : 0.0;
    for (int o = 1; o < kWaves; o <<= 1) v += __shfl_xor(v, o, 64);
  }
  if (tid == 0) {
    if constexpr (ONE) {
      *p.loss = (float)v;
    } else {
      // The sum is written through to memory and waited for, then a ticket is
      // taken; the last workgroup reads past its caches. (A release would write
      // back the whole L2, the gradient in it: 47 us for 65536 x 128.) Tickets of one
      // word are served one after another, some 11 ns each: every `round` workgroups
      // have one of their own, and the last of each takes one of all rounds.
      const uint32_t r = blockIdx.x / p.round, rounds = (gridDim.x - 1) / p.round + 1;
      const uint32_t mine = min((uint32_t)p.round, gridDim.x - r * p.round);
      __hip_atomic_store(p.sums + blockIdx.x, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      last = __hip_atomic_fetch_add(p.tickets + (1 + r) * kTicketStride, 1u, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT) == mine - 1 &&
             __hip_atomic_fetch_add(p.tickets, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == rounds - 1;
    }
  }
  if constexpr (!ONE) {
    __syncthreads();
    if (!last) return;
    v = 0.0;
    for (int64_t i = tid; i < (int64_t)gridDim.x; i += kThreads)
      v += __hip_atomic_load(p.sums + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
    if (lane == 0) part[tid >> 6] = v;
    __syncthreads();
    if (tid < 64) {
      v = lane < kWaves ? part[lane] : 0.0;
      for (int o = 1; o < kWaves; o <<= 1) v += __shfl_xor(v, o, 64);
      if (tid == 0) *p.loss = (float)v;
    }
  }
}

// Tokens that a workgroup has in flight: lanes a token and tokens a group of
// lanes as launch_main chooses them.
int tokens_at_once(int64_t E) {
  const int lanes = E <= 64 ? 16 : E <= 128 ? 32 : 64;
  return kThreads / lanes * (E <= 256 ? 4 : 1);
}

// One workgroup for a single sequence of at most two rounds of its tokens (in a graph, one launch of
// one workgroup and two launches: 64 experts, one round 7.7 and 11.7 us, two 11.1 and 12.3, three 15.3
// and 12.4; 512 experts 5.8 and 9.9, 7.8 and 10.6, 9.8 and 10.6).
bool balance_one(int64_t L, int64_t S, int64_t E) { return S == 1 && L <= 2 * tokens_at_once(E); }

template <typename TL, int LANES, int NC, bool VEC>
hipError_t run_main(const BalanceArgs& a, int sigmoid, hipStream_t stream) {
  const size_t lds = (size_t)(2 * a.E + 1) * 4;
  if (balance_one(a.L, a.S, a.E))
    hipLaunchKernelGGL((balance_main<TL, LANES, NC, VEC, true>), dim3(1), dim3(kThreads), lds, stream, a, sigmoid);
  else
    hipLaunchKernelGGL((balance_main<TL, LANES, NC, VEC, false>), dim3((unsigned)(a.S * a.G)), dim3(kThreads), lds, stream, a,
                       sigmoid);
  return hipGetLastError();
}

template <typename TL, bool VEC>
hipError_t launch_main(const BalanceArgs& a, int sigmoid, hipStream_t stream) {
  if (a.E <= 64) return run_main<TL, 16, 1, VEC>(a, sigmoid, stream);
  if (a.E <= 128) return run_main<TL, 32, 1, VEC>(a, sigmoid, stream);
  if (a.E <= 256) return run_main<TL, 64, 1, VEC>(a, sigmoid, stream);
  return run_main<TL, 64, 4, VEC>(a, sigmoid, stream);
}

int64_t align256(int64_t b) { return (b + 255) & ~int64_t(255); }

// chunks of a sequence in the count, workgroups of a sequence in the main pass
int count_chunks(int64_t L) { return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxChunks, (L + 255) / 256)); }
int main_groups(int64_t L, int64_t S, int64_t E) {
  const int tokens = tokens_at_once(E);
  return (int)std::max<int64_t>(1, std::min<int64_t>((L + tokens - 1) / tokens, std::max<int64_t>(1, kMainGroups / S)));
}

// Workgroups that share a ticket: about as many as there are tickets.
int ticket_round(int64_t n) {
  int r = 16;
  while ((int64_t)r * r < n) r *= 2;
  return r;
}
int64_t tickets_bytes(int64_t n) { return align256((1 + (n - 1) / ticket_round(n) + 1) * kTicketStride * 4); }

}  // namespace

size_t balance_workspace_bytes(int64_t T, int64_t S, int64_t E) {
  const int64_t L = T / S;
  if (balance_one(L, S, E)) return 0;
  const int64_t n = S * main_groups(L, S, E);
  return (size_t)(tickets_bytes(n) + align256(n * 8) + align256(S * count_chunks(L) * (E + 1) * 4));
}

hipError_t launch_balance(const Balance& b, int64_t T, int64_t S, int64_t E, int64_t topk, void* ws,
                          hipStream_t stream) {
  BalanceArgs a{};
  a.L = T / S;
  a.S = (int)S;
  a.E = (int)E;
  a.k = (int)topk;
  a.C = count_chunks(a.L);
  a.G = main_groups(a.L, S, E);
  a.chunk = (int)((a.L + a.C - 1) / a.C);
  a.coef = b.coef;
  a.logits = b.logits;
  a.ids = b.ids;
  a.loss = b.loss;
  a.counts = b.counts;
  a.grad = b.grad;
  uint8_t* w = static_cast<uint8_t*>(ws);
  const int64_t n = S * a.G;
  a.round = ticket_round(n);
  a.tickets = reinterpret_cast<uint32_t*>(w);
  a.sums = reinterpret_cast<double*>(w + tickets_bytes(n));
  a.part = reinterpret_cast<int32_t*>(w + tickets_bytes(n) + align256(n * 8));
  if (!balance_one(a.L, S, E)) {
    hipLaunchKernelGGL(balance_count, dim3((unsigned)(S * a.C)), dim3(kThreads), (size_t)(E + 1) * 4, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (E % 4 == 0) return b.bf16 ? launch_main<uint16_t, true>(a, b.sigmoid, stream) : launch_main<float, true>(a, b.sigmoid, stream);
  return b.bf16 ? launch_main<uint16_t, false>(a, b.sigmoid, stream) : launch_main<float, false>(a, b.sigmoid, stream);
}

}  // namespace w8a8
