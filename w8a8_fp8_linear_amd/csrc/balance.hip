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

constexpr int kCountThreads = 1024;
constexpr int kMaxChunks = 32;  // of a sequence: every workgroup of the main pass adds them up

struct BalanceArgs {
  const void* logits;   // [S L, E]
  const int32_t* ids;   // [S L, k]
  int32_t* part;        // [S, C, E + 1]: copies of a chunk's tokens by expert, its tokens that count
  double* sums;         // [S G]
  uint32_t* ticket;
  float* loss;          // [1]
  int32_t* counts;      // [S, E]
  void* grad;           // [S L, E] or NULL
  int64_t L;
  int S, E, k, C, G, chunk;
  float coef;
};

__global__ __launch_bounds__(kCountThreads) void balance_count(const BalanceArgs p) {
  extern __shared__ int hist[];  // E + 1
  const int s = blockIdx.x / p.C, c = blockIdx.x % p.C;
  for (int e = threadIdx.x; e <= p.E; e += kCountThreads) hist[e] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0u;
  __syncthreads();
  const int64_t hi = min(p.L, (int64_t)(c + 1) * p.chunk);
  for (int64_t t = (int64_t)c * p.chunk + threadIdx.x; t < hi; t += kCountThreads) {
    const int32_t* id = p.ids + ((int64_t)s * p.L + t) * p.k;
    bool any = false;
    for (int j = 0; j < p.k; ++j) {
      const int e = id[j];
      if (e >= 0 && e < p.E) {
        atomicAdd(&hist[e], 1);
        any = true;
      }
    }
    if (any) atomicAdd(&hist[p.E], 1);
  }
  __syncthreads();
  int32_t* out = p.part + (int64_t)blockIdx.x * (p.E + 1);
  for (int e = threadIdx.x; e <= p.E; e += kCountThreads) out[e] = hist[e];
}

// Four consecutive values of a row, at whatever alignment the row has.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4_any __attribute__((ext_vector_type(4), aligned(2)));

__device__ inline void load4(const float* p, int left, float* v) {
  if (left >= 4) {
    const f32x4_any x = *reinterpret_cast<const f32x4_any*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[i];
  } else {
    for (int i = 0; i < 4; ++i) v[i] = i < left ? p[i] : -INFINITY;
  }
}
__device__ inline void load4(const uint16_t* p, int left, float* v) {
  if (left >= 4) {
    const u16x4_any x = *reinterpret_cast<const u16x4_any*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float((uint32_t)x[i] << 16);
  } else {
    for (int i = 0; i < 4; ++i) v[i] = i < left ? __uint_as_float((uint32_t)p[i] << 16) : -INFINITY;
  }
}
__device__ inline void store4(float* p, int left, const float* v) {
  if (left >= 4)
    *reinterpret_cast<f32x4_any*>(p) = f32x4_any{v[0], v[1], v[2], v[3]};
  else
    for (int i = 0; i < left; ++i) p[i] = v[i];
}
__device__ inline void store4(uint16_t* p, int left, const float* v) {
  const uint32_t lo = bf16x2_rne(v[0], v[1]), hi = bf16x2_rne(v[2], v[3]);
  const uint16_t h[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
  if (left >= 4)
    *reinterpret_cast<u16x4_any*>(p) = u16x4_any{h[0], h[1], h[2], h[3]};
  else
    for (int i = 0; i < left; ++i) p[i] = h[i];
}

template <int LANES>
__device__ inline float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}
template <int LANES>
__device__ inline float group_max(float v) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

// LANES lanes a token, NC pieces of four values a lane.
template <typename TL, int LANES, int NC>
__global__ __launch_bounds__(256) void balance_main(const BalanceArgs p, int sigmoid) {
  extern __shared__ float up[];  // [E]: (f - 1) * coef / (S n)
  __shared__ int total;
  __shared__ double part[4];
  __shared__ bool last;
  const int s = blockIdx.x / p.G, gi = blockIdx.x % p.G;
  const int tid = threadIdx.x, lane = tid & 63;
  const int32_t* cnt = p.part + (int64_t)s * p.C * (p.E + 1);
  if (tid < 64) {
    int n = tid < p.C ? cnt[(int64_t)tid * (p.E + 1) + p.E] : 0;
    for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o, 64);
    if (tid == 0) total = n;
  }
  __syncthreads();
  const int n = total;
  const float base = n > 0 ? p.coef / ((float)p.S * (float)n) : 0.f;
  for (int e = tid; e < p.E; e += 256) {
    int c = 0;
    for (int i = 0; i < p.C; ++i) c += cnt[(int64_t)i * (p.E + 1) + e];
    const double kn = (double)p.k * (double)n;
    up[e] = n > 0 ? base * (float)(((double)c * (double)p.E - kn) / kn) : 0.f;
    if (gi == 0) p.counts[(int64_t)s * p.E + e] = c;
  }
  __syncthreads();
  constexpr int kTokens = 256 / LANES;
  const int l = lane % LANES;
  const uint64_t group = LANES == 64 ? ~0ull : ((1ull << (LANES & 63)) - 1) << (lane - l);
  const TL* logits = static_cast<const TL*>(p.logits);
  TL* grad = static_cast<TL*>(p.grad);
  float w[NC][4];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int e = 4 * (l + LANES * i) + r;
      w[i][r] = e < p.E ? up[e] : 0.f;
    }
  double sum = 0.0;
  for (int64_t t0 = (int64_t)gi * kTokens; t0 < p.L; t0 += (int64_t)p.G * kTokens) {
    const int64_t t = t0 + tid / LANES;
    const bool in = t < p.L;
    const int64_t row = (int64_t)s * p.L + (in ? t : 0);
    float x[NC][4];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int e = 4 * (l + LANES * i);
      load4(logits + row * p.E + e, p.E - e, x[i]);
    }
    bool any = false;
    for (int j = l; j < p.k; j += LANES) {
      const int e = p.ids[row * p.k + j];
      any |= e >= 0 && e < p.E;
    }
    const bool here = in && (__ballot(any) & group) != 0;
    float m = -INFINITY;
    if (!sigmoid) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = fmaxf(m, x[i][r]);
      m = group_max<LANES>(m);
      m = m == -INFINITY ? 0.f : m;
    }
    float slope[NC][4], z = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = sigmoid ? 1.0f / (1.0f + __expf(-x[i][r])) : __expf(x[i][r] - m);
        slope[i][r] = sigmoid ? 1.0f - v : 1.0f;
        x[i][r] = v;
        z += v;
      }
    z = group_sum<LANES>(z);
    const float inv = z > 0.f ? 1.0f / z : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[i][r] *= inv;
        dot = __builtin_fmaf(w[i][r], x[i][r], dot);
      }
    dot = group_sum<LANES>(dot);
    if (here) sum += (double)dot + (z > 0.f ? (double)base : 0.0);
    if (grad && in) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int e = 4 * (l + LANES * i);
        float d[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) d[r] = here ? x[i][r] * slope[i][r] * (w[i][r] - dot) : 0.f;
        store4(grad + row * p.E + e, p.E - e, d);
      }
    }
  }
  // the groups of a wave, its waves, then (the last workgroup) all of them, in a fixed order
  double v = l == 0 ? sum : 0.0;
  for (int o = LANES; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  if (lane == 0) part[tid >> 6] = v;
  __syncthreads();
  if (tid == 0) {
    __hip_atomic_store(p.sums + blockIdx.x, (part[0] + part[1]) + (part[2] + part[3]), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  v = 0.0;
  for (int64_t i = tid; i < (int64_t)gridDim.x; i += 256)
    v += __hip_atomic_load(p.sums + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  if (lane == 0) part[tid >> 6] = v;
  __syncthreads();
  if (tid == 0) *p.loss = (float)((part[0] + part[1]) + (part[2] + part[3]));
}

template <typename TL>
hipError_t run_main(const BalanceArgs& a, int sigmoid, hipStream_t stream) {
  const dim3 grid((unsigned)(a.S * a.G));
  const size_t lds = (size_t)a.E * 4;
  if (a.E <= 64)
    hipLaunchKernelGGL((balance_main<TL, 16, 1>), grid, dim3(256), lds, stream, a, sigmoid);
  else if (a.E <= 128)
    hipLaunchKernelGGL((balance_main<TL, 32, 1>), grid, dim3(256), lds, stream, a, sigmoid);
  else if (a.E <= 256)
    hipLaunchKernelGGL((balance_main<TL, 64, 1>), grid, dim3(256), lds, stream, a, sigmoid);
  else
    hipLaunchKernelGGL((balance_main<TL, 64, 4>), grid, dim3(256), lds, stream, a, sigmoid);
  return hipGetLastError();
}

int64_t align256(int64_t b) { return (b + 255) & ~int64_t(255); }

// chunks of a sequence in the count, workgroups of a sequence in the main pass
int count_chunks(int64_t L) { return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxChunks, (L + 255) / 256)); }
int main_groups(int64_t L, int64_t S, int64_t E) {
  const int tokens = E <= 64 ? 16 : E <= 128 ? 8 : 4;
  return (int)std::max<int64_t>(1, std::min<int64_t>((L + tokens - 1) / tokens, std::max<int64_t>(1, 1024 / S)));
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int64_t S, int64_t E) {
  const int64_t L = T / S;
  return (size_t)(256 + align256(S * main_groups(L, S, E) * 8) + align256(S * count_chunks(L) * (E + 1) * 4));
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
  a.ticket = reinterpret_cast<uint32_t*>(w);
  a.sums = reinterpret_cast<double*>(w + 256);
  a.part = reinterpret_cast<int32_t*>(w + 256 + align256(S * a.G * 8));
  hipLaunchKernelGGL(balance_count, dim3((unsigned)(S * a.C)), dim3(kCountThreads), (size_t)(E + 1) * 4, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return b.bf16 ? run_main<uint16_t>(a, b.sigmoid, stream) : run_main<float>(a, b.sigmoid, stream);
}

}  // namespace w8a8
