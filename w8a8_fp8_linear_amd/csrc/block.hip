// FP8 with a scale per block of 128: quantisers, the dense product, and the
// routed-expert pass.
//
// The pages' FP8 scheme rounds a layer's input to FP8 at run time and
// multiplies it with FP8 weights on the FP8 matrix units (Lernex/Metis-1.6-
// Logos-FP8, "What --fast-math does"), with one scale per token and one per
// output channel. Here a scale covers less: 128 consecutive values of a row of
// activations, 128 x 128 values of a weight matrix, so that one outlier costs
// 128 values their small digits and not a whole row. A K step of the
// 16x16x128 E4M3 MFMA is one block:
//   y[m,n] = sum_b sa[b,m] * sw[n/128,b] * sum_{k in block b} a[m,k] w[n,k]
// Every MFMA starts from C = 0 and its four results are added to the float32
// accumulators times the product of the two scales: four FMAs of the vector
// unit to an MFMA (16 of its 32 cycles).
#include <algorithm>

#include "device.h"
#include "grouped.h"
#include "launch.h"
#include "widen.h"

namespace w8a8 {
namespace {

// ---- quantisers ------------------------------------------------------------

// Maximum over each row of 16 lanes, in every lane: swaps inside quads, then
// mirrored halves and rows, all by DPP.
__device__ inline uint32_t row16_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  return v;
}

// Activations. A workgroup takes 16 rows x 4 blocks: a wave loads 1 KB of each
// of its four rows, 16 lanes a block. The scales meet in LDS: 16 rows' are one
// 64-byte piece of the [blocks, M] array.
constexpr int kQuantRows = 16, kQuantBlocks = 4;

__global__ __launch_bounds__(256) void quant_row_blocks(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                        int pieces, uint8_t* __restrict__ q,
                                                        float* __restrict__ scale) {
  __shared__ float sc[kQuantBlocks][kQuantRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = (int64_t)(blockIdx.x / (uint32_t)pieces) * kQuantRows;
  const int64_t b0 = (int64_t)(blockIdx.x % (uint32_t)pieces) * kQuantBlocks, k = (b0 << 7) + 8 * lane;
  v4i v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 4 * wave + i;
    v[i] = v4i{0, 0, 0, 0};
    if (row < M && k < K) v[i] = *reinterpret_cast<const v4i*>(x + row * K + k);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 4 * wave + i;
    const uint4 u = make_uint4((uint32_t)v[i].x, (uint32_t)v[i].y, (uint32_t)v[i].z, (uint32_t)v[i].w);
    const float s = row_scale(row16_max(absmax8(u)));
    if (row < M && k < K) *reinterpret_cast<uint2*>(q + row * K + k) = quant8(u, s, 1.0f / s);
    if ((lane & 15) == 0) sc[lane >> 4][4 * wave + i] = s;
  }
  __syncthreads();
  if (threadIdx.x < kQuantBlocks * kQuantRows) {
    const int b = threadIdx.x / kQuantRows, r = threadIdx.x % kQuantRows;
    if (row0 + r < M && (b0 + b) << 7 < K) scale[(b0 + b) * M + row0 + r] = sc[b][r];
  }
}

// Weights: a workgroup per 128 x 128 block, held in registers between the
// maximum and the codes.
__global__ __launch_bounds__(256) void quant_weight_blocks(const uint16_t* __restrict__ w, int64_t N, int64_t K,
                                                           int nb, int kb, uint8_t* __restrict__ q,
                                                           float* __restrict__ scale) {
  __shared__ uint32_t wmax[4];
  const int64_t e = blockIdx.x / (uint32_t)(nb * kb);
  const int rest = (int)(blockIdx.x - e * (nb * kb));
  const int64_t n0 = (int64_t)(rest / kb) * 128, k = (int64_t)(rest % kb) * 128 + 8 * (threadIdx.x & 15);
  const int r0 = threadIdx.x >> 4;
  const uint16_t* src = w + (e * N + n0) * K + k;
  v4i v[8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = v4i{0, 0, 0, 0};
    if (n0 + r0 + 16 * i < N && k < K) v[i] = *reinterpret_cast<const v4i*>(src + (int64_t)(r0 + 16 * i) * K);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    amax = max(amax, absmax8(make_uint4((uint32_t)v[i].x, (uint32_t)v[i].y, (uint32_t)v[i].z, (uint32_t)v[i].w)));
  amax = wave_max_u32(amax);
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = amax;
  __syncthreads();
  const float s = row_scale(max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])));
  const float r = 1.0f / s;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (n0 + r0 + 16 * i < N && k < K)
      *reinterpret_cast<uint2*>(q + (e * N + n0 + r0 + 16 * i) * K + k) =
          quant8(make_uint4((uint32_t)v[i].x, (uint32_t)v[i].y, (uint32_t)v[i].z, (uint32_t)v[i].w), s, r);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
}

// Weight scales, one value for a wave, are read through the constant address
// space: scalar loads, whose counter is not that of the loads into LDS.
typedef const __attribute__((address_space(4))) float* ScalarPtr;

// ---- products of at most 32 rows ---------------------------------------------

// Both kernels: NT tiles of 16 weight rows a workgroup, K split over 4 waves, 4
// steps of 128 columns in flight a wave; the waves' sums meet in LDS, and each
// wave adds and stores its share of the tiles.
constexpr int kSkinnyU = 4, kSkinnyCols = 4 * kSkinnyU * 128;  // columns of a round

// The weight fragments of a wave's steps kb0 + wave + 4 u, tile i from row
// i * stride of the resource on, and the scales of their NS blocks of rows.
template <int U, int NT, int NS>
__device__ inline void skinny_weights(__amdgpu_buffer_rsrc_t rW, uint32_t stride, const ScalarPtr (&sWrow)[NS], int kb0,
                                      int nk, int K, int wave, int r16, int g, v8i (&wf)[U][NT], float (&sw)[U][NS]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int kb = kb0 + wave + 4 * u;
    const bool live = kb < nk;
    const int c0 = (kb << 7) + 16 * g, c1 = c0 + 64;
    const uint32_t o0 = live && c0 < K ? (uint32_t)c0 : kOutOfRange;
    const uint32_t o1 = live && c1 < K ? (uint32_t)c1 : kOutOfRange;
#pragma unroll
    for (int i = 0; i < NS; ++i) sw[u][i] = sWrow[i][live ? kb : 0];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint32_t wrow = ((uint32_t)i * stride + (uint32_t)r16) * (uint32_t)K;
      const v4i lo = buffer_load16(rW, o0 == kOutOfRange ? o0 : wrow + o0);
      const v4i hi = buffer_load16(rW, o1 == kOutOfRange ? o1 : wrow + o1);
      wf[u][i] = v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    }
  }
}

// acc += (w . x) * s
__device__ inline void scaled_mfma(v4f& acc, v8i w, v8i x, float s) {
  const v4f d = mfma_16x16x128_e4m3(w, x, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
  for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(d[r], s, acc[r]);
}

// Sum of tile it over the waves, for a wave that has it.
template <int TILES>
__device__ inline v4f add_waves(const v4f* red, int it, int lane) {
  return red[it * 64 + lane] + red[(TILES + it) * 64 + lane] + red[(2 * TILES + it) * 64 + lane] +
         red[(3 * TILES + it) * 64 + lane];
}

template <int NT, int MT>
__device__ inline void skinny_store(const v4f (&acc)[NT][MT], v4f* red, int wave, int lane, int n0, uint16_t* Y, int M,
                                    int N) {
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) red[((wave * NT + i) * MT + t) * 64 + lane] = acc[i][t];
  lds_barrier();
#pragma unroll
  for (int o = 0; o < (NT * MT + 3) / 4; ++o) {
    const int it = wave + 4 * o;
    if (it >= NT * MT) break;
    const int n = n0 + it / MT * 16 + 4 * (lane >> 4), m = it % MT * 16 + (lane & 15);
    const v4f a = add_waves<NT * MT>(red, it, lane);
    if (n < N && m < M)
      *reinterpret_cast<uint2*>(Y + (int64_t)m * N + n) = make_uint2(bf16x2_rne(a[0], a[1]), bf16x2_rne(a[2], a[3]));
  }
}

// On codes. Up to 16 rows (MT = 1) their fragments come straight from memory;
// XL: through LDS, as whole 128-byte row pieces (8 rows an instruction, straight
// into LDS), for 17 to 32 rows.
template <int MT, int NT, bool XL>
__global__ __launch_bounds__(256) void block_skinny(const uint8_t* __restrict__ X, const float* __restrict__ sA,
                                                    const uint8_t* __restrict__ W, const float* __restrict__ sW,
                                                    uint16_t* __restrict__ Y, int M, int N, int K) {
  constexpr int U = kSkinnyU, kXRows = 16 * MT;
  constexpr int kXBytes = XL ? 4 * U * kXRows * 128 : 0, kRedBytes = 4 * NT * MT * 64 * 16;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kXBytes > kRedBytes ? kXBytes : kRedBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16 * NT;
  const auto rW = make_rsrc(W + (int64_t)n0 * K, (int64_t)(N - n0) * K);
  const auto rX = make_rsrc(X, (int64_t)M * K);
  const int r16 = lane & 15, g = lane >> 4;
  const int nk = (K + 127) >> 7;
  const auto rS = make_rsrc(sA, (int64_t)nk * M * 4);
  const ScalarPtr sWrow[1] = {(ScalarPtr)(sW + (int64_t)(n0 >> 7) * nk)};  // 16 NT rows of one weight block
  v4f acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[i][t] = v4f{0.f, 0.f, 0.f, 0.f};
  uint8_t* const xs = smem + wave * (U * kXRows * 128);  // XL: this wave's rows, by step
  for (int kb0 = 0; kb0 < nk; kb0 += 4 * U) {
    v8i wf[U][NT], xf[U][MT];
    float sx[U][MT], sw[U][1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + wave + 4 * u;
      const bool live = kb < nk;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int row = t * 16 + r16;
        sx[u][t] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            rS, live && row < M ? (uint32_t)(kb * M + row) * 4u : kOutOfRange, 0, 0));
      }
      if constexpr (XL) {
#pragma unroll
        for (int q = 0; q < 2 * MT; ++q) {
          if (8 * q < M) {
            const int row = 8 * q + (lane >> 3), c = (kb << 7) + 16 * ((lane & 7) ^ (row & 7));
            buffer_load16_lds(rX, xs + (u * kXRows + 8 * q) * 128,
                              live && row < M && c < K ? (uint32_t)row * (uint32_t)K + (uint32_t)c : kOutOfRange);
          }
        }
      } else {
        const int c0 = (kb << 7) + 16 * g, c1 = c0 + 64;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const uint32_t xrow = (uint32_t)(t * 16 + r16) * (uint32_t)K;
          const v4i lo = buffer_load16(rX, live && c0 < K ? xrow + (uint32_t)c0 : kOutOfRange);
          const v4i hi = buffer_load16(rX, live && c1 < K ? xrow + (uint32_t)c1 : kOutOfRange);
          xf[u][t] = v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        }
      }
    }
    // XL: the wait below counts on the weights' loads, 2 U NT of them, to be the last that were issued
    if constexpr (XL) __builtin_amdgcn_sched_barrier(0);
    skinny_weights(rW, 16, sWrow, kb0, nk, K, wave, r16, g, wf, sw);
    if constexpr (XL) {
      // the loads return in order: the rows have landed once only the weights' are outstanding
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt<2 * U * NT>();
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < MT; ++t) xf[u][t] = lds_frag(xs + u * kXRows * 128, t * 16 + r16, g);
    }
    // every load of the round ahead of the first MFMA
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const float s = sx[u][t] * sw[u][0];
#pragma unroll
        for (int i = 0; i < NT; ++i) scaled_mfma(acc[i][t], wf[u][i], xf[u][t], s);
      }
  }
  if constexpr (XL) lds_barrier();
  skinny_store<NT, MT>(acc, reinterpret_cast<v4f*>(smem), wave, lane, n0, Y, M, N);
}

// Some more rows: 16 SM x 16 SN outputs a workgroup, its 4 waves split K, U steps
// a wave in flight, fragments straight from memory (L2). No barrier until the
// sums meet: a few hundred rows have too few tiles to fill the GPU, and their time
// is the chain of loads, which a tile whose waves share K steps walks four times
// as often.
template <int SM, int SN, int U>
__global__ __launch_bounds__(256) void block_ksplit(const uint8_t* __restrict__ X, const float* __restrict__ sA,
                                                    const uint8_t* __restrict__ W, const float* __restrict__ sW,
                                                    uint16_t* __restrict__ Y, int M, int N, int K, int tiles_m,
                                                    int tiles_n) {
  constexpr int kTiles = SM * SN;
  static_assert(kTiles % 4 == 0 && 128 % (16 * SN) == 0, "tiles go round the waves; one block of weight rows");
  __shared__ v4f red[4 * kTiles * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn;
  map_tile<4>(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int m0 = tm * 16 * SM, n0 = tn * 16 * SN;
  const auto rW = make_rsrc(W + (int64_t)n0 * K, (int64_t)(N - n0) * K);
  const auto rX = make_rsrc(X + (int64_t)m0 * K, (int64_t)(M - m0) * K);
  const int r16 = lane & 15, g = lane >> 4;
  const int nk = (K + 127) >> 7;
  const ScalarPtr sWrow[1] = {(ScalarPtr)(sW + (int64_t)(n0 >> 7) * nk)};
  v4f acc[SN][SM];
#pragma unroll
  for (int i = 0; i < SN; ++i)
#pragma unroll
    for (int j = 0; j < SM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int kb0 = 0; kb0 < nk; kb0 += 4 * U) {
    v8i wf[U][SN], xf[U][SM];
    float sx[U][SM], sw[U][1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + wave + 4 * u;
      const bool live = kb < nk;
      const int c0 = (kb << 7) + 16 * g, c1 = c0 + 64;
      const auto rS = make_rsrc(sA + (int64_t)(live ? kb : 0) * M + m0, (int64_t)(M - m0) * 4);
#pragma unroll
      for (int j = 0; j < SM; ++j) {
        const uint32_t row = (uint32_t)(j * 16 + r16);
        sx[u][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rS, live ? row * 4u : kOutOfRange, 0, 0));
        const v4i lo = buffer_load16(rX, live && c0 < K ? row * (uint32_t)K + (uint32_t)c0 : kOutOfRange);
        const v4i hi = buffer_load16(rX, live && c1 < K ? row * (uint32_t)K + (uint32_t)c1 : kOutOfRange);
        xf[u][j] = v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      }
    }
    skinny_weights(rW, 16, sWrow, kb0, nk, K, wave, r16, g, wf, sw);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < SN; ++i)
#pragma unroll
        for (int j = 0; j < SM; ++j) scaled_mfma(acc[i][j], wf[u][i], xf[u][j], sx[u][j] * sw[u][0]);
  }
#pragma unroll
  for (int i = 0; i < SN; ++i)
#pragma unroll
    for (int j = 0; j < SM; ++j) red[((wave * SN + i) * SM + j) * 64 + lane] = acc[i][j];
  lds_barrier();
#pragma unroll
  for (int o = 0; o < kTiles / 4; ++o) {
    const int it = wave + 4 * o, n = n0 + it / SM * 16 + 4 * g, m = m0 + it % SM * 16 + r16;
    const v4f a = add_waves<kTiles>(red, it, lane);
    if (n < N && m < M)
      *reinterpret_cast<uint2*>(Y + (int64_t)m * N + n) = make_uint2(bf16x2_rne(a[0], a[1]), bf16x2_rne(a[2], a[3]));
  }
}

// On BF16 input of at most 16 rows: the workgroup quantises it into LDS, 8
// values of a row a thread and 16 lanes a block, every value once a workgroup
// (in the MFMA's own layout, with its 16 columns for a single row, this took
// 8.8 us for one row of 8192 x 2048). XR rows are taken, of which M are there.
template <int XR, int NT>
__global__ __launch_bounds__(256) void block_skinny_bf16(const uint16_t* __restrict__ X, const uint8_t* __restrict__ W,
                                                         const float* __restrict__ sW, uint16_t* __restrict__ Y, int M,
                                                         int N, int K) {
  constexpr int U = kSkinnyU;
  // codes [step of the round][row][128 bytes, 16-byte pieces swizzled by row], the
  // steps' scales; then the waves' sums
  constexpr int kCodeBytes = 4 * U * 16 * 128;
  static_assert(kCodeBytes >= 4 * NT * 64 * 16, "the sums take the codes' place");
  __shared__ __attribute__((aligned(16))) uint8_t smem[kCodeBytes + 4 * U * 16 * 4];
  float* const xs = reinterpret_cast<float*>(smem + kCodeBytes);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16 * NT;
  const auto rW = make_rsrc(W + (int64_t)n0 * K, (int64_t)(N - n0) * K);
  const auto rX = make_rsrc(X, (int64_t)M * K * 2);
  const int r16 = lane & 15, g = lane >> 4;
  const int nk = (K + 127) >> 7;
  const ScalarPtr sWrow[1] = {(ScalarPtr)(sW + (int64_t)(n0 >> 7) * nk)};  // 16 NT rows of one weight block
  v4f acc[NT][1];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = v4f{0.f, 0.f, 0.f, 0.f};
  const int step = tid >> 4, piece = (tid & 15) >> 1;  // the block of the round that this thread's columns lie in
  for (int k0 = 0; k0 < K; k0 += kSkinnyCols) {
    // the round's loads: 8 columns of the rows, then the weights (the counter is
    // in order, and the rows are needed first)
    const int c = k0 + 8 * tid;
    v4i xv[XR];
#pragma unroll
    for (int m = 0; m < XR; ++m)
      xv[m] = buffer_load16(rX, c < K && m < M ? ((uint32_t)m * (uint32_t)K + (uint32_t)c) * 2u : kOutOfRange);
    v8i wf[U][NT];
    float sw[U][1];
    skinny_weights(rW, 16, sWrow, k0 >> 7, nk, K, wave, r16, g, wf, sw);
    // every load of the round ahead of the first use
    __builtin_amdgcn_sched_barrier(0);
    if (k0) lds_barrier();  // the round before has been read
#pragma unroll
    for (int m = 0; m < XR; ++m) {
      const uint4 b = make_uint4((uint32_t)xv[m].x, (uint32_t)xv[m].y, (uint32_t)xv[m].z, (uint32_t)xv[m].w);
      const float s = row_scale(row16_max(absmax8(b)));
      *reinterpret_cast<uint2*>(smem + (step * 16 + m) * 128 + ((piece ^ (m & 7)) << 4) + (tid & 1) * 8) =
          quant8(b, s, 1.0f / s);
      if ((tid & 15) == 0) xs[step * 16 + m] = s;
    }
    lds_barrier();
    // rows from XR on are whatever the LDS held: their columns are not stored
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int st = wave + 4 * u;
      if ((k0 >> 7) + st >= nk) break;
      const v8i xf = lds_frag(smem + st * 16 * 128, r16, g);
      const float s = xs[st * 16 + r16] * sw[u][0];
#pragma unroll
      for (int i = 0; i < NT; ++i) scaled_mfma(acc[i][0], wf[u][i], xf, s);
    }
  }
  lds_barrier();
  skinny_store<NT, 1>(acc, reinterpret_cast<v4f*>(smem), wave, lane, n0, Y, M, N);
}

// E4M3 codes of four float32 values over a block's scale s, r = fl32(1 / s): the
// quotient by one residual correction (quant8); tiny scales divide.
__device__ inline uint32_t codes4(const float* h, float s, float r) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q0 = h[i] * r;
    v[i] = clamp448(s >= kQuotientMinScale ? __builtin_fmaf(__builtin_fmaf(-q0, s, h[i]), r, q0) : h[i] / s);
  }
  return e4m3x4(v[0], v[1], v[2], v[3]);
}

// Scale of a block of float32 values from the bits of its largest magnitude
// (infinity and NaN come last among the bits and stay).
__device__ inline float block_scale_f32(uint32_t amax) { return amax == 0u ? 1.0f : __uint_as_float(amax) / 448.0f; }

// ---- routed experts, few rows each -----------------------------------------------

// A group's rows are few: the weights are streamed as for the dense products of
// few rows, 16 rows of x at a time, and the groups are found from the ids by
// each workgroup itself, without the launches that sort them. With no more
// routed copies (slots) than experts a group is a slot, and the first slot of
// an expert works for all of them; otherwise a group is an expert.
constexpr int kFewSlots = 256;

struct BlockFewArgs {
  const uint8_t* x;    // [T, H] codes
  const float* sx;     // [blocks of H, T]
  const int32_t* ids;  // [T, topk]
  const float* tw;     // [T, topk]
  const uint8_t *w13, *w2;
  const float *s13, *s2;
  float* h;            // [slots, I]
  float* y;            // [slots, H] weighted rows
  int T, H, I, E, topk, n, by_slot;
};

// The expert of group `grp` and, in LDS, its slots in order; the number of slots
// (0: nothing to do). Every wave writes the same list; a barrier follows. All ids
// are loaded at once, the group's own among them: one latency before the weights.
__device__ inline int few_group(const BlockFewArgs& p, int grp, int lane, int* list, int& e) {
  constexpr int kPer = kFewSlots / 64;
  int id[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (64 * i < p.n) id[i] = p.ids[64 * i + lane < p.n ? 64 * i + lane : 0];
  e = grp;
  if (p.by_slot) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (grp >> 6 == i) e = __builtin_amdgcn_readlane(id[i], grp & 63);
  }
  if (e < 0 || e >= p.E) return 0;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (64 * i >= p.n) break;
    const int s = 64 * i + lane;
    const bool mine = s < p.n && id[i] == e;
    const uint64_t m = __ballot(mine);
    if (mine) list[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u))] = s;
    if (p.by_slot && n == 0 && m != 0 && 64 * i + __builtin_ctzll(m) != grp) return 0;  // not the first
    n += __builtin_popcountll(m);
  }
  return n;
}

// 32 E4M3 codes of a lane (an FP8 fragment) -> four BF16 fragments of 8 values,
// two values an instruction, exactly.
__device__ inline void widen32(v8i q, v4i (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t c = (uint32_t)q[2 * i + j];
      w[i][2 * j] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
      w[i][2 * j + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true));
    }
}

// h of 16 columns: 16 gate and 16 up rows of W13, K split over the waves. The
// codes of both operands are widened to BF16, whose matrix unit sums near
// float32 (2^-21.7 of the terms against the FP8 unit's 2^-11.6): h is quantised
// next, and each of its values that the FP8 unit's sum puts on the other side of
// an E4M3 border moves every output of the token. With the weight stream as the
// bound the conversions (48 a step) cost little.
template <int U>
__global__ __launch_bounds__(256) void block_few_gate_up(const BlockFewArgs p) {
  __shared__ int list[kFewSlots];
  __shared__ v4f red[4 * 2 * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = p.I / 16, grp = blockIdx.x / tiles, i0 = (blockIdx.x % tiles) * 16;
  int e;
  const int n = few_group(p, grp, lane, list, e);
  if (n == 0) return;
  lds_barrier();
  const int H = p.H, I = p.I, nk = (H + 127) >> 7;
  const int r16 = lane & 15, g = lane >> 4;
  const auto rW = make_rsrc(p.w13 + ((int64_t)e * 2 * I + i0) * H, (int64_t)(2 * I - i0) * H);
  const auto rX = make_rsrc(p.x, (int64_t)p.T * H);
  const auto rS = make_rsrc(p.sx, (int64_t)nk * p.T * 4);
  const float* s13 = p.s13 + ((int64_t)e * (I / 64) + (i0 >> 7)) * nk;
  const ScalarPtr sWrow[2] = {(ScalarPtr)s13, (ScalarPtr)(s13 + (int64_t)(I / 128) * nk)};
  for (int r0 = 0; r0 < n; r0 += 16) {
    const int slot = r0 + r16 < n ? list[r0 + r16] : -1;
    const uint32_t tok = slot < 0 ? 0u : (uint32_t)(slot / p.topk);
    v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
    for (int kb0 = 0; kb0 < nk; kb0 += 4 * U) {
      v8i wf[U][2], xf[U];
      float sx[U], sw[U][2];
      skinny_weights(rW, (uint32_t)I, sWrow, kb0, nk, H, wave, r16, g, wf, sw);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kb = kb0 + wave + 4 * u;
        const bool live = kb < nk && slot >= 0;
        const int c0 = (kb << 7) + 16 * g, c1 = c0 + 64;
        const v4i lo = buffer_load16(rX, live && c0 < H ? tok * (uint32_t)H + (uint32_t)c0 : kOutOfRange);
        const v4i hi = buffer_load16(rX, live && c1 < H ? tok * (uint32_t)H + (uint32_t)c1 : kOutOfRange);
        xf[u] = v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        sx[u] = __uint_as_float(
            __builtin_amdgcn_raw_buffer_load_b32(rS, live ? ((uint32_t)kb * (uint32_t)p.T + tok) * 4u : kOutOfRange, 0, 0));
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v4i x[4];
        widen32(xf[u], x);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          v4i w[4];
          widen32(wf[u][i], w);
          v4f d = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 4; ++c) d = mfma_16x16x32_bf16(w[c], x[c], d);
          const float s = sx[u] * sw[u][i];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][r] = __builtin_fmaf(d[r], s, acc[i][r]);
        }
      }
    }
    if (r0) lds_barrier();  // the tile before has been added
#pragma unroll
    for (int i = 0; i < 2; ++i) red[(wave * 2 + i) * 64 + lane] = acc[i];
    lds_barrier();
    if (wave == 0 && slot >= 0) {
      const v4f a = add_waves<2>(red, 0, lane), u = add_waves<2>(red, 1, lane);
      *reinterpret_cast<float4*>(p.h + (int64_t)slot * I + i0 + 4 * g) =
          make_float4(silu_f32(a[0]) * u[0], silu_f32(a[1]) * u[1], silu_f32(a[2]) * u[2], silu_f32(a[3]) * u[3]);
    }
  }
}

// y of 64 columns: 64 rows of W2, K split over the waves, one step of 128 each a
// round. h is quantised on its way into LDS, 8 values a thread and 16 lanes a block.
__global__ __launch_bounds__(256) void block_few_down(const BlockFewArgs p) {
  constexpr int NT = 4, kCols = 512;  // columns of a round
  __shared__ int list[kFewSlots];
  __shared__ __attribute__((aligned(16))) uint8_t smem[4 * NT * 64 * 16];  // codes [4][16][128], then the waves' sums
  __shared__ float xs[4 * 16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = (p.H + 63) / 64, grp = blockIdx.x / tiles, n0 = (blockIdx.x % tiles) * 64;
  int e;
  const int n = few_group(p, grp, lane, list, e);
  if (n == 0) return;
  lds_barrier();
  const int H = p.H, I = p.I, nk = I >> 7;
  const int r16 = lane & 15, g = lane >> 4;
  const auto rW = make_rsrc(p.w2 + ((int64_t)e * H + n0) * I, (int64_t)(H - n0) * I);
  const ScalarPtr sWrow[1] = {(ScalarPtr)(p.s2 + ((int64_t)e * ((H + 127) >> 7) + (n0 >> 7)) * nk)};
  for (int r0 = 0; r0 < n; r0 += 16) {
    const int rows = min(16, n - r0);
    v4f acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < I; k0 += kCols) {
      const int c = k0 + 8 * lane, step = lane >> 4, piece = (lane & 15) >> 1;
      v4i ha, hb;
      auto load_h = [&](int r) {  // zeros past the row's end
        const int slot = __builtin_amdgcn_readfirstlane(list[r0 + min(r, rows - 1)]);
        const auto rH = make_rsrc(p.h + (int64_t)slot * I, (int64_t)I * 4);
        ha = buffer_load16(rH, (uint32_t)c * 4u);
        hb = buffer_load16(rH, (uint32_t)c * 4u + 16u);
      };
      // the first rows, then the weights: loads return in order, and the rows are needed first
      load_h(wave);
      v8i wf[1][NT];
      float sw[1][1];
      skinny_weights(rW, 16, sWrow, k0 >> 7, nk, I, wave, r16, g, wf, sw);
      __builtin_amdgcn_sched_barrier(0);
      if (r0 || k0) lds_barrier();  // the codes or sums before have been read
      for (int r = wave; r < rows; r += 4) {
        if (r != wave) load_h(r);
        const float v[8] = {__int_as_float(ha.x), __int_as_float(ha.y), __int_as_float(ha.z), __int_as_float(ha.w),
                            __int_as_float(hb.x), __int_as_float(hb.y), __int_as_float(hb.z), __int_as_float(hb.w)};
        uint32_t am = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        const float s = block_scale_f32(row16_max(am)), inv = 1.0f / s;
        *reinterpret_cast<uint2*>(smem + (step * 16 + r) * 128 + ((piece ^ (r & 7)) << 4) + (lane & 1) * 8) =
            make_uint2(codes4(v, s, inv), codes4(v + 4, s, inv));
        if ((lane & 15) == 0) xs[step * 16 + r] = s;
      }
      lds_barrier();
      // rows from `rows` on are whatever the LDS held: their columns are not stored
      if ((k0 >> 7) + wave < nk) {
        const v8i xf = lds_frag(smem + wave * 16 * 128, r16, g);
        const float s = xs[wave * 16 + r16] * sw[0][0];
#pragma unroll
        for (int i = 0; i < NT; ++i) scaled_mfma(acc[i], wf[0][i], xf, s);
      }
    }
    lds_barrier();
    v4f* const red = reinterpret_cast<v4f*>(smem);
#pragma unroll
    for (int i = 0; i < NT; ++i) red[(wave * NT + i) * 64 + lane] = acc[i];
    lds_barrier();
    const int col = n0 + wave * 16 + 4 * g;
    if (r16 < rows && col < H) {
      const int slot = list[r0 + r16];
      const float w = p.tw[slot];
      const v4f a = add_waves<NT>(red, wave, lane);
      *reinterpret_cast<float4*>(p.y + (int64_t)slot * H + col) = make_float4(a[0] * w, a[1] * w, a[2] * w, a[3] * w);
    }
  }
}

// The smallest steps: the down projection with the sum over a token's copies,
// one launch instead of two. A workgroup has 16 columns and quantises all
// slots' h into LDS; its 16 waves take the steps of 128 of the picked experts
// in turn, the step's columns being the tokens.
constexpr int kSmallSlots = 16, kSmallCodes = 16384;  // most slots, codes of h

__global__ __launch_bounds__(1024) void block_small_down(const BlockFewArgs p, uint16_t* __restrict__ out) {
  constexpr int U = 4, kWaves = 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // codes [I/128][slots][128]; then the waves' sums
  __shared__ float hs[kSmallCodes / 128];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = p.H, I = p.I, nk = I >> 7, n = p.n, n0 = blockIdx.x * 16;
  const int r16 = lane & 15, g = lane >> 4;
  const int nb = (H + 127) >> 7;
  // h's loads first, then the ids and the first steps' weights
  const int per = I >> 3, chunks = n * per;  // pieces of 8 values
  float4 ha, hb;
  auto load_h = [&](int c) {
    const float* src = p.h + (int64_t)c * 8;
    ha = *reinterpret_cast<const float4*>(src);
    hb = *reinterpret_cast<const float4*>(src + 4);
  };
  if (tid < chunks) load_h(tid);
  int id = -1;
  float tw = 0.f;
  if (lane < n) {
    id = p.ids[lane];
    tw = p.tw[lane];
    if (id >= p.E) id = -1;
  }
  v8i wf[U];
  auto load_w = [&](int u0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = u0 + kWaves * u, slot = unit / nk, kb = unit - slot * nk;
      const int e = slot < n ? __builtin_amdgcn_readlane(id, slot) : -1;
      // an expert's first slot works for all of its tokens
      const bool mine = e >= 0 && (__ballot(id == e) & ((1ull << slot) - 1)) == 0;
      const auto rW = make_rsrc(p.w2 + ((int64_t)(mine ? e : 0) * H + n0) * I, mine ? (int64_t)(H - n0) * I : 0);
      const uint32_t at = (uint32_t)r16 * (uint32_t)I + (uint32_t)(kb << 7) + 16u * (uint32_t)g;
      const v4i lo = buffer_load16(rW, at), hi = buffer_load16(rW, at + 64u);
      wf[u] = v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    }
  };
  const int units = n * nk;
  load_w(wave);
  __builtin_amdgcn_sched_barrier(0);
  for (int c = tid; c < chunks; c += 1024) {
    if (c != tid) load_h(c);
    const float v[8] = {ha.x, ha.y, ha.z, ha.w, hb.x, hb.y, hb.z, hb.w};
    uint32_t am = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const float s = block_scale_f32(row16_max(am)), inv = 1.0f / s;
    const int slot = c / per, col = c - slot * per, kb = col >> 4, piece = (col & 15) >> 1;
    *reinterpret_cast<uint2*>(smem + (kb * n + slot) * 128 + ((piece ^ (slot & 7)) << 4) + (col & 1) * 8) =
        make_uint2(codes4(v, s, inv), codes4(v + 4, s, inv));
    if ((col & 15) == 0) hs[kb * n + slot] = s;
  }
  lds_barrier();
  v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
  for (int u0 = wave; u0 < units; u0 += kWaves * U) {
    if (u0 != wave) load_w(u0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = u0 + kWaves * u, slot = unit / nk, kb = unit - slot * nk;
      if (slot >= n) break;
      const int e = __builtin_amdgcn_readlane(id, slot);
      const uint64_t all = __ballot(id == e);
      if (e < 0 || (all & ((1ull << slot) - 1)) != 0) continue;
      const float sw = ((ScalarPtr)(p.s2 + ((int64_t)e * nb + (n0 >> 7)) * nk))[kb];
      // this lane's token: its copies for the expert, one row of h, their weights added
      const uint64_t own = r16 < p.T ? (all >> (r16 * p.topk)) & (~0ull >> (64 - p.topk)) : 0ull;
      const int row = own ? r16 * p.topk + __builtin_ctzll(own) : 0;
      float w = 0.f;
      for (int j = 0; j < p.topk; ++j) {
        const float x = __uint_as_float(__builtin_amdgcn_ds_bpermute(((r16 * p.topk + j) & 63) << 2, (int)__float_as_uint(tw)));
        w += (own >> j) & 1 ? x : 0.f;
      }
      const uint8_t* at = smem + (kb * n + row) * 128;
      const v4i lo = *reinterpret_cast<const v4i*>(at + ((g ^ (row & 7)) << 4));
      const v4i hi = *reinterpret_cast<const v4i*>(at + (((g + 4) ^ (row & 7)) << 4));
      const v4f d = mfma_16x16x128_e4m3(wf[u], v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}, v4f{0.f, 0.f, 0.f, 0.f});
      const float s = hs[kb * n + row] * sw * w;
      // a token without this expert keeps its sum, whatever the expert's weights hold
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = own ? __builtin_fmaf(d[r], s, acc[r]) : acc[r];
    }
  }
  lds_barrier();
  v4f* const red = reinterpret_cast<v4f*>(smem);
  red[wave * 64 + lane] = acc;
  lds_barrier();
  if (wave != 0) return;
  v4f sum = red[lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += red[w * 64 + lane];
  if (r16 < p.T)
    *reinterpret_cast<uint2*>(out + (int64_t)r16 * H + n0 + 4 * g) =
        make_uint2(bf16x2_rne(sum[0], sum[1]), bf16x2_rne(sum[2], sum[3]));
}

// ---- tiled products ------------------------------------------------------------

enum { kDense = 0, kGateUp = 1, kDown = 2 };

struct BlockArgs {
  const uint8_t* A;        // codes: dense [M, K]; gate/up tokens [T, K]; down sorted h rows [T topk, K]
  const float* sA;         // their scales [blocks of K, a_rows]
  int64_t a_rows;
  const uint8_t* B;        // [E, N, K] codes (dense: E = 1)
  const float* sB;         // [E, blocks of N, blocks of K]
  const int4* tiles;       // grouped: {their number}, then each one's expert, first sorted row and rows
  const int32_t* tok;      // gate/up: token of a sorted row
  const float* tw;         // down: router weight of a sorted row
  uint16_t* y;             // dense [M, N]
  uint8_t* hq;             // gate/up: codes of h [T topk, N / 2]
  float* hs;               // gate/up: their scales [N / 256, T topk]
  uint16_t* y16;           // down: weighted rows in sorted order [T topk, N], float16 times ys
  float* ys;               // down: [blocks of N, T topk]
  int topk, N, K, tiles_m, tiles_n;  // topk: gate/up
};

template <int BM, int BN, int WGM, int WGN, int MODE, int NS>
struct BlockTile {
  static constexpr int kThreads = 64 * WGM * WGN;
  static constexpr int WM = BM / WGM, WN = BN / WGN;  // a wave's part
  static constexpr int SM = WM / 16, SN = WN / 16;
  static constexpr int kRows = BM + BN;
  static constexpr int kCodes = kRows * 128;                              // bytes of a stage's codes
  static constexpr int kStage = kCodes + (BM * 4 + 1023) / 1024 * 1024;   // and its row scales
  static constexpr int kRowsPerPass = kThreads / 8;
  static constexpr int kLoadsB = BN / kRowsPerPass, kLoadsA = BM / kRowsPerPass;
  static constexpr int kEpiStride = BN * 2 + 16;  // dense, down: staged 16-bit row
  static constexpr int kHStride = 128 + 16;       // gate/up: staged row of h codes
  static constexpr int kEpi = MODE == kGateUp ? BM * kHStride + WGN * BM * 4 : BM * kEpiStride;
  static constexpr int kLds = NS * kStage > kEpi ? NS * kStage : kEpi;
  static_assert(BN % kRowsPerPass == 0 && BM % kRowsPerPass == 0 && kRowsPerPass % 8 == 0, "stages split evenly");
  static_assert(WM % 16 == 0 && WN % 16 == 0 && BM <= kThreads, "wave tiles");
  static_assert(MODE != kGateUp || (BN == 256 && SN % 2 == 0), "a gate/up tile is one block of 128 h columns");
};

// acc[i][j] += (w_i . x_j) * (sx[j] * sw[i]): kAhead MFMAs are under way before
// the first result is added, then every MFMA is followed by the four FMAs of an
// earlier one, which run while the matrix unit works.
template <int SN, int SM, int NB>
__device__ inline void scaled_mfmas(v4f (&acc)[SN][SM], const v8i (&wf)[SN], const v8i (&xf)[SM], const float (&sx)[SM],
                                    const float (&sw)[NB]) {
  constexpr int kAhead = 2, kN = SN * SM;
#pragma unroll
  for (int i = 0; i < SN; ++i)
#pragma unroll
    for (int j = 0; j < SM; ++j) {
      const v4f d = mfma_16x16x128_e4m3(wf[i], xf[j], v4f{0.f, 0.f, 0.f, 0.f});
      const float s = sx[j] * sw[i % NB];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[r], s, acc[i][j][r]);
    }
  // the order of issue: groups of MFMAs (mask 8) and vector instructions (2)
  __builtin_amdgcn_sched_group_barrier(8, kAhead, 0);
#pragma unroll
  for (int n = kAhead; n < kN; ++n) {
    __builtin_amdgcn_sched_group_barrier(8, 1, 0);
    __builtin_amdgcn_sched_group_barrier(2, 5, 0);
  }
  __builtin_amdgcn_sched_group_barrier(2, 5 * kAhead, 0);
  // every sum is there by here: left free, the compiler holds all results of a step in registers and adds them later
#pragma unroll
  for (int i = 0; i < SN; ++i)
#pragma unroll
    for (int j = 0; j < SM; ++j) asm volatile("" : "+v"(acc[i][j]));
}

// The same on BF16 matrix cores: the codes are widened, the sums near float32.
template <int SN, int SM, int NB>
__device__ inline void wide_mfmas(v4f (&acc)[SN][SM], const v8i (&wf)[SN], const v8i (&xf)[SM], const float (&sx)[SM],
                                  const float (&sw)[NB]) {
  v4i x[SM][4];
#pragma unroll
  for (int j = 0; j < SM; ++j) widen32(xf[j], x[j]);
#pragma unroll
  for (int i = 0; i < SN; ++i) {
    v4i w[4];
    widen32(wf[i], w);
    v4f d[SM];
#pragma unroll
    for (int j = 0; j < SM; ++j) d[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < SM; ++j) d[j] = mfma_16x16x32_bf16(w[c], x[j][c], d[j]);
#pragma unroll
    for (int j = 0; j < SM; ++j) {
      const float s = sx[j] * sw[i % NB];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[j][r], s, acc[i][j][r]);
    }
  }
#pragma unroll
  for (int i = 0; i < SN; ++i)
#pragma unroll
    for (int j = 0; j < SM; ++j) asm volatile("" : "+v"(acc[i][j]));
}

// Fragment of the 16 staged rows from `row0` on, lds_frag's chunks c and c + 4
// of this lane's row: lane_off is the lane's own offset (its row lane % 16 and
// chunk), so that every fragment of a stage is one address and a constant.
__device__ inline int frag_lane_off(int r16, int g) { return r16 * 128 + ((g ^ (r16 & 7)) << 4); }
__device__ inline v8i frag_at(const uint8_t* st, int lane_off, int row0) {
  const v4i lo = *reinterpret_cast<const v4i*>(st + lane_off + row0 * 128);
  const v4i hi = *reinterpret_cast<const v4i*>(st + (lane_off ^ 64) + row0 * 128);
  return v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}

// One 128-deep K step is one block of scales. Stages are double-buffered in
// LDS: the codes by direct 16-byte loads (rows of 128 bytes, 16-byte pieces
// swizzled), the step's row scales by direct 4-byte loads behind them; the
// weight scale is one value a wave (a wave's columns lie in one block where
// their number divides 128), read by scalar loads.
//  kDense   y = bf16(a . w^T)
//  kGateUp  rows gathered through the sorted order; stage rows alternate 16
//           gate and the 16 matching up rows, so that g and u of an element meet
//           in one lane. A tile's 128 columns of h are one block: its row maxima
//           meet in LDS, and h leaves as codes and scales.
//  kDown    y = router weight * (h . w2^T), a row per sorted row, written in 16
//           bits: float16 times a power of two for each 128 columns of a row, which
//           rounds a copy by at most 2^-11 of its value where the sum over the copies
//           is rounded to BF16 by up to 2^-8. In float32 these rows, written here and
//           read once by the combine, were 536 MB of a pass of 4096 tokens, top-8, H
//           2048. The power comes from a bound on the row's sums, |h| <= 448 hs and
//           |w| <= 448 sw, so that no value can overflow and no maximum has to be
//           found: what is 2^-27 of the bound and more keeps all 11 bits.
// NS: stages. With one, half the LDS lets more workgroups run on a CU, and they
// fill each other's waits: every tile of the larger sizes has one.
template <int BM, int BN, int WGM, int WGN, int MODE, int OCC, int NS, bool WIDE>
__global__ __launch_bounds__(64 * WGM * WGN) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void block_tiled(const BlockArgs p) {
  using C = BlockTile<BM, BN, WGM, WGN, MODE, NS>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::kLds + (MODE == kDown ? BM * 4 : 0)];
  float* const row_w = reinterpret_cast<float*>(smem + C::kLds);  // down: router weight of a tile row
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = p.N, K = p.K;
  int row0, rows, nt, e = 0;
  if constexpr (MODE == kDense) {
    int tm;
    map_tile<4>(blockIdx.x, p.tiles_m, p.tiles_n, tm, nt);
    row0 = tm * BM;
    rows = min(BM, (int)p.a_rows - row0);
  } else {
    // the tiles there are, an eighth of them, consecutive, on each XCD
    typedef const __attribute__((address_space(4))) int* ScalarInt;
    const ScalarInt table = (ScalarInt)p.tiles;
    const int64_t total = (int64_t)table[0] * p.tiles_n;
    const int xcd = blockIdx.x & 7;
    const int t = (int)(total * xcd / 8) + (int)(blockIdx.x >> 3);
    if (t >= (int)(total * (xcd + 1) / 8)) return;
    const int mt = t / p.tiles_n;
    nt = t - mt * p.tiles_n;
    e = table[4 * mt + 4];
    row0 = table[4 * mt + 5];
    rows = table[4 * mt + 6];
  }
  const int n0 = nt * BN;
  const int nb = (N + 127) >> 7, nk = (K + 127) >> 7;
  const auto rB = MODE == kGateUp ? make_rsrc(p.B + (int64_t)e * N * K, (int64_t)N * K)
                                  : make_rsrc(p.B + ((int64_t)e * N + n0) * K, (int64_t)(N - n0) * K);
  const auto rA = MODE == kGateUp ? make_rsrc(p.A, p.a_rows * K) : make_rsrc(p.A + (int64_t)row0 * K, (int64_t)rows * K);

  const int lchunk = ((tid & 7) ^ ((tid >> 3) & 7)) << 4;
  const int lrow = tid >> 3;
  // Byte offset of a thread's i-th 16-byte piece at K = 0. Rows past the end lie
  // outside the buffer and read as zeros. A gathered row's offset is kept in a
  // register, the others follow from the first.
  const uint32_t lbase = (uint32_t)lrow * (uint32_t)K + (uint32_t)lchunk;
  uint32_t arow[MODE == kGateUp ? C::kLoadsA : 1];
  uint32_t soff = kOutOfRange;  // of this lane's row scale of a step: lane l of the first waves loads row 64 w + l
  if constexpr (MODE == kGateUp) {
    const auto rT = make_rsrc(p.tok + row0, (int64_t)rows * 4);  // tokens of the tile's rows
    uint32_t tok[C::kLoadsA + 1];
#pragma unroll
    for (int j = 0; j < C::kLoadsA; ++j)
      tok[j] = __builtin_amdgcn_raw_buffer_load_b32(rT, (uint32_t)(lrow + C::kRowsPerPass * j) * 4u, 0, 0);
    tok[C::kLoadsA] = __builtin_amdgcn_raw_buffer_load_b32(rT, (uint32_t)tid * 4u, 0, 0);
#pragma unroll
    for (int j = 0; j < C::kLoadsA; ++j)
      arow[j] = lrow + C::kRowsPerPass * j < rows ? tok[j] * (uint32_t)K + (uint32_t)lchunk : kOutOfRange;
    if (tid < rows) soff = tok[C::kLoadsA] * 4u;
  } else if (tid < rows) {
    soff = (uint32_t)tid * 4u;
  }
  auto boff = [&](int i) {
    if constexpr (MODE == kGateUp) {  // 16-row piece b: even = gate rows, odd = the matching up rows
      const int r = lrow + C::kRowsPerPass * i;
      const int wr = ((r >> 4) & 1 ? N / 2 : 0) + (n0 >> 1) + (r >> 5) * 16 + (r & 15);
      return (uint32_t)wr * (uint32_t)K + (uint32_t)lchunk;
    } else {
      return lbase + (uint32_t)(C::kRowsPerPass * i) * (uint32_t)K;
    }
  };
  auto aoff = [&](int j) {
    if constexpr (MODE == kGateUp)
      return arow[j];
    else
      return lbase + (uint32_t)(C::kRowsPerPass * j) * (uint32_t)K;
  };
  auto issue = [&](int stage, int kt) {
    uint8_t* base = smem + stage * C::kStage;
    const int k0 = kt << 7;
    const bool kin = k0 + lchunk < K;
#pragma unroll
    for (int i = 0; i < C::kLoadsB + C::kLoadsA; ++i) {
      const int s0 = wave * 64 + C::kThreads * i;
      if (i < C::kLoadsB) {
        buffer_load16_lds(rB, base + s0 * 16, kin ? boff(i) + (uint32_t)k0 : kOutOfRange);
      } else {
        const uint32_t a = aoff(i - C::kLoadsB);
        buffer_load16_lds(rA, base + s0 * 16, kin && a != kOutOfRange ? a + (uint32_t)k0 : kOutOfRange);
      }
    }
    if (wave < (BM + 63) / 64) {
      const float* s = p.sA + (int64_t)kt * p.a_rows + (MODE == kGateUp ? 0 : row0);
      const auto rS = make_rsrc(s, (MODE == kGateUp ? p.a_rows : (int64_t)rows) * 4);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rS, (lds_void*)(base + C::kCodes + wave * 256), 4, soff, 0, 0, 0);
    }
  };

  const int wm = wave % WGM, wn = wave / WGM;
  const int r16 = lane & 15, g = lane >> 4;
  const int lane_off = frag_lane_off(r16, g);
  const int a_base = (BN + wm * C::WM) * 128, b_base = wn * C::WN * 128, s_base = C::kCodes + (wm * C::WM + r16) * 4;
  // weight blocks of the wave's column tiles (gate/up: even tiles are gate columns, odd ones up columns)
  const float* sBe = p.sB + (int64_t)e * nb * nk;
  constexpr int kBlocks = MODE == kGateUp ? 2 : 1;
  static_assert(MODE == kGateUp || 128 % C::WN == 0, "a wave's columns lie in one block");
  ScalarPtr sBp[kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const int b = MODE == kGateUp ? nt + i * (nb >> 1) : min((n0 + wn * C::WN) >> 7, nb - 1);
    sBp[i] = (ScalarPtr)(sBe + (int64_t)b * nk);
  }
  v4f acc[C::SN][C::SM];
  float size[C::SM];  // down: sum over the steps of the products of the scales
#pragma unroll
  for (int j = 0; j < C::SM; ++j) size[j] = 0.f;
#pragma unroll
  for (int i = 0; i < C::SN; ++i)
#pragma unroll
    for (int j = 0; j < C::SM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  issue(0, 0);
  if constexpr (MODE == kDown) {
    // the rows' weights, used after the K loop, whose barriers order them
    if (tid < BM) row_w[tid] = tid < rows ? p.tw[row0 + tid] : 0.f;
  }
  for (int kt = 0; kt < nk; ++kt) {
    float sw[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) sw[i] = sBp[i][kt];
    wait_vmem_all();
    lds_barrier();
    if (NS == 2 && kt + 1 < nk) issue((kt + 1) & 1, kt + 1);
    const uint8_t* st = smem + (NS == 2 ? (kt & 1) * C::kStage : 0);
    v8i xf[C::SM], wf[C::SN];
    float sx[C::SM];
#pragma unroll
    for (int j = 0; j < C::SM; ++j) {
      xf[j] = frag_at(st + a_base, lane_off, j * 16);
      sx[j] = *reinterpret_cast<const float*>(st + s_base + j * 64);
    }
#pragma unroll
    for (int i = 0; i < C::SN; ++i) wf[i] = frag_at(st + b_base, lane_off, i * 16);
    if (NS == 1) {
      // one stage: once every wave has its fragments the next step's loads go out, and overlap the MFMAs
      lds_barrier();
      if (kt + 1 < nk) issue(0, kt + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (MODE == kDown) {
#pragma unroll
      for (int j = 0; j < C::SM; ++j) size[j] = __builtin_fmaf(fabsf(sx[j]), fabsf(sw[0]), size[j]);
    }
    if constexpr (WIDE)
      wide_mfmas<C::SN, C::SM, kBlocks>(acc, wf, xf, sx, sw);
    else
      scaled_mfmas<C::SN, C::SM, kBlocks>(acc, wf, xf, sx, sw);
    __builtin_amdgcn_sched_barrier(0);
  }
  __syncthreads();

  // acc[i][j][r]: tile row wm WM + 16 j + lane % 16, stage row wn WN + 16 i + 4 (lane / 16) + r
  if constexpr (MODE == kDense) {
#pragma unroll
    for (int i = 0; i < C::SN; ++i) {
      const int nl = wn * C::WN + i * 16 + 4 * g;
#pragma unroll
      for (int j = 0; j < C::SM; ++j) {
        const int ml = wm * C::WM + j * 16 + r16;
        const v4f a = acc[i][j];
        *reinterpret_cast<uint2*>(smem + ml * C::kEpiStride + nl * 2) =
            make_uint2(bf16x2_rne(a[0], a[1]), bf16x2_rne(a[2], a[3]));
      }
    }
    __syncthreads();
    constexpr int kRowChunks = BN / 8;
    for (int c = tid; c < BM * kRowChunks; c += C::kThreads) {
      const int row = c / kRowChunks, col = (c % kRowChunks) * 8;
      if (row < rows && n0 + col < N)
        store16_nt(p.y + (int64_t)(row0 + row) * N + n0 + col,
                   *reinterpret_cast<const uint4*>(smem + row * C::kEpiStride + col * 2));
    }
  }
  if constexpr (MODE == kGateUp) {
    // maxima of |h| on the bits, where infinity and NaN come last and reach the
    // scale, and through it the token
    uint32_t* const rmax = reinterpret_cast<uint32_t*>(smem + BM * C::kHStride);  // [WGN][BM]
    uint32_t am[C::SM];
#pragma unroll
    for (int j = 0; j < C::SM; ++j) {
      am[j] = 0u;
#pragma unroll
      for (int i = 0; i < C::SN; i += 2)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float h = silu_f32(acc[i][j][r]) * acc[i + 1][j][r];
          acc[i][j][r] = h;
          am[j] = max(am[j], __float_as_uint(h) & 0x7FFFFFFFu);
        }
      am[j] = max(am[j], (uint32_t)__shfl_xor((int)am[j], 16, 64));
      am[j] = max(am[j], (uint32_t)__shfl_xor((int)am[j], 32, 64));
      if (g == 0) rmax[wn * BM + wm * C::WM + j * 16 + r16] = am[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < C::SM; ++j) {
      const int ml = wm * C::WM + j * 16 + r16;
      uint32_t a = 0u;
#pragma unroll
      for (int w = 0; w < WGN; ++w) a = max(a, rmax[w * BM + ml]);
      const float s = block_scale_f32(a), inv = 1.0f / s;
      if (wn == 0 && g == 0 && ml < rows) p.hs[(int64_t)nt * (p.a_rows * p.topk) + row0 + ml] = s;
#pragma unroll
      for (int i = 0; i < C::SN; i += 2) {
        const float h[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        const int hc = ((wn * C::WN + i * 16) >> 1) + 4 * g;
        *reinterpret_cast<uint32_t*>(smem + ml * C::kHStride + hc) = codes4(h, s, inv);
      }
    }
    __syncthreads();
    for (int c = tid; c < BM * 8; c += C::kThreads) {
      const int row = c >> 3, col = (c & 7) << 4;
      if (row < rows)
        *reinterpret_cast<uint4*>(p.hq + (int64_t)(row0 + row) * (N / 2) + (n0 >> 1) + col) =
            *reinterpret_cast<const uint4*>(smem + row * C::kHStride + col);
    }
  }
  if constexpr (MODE == kDown) {
#pragma unroll
    for (int j = 0; j < C::SM; ++j) {
      const int ml = wm * C::WM + j * 16 + r16;
      const float w = row_w[ml];
      // size < 2^(bs - 126), 2 * 128 * 448^2 < 2^26 with a factor of two for the roundings of the sums, and
      // a float32 is below 2^128: |a| < 2^ea. |w| < 2^(bw - 126): the row's values stay below 2^e.
      const int bs = (int)(__float_as_uint(size[j]) >> 23) & 0xFF, bw = (int)(__float_as_uint(w) >> 23) & 0xFF;
      const int ea = min(bs - 126 + 26, 128), e = ea + bw - 126;
      // 2^(15 - e) and back, which neither take w out of range: w 2^up is about 2^(14 - ea), a normal float32,
      // also where the sum of the scales is infinite and the values are not
      const int up = max(-113, min(15 - e, min(126, 253 - bw)));
      const float to = __uint_as_float((uint32_t)(127 + up) << 23), from = __uint_as_float((uint32_t)(127 - up) << 23);
      const int col = n0 + wn * C::WN;
      if (g == 0 && (col & 127) == 0 && ml < rows && col < N) p.ys[(int64_t)(col >> 7) * p.a_rows + row0 + ml] = from;
      const float f = w * to;
#pragma unroll
      for (int i = 0; i < C::SN; ++i) {
        const int nl = wn * C::WN + i * 16 + 4 * g;
        const v4f a = acc[i][j];
        typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
        const half2_t lo = {(_Float16)(a[0] * f), (_Float16)(a[1] * f)}, hi = {(_Float16)(a[2] * f), (_Float16)(a[3] * f)};
        *reinterpret_cast<uint2*>(smem + ml * C::kEpiStride + nl * 2) =
            make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
      }
    }
    __syncthreads();
    constexpr int kRowChunks = BN / 8;
    for (int c = tid; c < BM * kRowChunks; c += C::kThreads) {
      const int row = c / kRowChunks, col = (c % kRowChunks) * 8;
      if (row < rows && n0 + col < N) {
        const uint4 v = *reinterpret_cast<const uint4*>(smem + row * C::kEpiStride + col * 2);
        uint4* const to = reinterpret_cast<uint4*>(p.y16 + (int64_t)(row0 + row) * N + n0 + col);
        // Rows that the caches may keep for the combine, unless a group's rows outweigh its
        // weights (tiles of 128 rows) and would drive these out (whole passes in a graph, kept
        // and streamed. Tiles of 64 rows: top-8 of 64, H 2048, 2048 tokens 130 and 136 us; top-4
        // of 192, H 1024, 4096 tokens 110 and 113. Tiles of 128 rows: top-8 of 64, 4096 tokens
        // 215 and 217, 8192 tokens 377 and 372).
        if constexpr (BM >= 128)
          store16_nt(to, v);
        else
          *to = v;
      }
    }
  }
}

// out[t] = bf16(sum over the token's valid slots, in order, of their rows of y16
// times their scales), 8 columns a thread, 16 threads a block; with q also the
// next pass's quantisation, as quantize_blocks does it. The rows are loaded
// before any is added; a dropped slot's is not used.
__global__ __launch_bounds__(256) void combine_half(const uint16_t* __restrict__ y, const float* __restrict__ ys,
                                                    const int32_t* __restrict__ ids, const int32_t* __restrict__ slot_row,
                                                    int64_t T, int topk, int E, int H, uint16_t* __restrict__ out,
                                                    uint8_t* __restrict__ q, float* __restrict__ scale) {
  const int kb = (H + 127) >> 7;
  const int64_t b = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t t = b / kb;
  if (t >= T) return;
  const int blk = (int)(b - t * kb), c = blk * 128 + 8 * (threadIdx.x & 15), at = c < H ? c : 0;
  const int64_t cap = T * topk;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  constexpr int kBatch = 8;
  for (int j0 = 0; j0 < topk; j0 += kBatch) {
    v4i v[kBatch];
    float f[kBatch];
    bool ok[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t slot = t * topk + (j0 + i < topk ? j0 + i : 0);
      const int id = ids[slot];
      ok[i] = j0 + i < topk && id >= 0 && id < E;
      const int64_t row = ok[i] ? slot_row[slot] : 0;
      v[i] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(y + row * H + at));
      f[i] = ys[(int64_t)blk * cap + row];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (!ok[i]) continue;
      typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
      const half8_t h = __builtin_bit_cast(half8_t, v[i]);
#pragma unroll
      for (int r = 0; r < 8; ++r) sum[r] = __builtin_fmaf((float)h[r], f[i], sum[r]);
    }
  }
  uint4 o = to_bf16x8(make_float4(sum[0], sum[1], sum[2], sum[3]), make_float4(sum[4], sum[5], sum[6], sum[7]));
  if (c < H)
    *reinterpret_cast<uint4*>(out + t * H + c) = o;
  else
    o = make_uint4(0u, 0u, 0u, 0u);
  if (q == nullptr) return;
  const float s = row_scale(row16_max(absmax8(o)));
  if (c < H) *reinterpret_cast<uint2*>(q + t * H + c) = quant8(o, s, 1.0f / s);
  if ((threadIdx.x & 15) == 0) scale[(int64_t)blk * T + t] = s;
}

// The combine of float32 rows (few tokens) with the next pass's quantisation by
// blocks: 16 threads sum a block of 128 columns of a token (in the order of
// combine_slots) and quantise it as quantize_blocks does.
__global__ __launch_bounds__(256) void combine_block_quant(const float* __restrict__ y, const int32_t* __restrict__ ids,
                                                           int64_t T, int topk, int E, int H, uint16_t* __restrict__ out,
                                                           uint8_t* __restrict__ q, float* __restrict__ scale) {
  const int kb = (H + 127) >> 7;
  const int64_t b = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t t = b / kb;
  if (t >= T) return;
  const int blk = (int)(b - t * kb), c = blk * 128 + 8 * (threadIdx.x & 15);
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (c < H) {
    float4 lo, hi;
    sum_slots8(y, ids, nullptr, t, topk, E, H, c, lo, hi);
    v = to_bf16x8(lo, hi);
    *reinterpret_cast<uint4*>(out + t * H + c) = v;
  }
  const float s = row_scale(row16_max(absmax8(v)));
  if (c < H) *reinterpret_cast<uint2*>(q + t * H + c) = quant8(v, s, 1.0f / s);
  if ((threadIdx.x & 15) == 0) scale[(int64_t)blk * T + t] = s;
}

// ---- the sorted order of the routed slots and its tiles

struct RouteArgs {
  const int32_t* ids;
  const float* tw;
  int32_t* tok;       // token of a sorted row
  float* w;           // its router weight
  int32_t* slot_row;  // slot -> sorted row
  int4* tiles[2];     // of bm[0] and bm[1] rows (one table where these are equal), see BlockArgs
  int n, E, topk, bm[2];
};

// Exclusive prefix sums of value(e) over the experts into out, by one wave; their total.
template <class F>
__device__ inline int expert_prefix(int E, int lane, F value, int* out) {
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane, v = e < E ? value(e) : 0;
    int incl = v;
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x111, 0xF, 0xF, false);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x112, 0xF, 0xF, false);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x114, 0xF, 0xF, false);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x118, 0xF, 0xF, false);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x142, 0xA, 0xF, false);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x143, 0xC, 0xF, false);
    if (e < E) out[e] = before + incl - v;
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return before;
}

// Tile i of a table, whose experts' first tiles are first[e], of `total`: its expert is
// the last whose first tile is not behind it.
__device__ inline void write_tile(int4* tiles, int bm, int i, int total, int E, const int* first, const int* start,
                                  const int* count) {
  if (i == 0) tiles[0] = make_int4(total, 0, 0, 0);
  if (i >= total) return;
  int e = 0;
  for (int half = 512; half > 0; half >>= 1)
    if (e + half < E && first[e + half] <= i) e += half;
  const int r = (i - first[e]) * bm;
  tiles[i + 1] = make_int4(e, start[e] + r, min(bm, count[e] - r), 0);
}

// The slots of 1024 consecutive ids a workgroup, grouped by expert in a stable
// order (as route_count and route_scatter of the other expert formats): every
// workgroup counts all ids for itself, those before its own and the others, so
// that one launch does for up to kRouteOneSlots slots. A counter has kRouteCopies
// copies in LDS, for the lanes that meet at one expert. There are no more tiles
// than slots: each thread writes at most one of each table.
constexpr int kRouteThreads = 1024, kRouteWaves = 16, kRouteCopies = 8;

__global__ __launch_bounds__(kRouteThreads) void block_route(const RouteArgs p) {
  extern __shared__ int route_lds[];
  const int n = p.n, E = p.E;
  int* const before = route_lds;          // [E] ids of the chunks before, then the expert's next row
  int* const count = route_lds + E;       // [E]
  int* const start = route_lds + 2 * E;   // [E]
  int* const first = route_lds + 3 * E;   // [2][E]
  int* const hist = route_lds + 5 * E;    // [2][E][kRouteCopies], then [waves][E]
  __shared__ int totals[2];
  static_assert(kRouteWaves == 2 * kRouteCopies, "both take the same room");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lo = blockIdx.x * kRouteThreads, s = lo + tid;
  const auto rI = make_rsrc(p.ids, (int64_t)n * 4);
  const int own = (int)__builtin_amdgcn_raw_buffer_load_b32(rI, (uint32_t)s * 4u, 0, 0);
  const float own_w = s < n ? p.tw[s] : 0.f;
  for (int e = tid; e < 2 * E * kRouteCopies; e += kRouteThreads) hist[e] = 0;
  __syncthreads();
  constexpr int kBatch = 8;
  for (int i0 = 0; i0 < n; i0 += kBatch * 4 * kRouteThreads) {
    v4i v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) v[b] = buffer_load16(rI, (uint32_t)(i0 + 4 * (b * kRouteThreads + tid)) * 4u);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + 4 * (b * kRouteThreads + tid);
      int* const h = hist + (i < lo ? 0 : E * kRouteCopies) + (lane & (kRouteCopies - 1));
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (i + r < n && v[b][r] >= 0 && v[b][r] < E) atomicAdd(h + v[b][r] * kRouteCopies, 1);
    }
  }
  __syncthreads();
  for (int e = tid; e < E; e += kRouteThreads) {
    int b = 0, a = 0;
#pragma unroll
    for (int c = 0; c < kRouteCopies; ++c) {
      b += hist[e * kRouteCopies + c];
      a += hist[(E + e) * kRouteCopies + c];
    }
    before[e] = b;
    count[e] = a + b;
  }
  __syncthreads();
  for (int e = tid; e < kRouteWaves * E; e += kRouteThreads) hist[e] = 0;
  if (wave == 0) expert_prefix(E, lane, [&](int e) { return count[e]; }, start);
  if (wave == 1 || wave == 2) {
    const int bm = p.bm[wave - 1];
    const int t = expert_prefix(E, lane, [&](int e) { return (count[e] + bm - 1) / bm; }, first + (wave - 1) * E);
    if (lane == 0) totals[wave - 1] = t;
  }
  __syncthreads();
  // the lanes of the wave that share this lane's expert (dropped ids share E)
  const int key = s < n && own >= 0 && own < E ? own : E;
  uint64_t peers = ~0ull;
  for (int b = 0; (E >> b) != 0; ++b) {
    const bool bit = (key >> b) & 1;
    const uint64_t m = __ballot(bit);
    peers &= bit ? m : ~m;
  }
  const int rank = __popcll(peers & ((1ull << lane) - 1));
  if (rank == 0 && key < E) hist[wave * E + key] = __popcll(peers);
  write_tile(p.tiles[0], p.bm[0], s, totals[0], E, first, start, count);
  if (p.tiles[1] != p.tiles[0]) write_tile(p.tiles[1], p.bm[1], s, totals[1], E, first + E, start, count);
  __syncthreads();
  for (int e = tid; e < E; e += kRouteThreads) {
    int row = start[e] + before[e];
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) {
      const int c = hist[w * E + e];
      hist[w * E + e] = row;
      row += c;
    }
  }
  __syncthreads();
  if (key < E) {
    const int row = hist[wave * E + key] + rank;
    p.tok[row] = (int)((uint32_t)s / (uint32_t)p.topk);
    p.w[row] = own_w;
    p.slot_row[s] = row;
  }
}

// What block_route writes, from the order of route_scatter.
__global__ __launch_bounds__(kRouteThreads) void block_route_rest(const RouteArgs p, const int32_t* __restrict__ offsets,
                                                                  const int32_t* __restrict__ perm) {
  __shared__ int start[1024], count[1024], first[2][1024], totals[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t i = (int64_t)blockIdx.x * kRouteThreads + tid;
  const int slot = i < p.n ? perm[i] : -1;
  if (tid < p.E) {
    start[tid] = offsets[tid];
    count[tid] = offsets[tid + 1] - offsets[tid];
  }
  __syncthreads();
  if (wave < 2) {
    const int bm = p.bm[wave];
    const int t = expert_prefix(p.E, lane, [&](int e) { return (count[e] + bm - 1) / bm; }, first[wave]);
    if (lane == 0) totals[wave] = t;
  }
  if (slot >= 0) {
    p.tok[i] = (int)((uint32_t)slot / (uint32_t)p.topk);
    p.w[i] = p.tw[slot];
  }
  __syncthreads();
  if (i >= p.n) return;
  write_tile(p.tiles[0], p.bm[0], (int)i, totals[0], p.E, first[0], start, count);
  if (p.tiles[1] != p.tiles[0]) write_tile(p.tiles[1], p.bm[1], (int)i, totals[1], p.E, first[1], start, count);
}

// One launch up to here, where LDS holds the counters, and three beyond, two of them
// the other formats' (whole passes in a graph, H 256, I 128, one launch and three: 8192 slots,
// 64 experts 25.1 and 30.2 us, 65536 slots 61.8 and 68.8, of 8 experts 60.8 and 66.1, of
// 512 experts 65.6 and 76.9).
constexpr int64_t kRouteOneSlots = 65536, kRouteOneExperts = 512;

bool route_one(int64_t n, int64_t E) { return n <= kRouteOneSlots && E <= kRouteOneExperts; }

template <int BM, int BN, int WGM, int WGN, int MODE, int OCC, int NS, bool WIDE = false>
hipError_t run_tiled(BlockArgs a, int64_t tiles_m, hipStream_t stream) {
  a.tiles_n = (a.N + BN - 1) / BN;
  a.tiles_m = (int)tiles_m;
  // the same number of workgroups on each XCD, which takes an eighth of the tiles
  const int64_t grid = MODE == kDense ? tiles_m * a.tiles_n : (tiles_m * a.tiles_n + 7) / 8 * 8;
  hipLaunchKernelGGL((block_tiled<BM, BN, WGM, WGN, MODE, OCC, NS, WIDE>), dim3((unsigned)grid), dim3(64 * WGM * WGN), 0,
                     stream, a);
  return hipGetLastError();
}

template <int XR, int NT>
hipError_t run_skinny_bf16(const uint16_t* x, const uint8_t* w, const float* sw, uint16_t* y, int64_t M, int64_t N,
                           int64_t K, hipStream_t stream) {
  hipLaunchKernelGGL((block_skinny_bf16<XR, NT>), dim3((unsigned)((N + 16 * NT - 1) / (16 * NT))), dim3(256), 0, stream, x, w,
                     sw, y, (int)M, (int)N, (int)K);
  return hipGetLastError();
}

template <int SM, int SN, int U>
hipError_t run_ksplit(const uint8_t* x, const float* sa, const uint8_t* w, const float* sw, uint16_t* y, int64_t M,
                      int64_t N, int64_t K, hipStream_t stream) {
  const int tiles_m = (int)((M + 16 * SM - 1) / (16 * SM)), tiles_n = (int)((N + 16 * SN - 1) / (16 * SN));
  hipLaunchKernelGGL((block_ksplit<SM, SN, U>), dim3((unsigned)((int64_t)tiles_m * tiles_n)), dim3(256), 0, stream, x, sa, w,
                     sw, y, (int)M, (int)N, (int)K, tiles_m, tiles_n);
  return hipGetLastError();
}

template <int MT, int NT, bool XL>
hipError_t run_skinny(const uint8_t* x, const float* sa, const uint8_t* w, const float* sw, uint16_t* y, int64_t M,
                      int64_t N, int64_t K, hipStream_t stream) {
  hipLaunchKernelGGL((block_skinny<MT, NT, XL>), dim3((unsigned)((N + 16 * NT - 1) / (16 * NT))), dim3(256), 0, stream, x,
                     sa, w, sw, y, (int)M, (int)N, (int)K);
  return hipGetLastError();
}

int64_t align256(int64_t b) { return (b + 255) & ~int64_t(255); }

}  // namespace

hipError_t launch_quantize_blocks(const uint16_t* x, int64_t M, int64_t K, uint8_t* q, float* scale,
                                  hipStream_t stream) {
  const int64_t pieces = (K + 128 * kQuantBlocks - 1) / (128 * kQuantBlocks);
  hipLaunchKernelGGL(quant_row_blocks, dim3((unsigned)((M + kQuantRows - 1) / kQuantRows * pieces)), dim3(256), 0, stream, x,
                     M, K, (int)pieces, q, scale);
  return hipGetLastError();
}

hipError_t launch_quantize_weight_blocks(const uint16_t* w, int64_t E, int64_t N, int64_t K, uint8_t* q, float* scale,
                                         hipStream_t stream) {
  const int64_t nb = (N + 127) / 128, kb = (K + 127) / 128;
  hipLaunchKernelGGL(quant_weight_blocks, dim3((unsigned)(E * nb * kb)), dim3(256), 0, stream, w, N, K, (int)nb, (int)kb, q,
                     scale);
  return hipGetLastError();
}

hipError_t launch_block_gemm(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, uint16_t* y,
                             int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  // One tile of 16 weight rows a workgroup up to 4 rows, two up to 32. A second tile pays from
  // some 6,000 weight rows on, and the more rows the more, because the two share the rows'
  // fragments; fewer weight rows leave CUs idle (in a graph, one tile and two. 4 rows: 2048 x
  // 2048 3.5 and 4.3 us, 8192 x 2048 5.2 and 5.1; 12 rows: 2048 x 2048 3.8 and 4.6, 8192 x 2048
  // 5.6 and 5.3, 6144 x 4096 9.4 and 8.5, 16384 x 2048 8.6 and 7.5).
  if (M <= 4) return run_skinny<1, 1, false>(a, sa, w, sw, y, M, N, K, stream);
  if (M <= 16) return run_skinny<1, 2, false>(a, sa, w, sw, y, M, N, K, stream);
  if (M <= 32) return run_skinny<2, 2, true>(a, sa, w, sw, y, M, N, K, stream);
  BlockArgs p{};
  p.A = a;
  p.sA = sa;
  p.a_rows = M;
  p.B = w;
  p.sB = sw;
  p.y = y;
  p.N = (int)N;
  p.K = (int)K;
  // By the number of tiles (times of the product alone in a graph). One workgroup a CU, waves
  // splitting K, while 32 x 32 or 64 x 32 tiles are no more than the CUs (64 x 1024 x 2048:
  // 6.8 us in 32 x 32 against 7.9 in 64 x 64 of two stages and 7.4 of one; 301 x 1040 x 1056: 5.4
  // in 64 x 32 against 6.1 and 5.8, 128 x 128 10.0; 256 x 2048 x 2048, the last of these: 8.7
  // against 8.2 and 7.8); 64 x 64 tiles with two stages up to two a CU (512 x 2048 x 2048: 9.8; K
  // split 14.1; one stage 10.7), with one up to three (512 x 6144 x 2048: 12.5; two stages 18.4);
  // 64 x 128 up to three (1024 x 6144 x 2048: 18.4; 64 x 64 23.8; 128 x 128 18.6). Beyond,
  // rounds of the GPU: 768 tiles of 128 x 128 or 512 of 128 x 256, whose round takes about 1.3
  // to 1.45 times as long (4096 x 6144 x 2048, 2 rounds each: 54 against 68 us; 8192 x 2048 x
  // 6144, 2 against 1: 107 against 98 to 103). Two groups of waves in turns on 256 x 192 tiles,
  // as the product with row scales has them, were 3 % slower in the one and 38 % in the other.
  const auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  if (tiles(32, 32) <= 256) return run_ksplit<2, 2, 3>(a, sa, w, sw, y, M, N, K, stream);
  if (tiles(64, 32) <= 256) return run_ksplit<4, 2, 1>(a, sa, w, sw, y, M, N, K, stream);
  if (tiles(64, 64) <= 512) return run_tiled<64, 64, 2, 2, kDense, 2, 2>(p, (M + 63) / 64, stream);
  if (tiles(64, 64) <= 768) return run_tiled<64, 64, 2, 2, kDense, 4, 1>(p, (M + 63) / 64, stream);
  if (tiles(64, 128) <= 768) return run_tiled<64, 128, 2, 2, kDense, 4, 1>(p, (M + 63) / 64, stream);
  if (3 * ((tiles(128, 256) + 511) / 512) < 2 * ((tiles(128, 128) + 767) / 768))
    return run_tiled<128, 256, 2, 2, kDense, 2, 1>(p, (M + 127) / 128, stream);
  return run_tiled<128, 128, 2, 2, kDense, 3, 1>(p, (M + 127) / 128, stream);
}

// Rows that are quantised inside the product, by every workgroup for itself: up to 8, or 16 of at
// most one round of columns. In a graph, one launch and two: 12 rows of 8192 x 2048 8.9 and 8.3 us,
// where the one launch takes the host 3 to 4 us less; 12 rows of 6144 x 4096 17.0 and 11.5; 24 rows of
// 6160 x 2048 14.6 and 8.5.
static bool block_fused(int64_t M, int64_t K) { return M <= 8 || (M <= 16 && K <= kSkinnyCols); }

hipError_t launch_block_linear(const uint16_t* x, const uint8_t* w, const float* sw, uint16_t* y, int64_t M, int64_t N,
                               int64_t K, void* ws, hipStream_t stream) {
  // One tile of 16 weight rows a workgroup up to 4 rows, two beyond, which halve the quantiser's
  // work (in a graph, one tile and two. 4 rows: 2048 x 2048 4.4 and 4.5 us, 8192 x 2048 5.4 and
  // 5.2; 8 rows: 2048 x 2048 5.2 and 5.8, 8192 x 2048 7.4 and 6.4, 6144 x 4096 12.5 and 11.1; 16
  // rows: 2048 x 2048 7.4 and 8.4, 8192 x 2048 11.3 and 9.2).
  if (M == 1) return run_skinny_bf16<1, 1>(x, w, sw, y, M, N, K, stream);
  if (M <= 4) return run_skinny_bf16<4, 1>(x, w, sw, y, M, N, K, stream);
  if (M <= 8) return run_skinny_bf16<8, 2>(x, w, sw, y, M, N, K, stream);
  if (block_fused(M, K)) return run_skinny_bf16<16, 2>(x, w, sw, y, M, N, K, stream);
  uint8_t* q = static_cast<uint8_t*>(ws);
  float* s = reinterpret_cast<float*>(q + align256(M * K));
  const hipError_t e = launch_quantize_blocks(x, M, K, q, s, stream);
  if (e != hipSuccess) return e;
  return launch_block_gemm(q, s, w, sw, y, M, N, K, stream);
}

size_t block_linear_workspace_bytes(int64_t M, int64_t K) {
  if (block_fused(M, K)) return 0;
  return (size_t)(align256(M * K) + align256((K + 127) / 128 * M * 4));
}

// Whether the pass takes the kernels for groups of few rows: up to 8 on average, and few ids for
// every workgroup to look through (whole passes in a graph, these kernels and tiles. I 512: top-8 of
// 64, H 2048, 16 tokens 43 and 49 us, 32 tokens 51 and 52, 48 tokens 57 and 53; H 4096, 32 tokens 96
// and 104; top-4 of 192, H 1024, 37 tokens 43 and 44, 64 tokens 51 and 49; top-2 of 8, H 1024, 32
// tokens 17 and 28. I 1024: top-8 of 64, H 2048, 16 tokens 80 and 84, 32 tokens 90 and 88. I 1536,
// top-4 of 16, H 4096: 32 tokens 75 and 83, 48 tokens 85 and 84, 64 tokens 104 and 84).
static bool block_few(int64_t T, int64_t E, int64_t topk) { return T * topk <= kFewSlots && T * topk <= 8 * E; }

// And of those, the ones whose down projection makes the sum too, a launch less, which takes the
// host 3 us less (whole passes in a graph, two kernels and three. I 512, H 1024, top-4 of 128: 1 token
// 9.1 and 10.5 us, 2 tokens 10.3 and 11.2, 4 tokens 15.0 and 14.0; top-8 of 64, H 2048: 1 token 13.3
// and 14.5, 2 tokens 18.5 and 18.3; I 1536, top-4 of 16, H 4096: 1 token 22.4 and 24.6, 2 tokens
// 33.7 and 34.9).
static bool block_small(int64_t T, int64_t I, int64_t topk) {
  return T * topk <= kSmallSlots && T * topk * I <= kSmallCodes;
}

// small: where the sum goes, or NULL: y is left for the combine.
static hipError_t launch_block_few(const BlockFewArgs& a, uint16_t* small, hipStream_t stream) {
  const int groups = a.by_slot ? a.n : a.E;
  const dim3 gate((unsigned)(groups * (a.I / 16)));
  // Steps of 128 columns that a wave has in flight: a round of the four waves is 1024 columns with two
  // and 2048 with four, half of it empty up to 1024 (whole passes in a graph, two and four: 37 tokens, top-4 of 192, H 1024
  // 46.8 and 53.7 us, 1 token, top-4 of 128, H 1024 9.0 and 9.5, H 1536 10.1 and 9.9; 1 token, top-8
  // of 64, H 2048 13.7 and 13.3, H 4096 17.2 and 16.9; 16 tokens, H 4096 82.0 and 83.8)
  if (a.H <= 1024)
    hipLaunchKernelGGL(block_few_gate_up<2>, gate, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(block_few_gate_up<4>, gate, dim3(256), 0, stream, a);
  if (small)
    hipLaunchKernelGGL(block_small_down, dim3((unsigned)(a.H / 16)), dim3(1024), (size_t)std::max(a.n * a.I, 16 * 64 * 16),
                       stream, a, small);
  else
    hipLaunchKernelGGL(block_few_down, dim3((unsigned)(groups * ((a.H + 63) / 64))), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// Rows of the gate/up and the down tiles. One stage, three workgroups a CU. Groups of up to 48 rows
// on average take 32 rows a tile and the near-exact sums of the widened codes; larger ones 64 rows on
// FP8. The narrow tiles are the faster for up to some 20 rows, where the weights are the bound, and
// at most 13 % slower up to 48, where their sums are what they are kept for: a pass is off by 0.0017
// of its norm instead of 0.0020 to 0.0025. (Whole passes in a graph, 32 rows and 64, for 16, 32, 48 and 64 rows a
// group: top-8 of 64, H 2048, I 512 57 and 60, 63 and 62, 72 and 72, 77 and 72 us; I 1024 92 and 94, 99
// and 97, 113 and 112, 125 and 116; top-4 of 192, H 1024, I 512 74 and 75, 84 and 79, 91 and 88, 103 and
// 96; top-4 of 16, H 4096, I 1536 88 and 89, 101 and 91, 97 and 93, 103 and 108.) Widened sums in the
// 64-row tiles cost more: 4096 tokens, top-8 of 64 take 269 us against 211 (two workgroups a CU; at
// three the registers spill, 608).
static bool block_narrow(int64_t T, int64_t E, int64_t topk) { return T * topk <= 48 * E; }
static int gate_rows(int64_t T, int64_t E, int64_t topk) { return block_narrow(T, E, topk) ? 32 : 64; }
// 64 x 128 and 128 x 128 tiles, for 128, 256, 350, 512 and 1024 rows a group (whole passes in a graph):
// top-8 of 64, H 2048, I 512 90 and 96, 130 and 134, 150 and 155, 209 and 208, 369 and 356 us; I 1024 143 and
// 148, 208 and 206, 255 and 246, 349 and 336, 633 and 599; top-4 of 192, H 1024, I 512 126 and 129, 190
// and 192, 250 and 245, 346 and 334, 646 and 615; top-4 of 16, H 4096, I 1536 124 and 118, 178 and 172,
// 209 and 197, 283 and 262, 510 and 456.
static int down_rows(int64_t T, int64_t E, int64_t topk) {
  return block_narrow(T, E, topk) ? 32 : T * topk / E < 350 ? 64 : 128;
}
// A group adds at most one partial tile, and no tile is empty.
static int64_t max_tiles(int64_t n, int64_t E, int64_t bm) { return std::min(n, n / bm + E); }

struct BlockMoeLayout {
  int64_t tok, w, slot_row, tiles[2], hq, hs, y, ys, route, total;
};

static BlockMoeLayout block_moe_layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk) {
  BlockMoeLayout L;
  const int64_t n = T * topk;
  int64_t o = 0;
  const int64_t bm[2] = {gate_rows(T, E, topk), down_rows(T, E, topk)};
  L.tok = o, o += align256(n * 4);
  L.w = o, o += align256(n * 4);
  L.slot_row = o, o += align256(n * 4);
  for (int i = 0; i < 2; ++i) {
    L.tiles[i] = o;
    if (i == 0 || bm[1] != bm[0])
      o += align256((1 + max_tiles(n, E, bm[i])) * 16);
    else
      L.tiles[1] = L.tiles[0];
  }
  L.hq = o, o += align256(n * I);
  L.hs = o, o += align256(I / 128 * n * 4);
  L.y = o, o += align256(n * H * 2);
  L.ys = o, o += align256((H + 127) / 128 * n * 4);
  // where the order takes three launches: route_scatter's part
  L.route = o;
  if (!route_one(n, E))
    o += align256(E * 4) + align256((E + 1) * 4) + align256(n * 4) + (int64_t)route_workspace_bytes(T, topk, E);
  L.total = o;
  return L;
}

size_t block_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk) {
  const int64_t few = block_few(T, E, topk) ? align256(T * topk * I * 4) + align256(T * topk * H * 4) : 0;
  return (size_t)std::max(block_moe_layout(T, H, I, E, topk).total, few);
}

hipError_t launch_block_moe(const uint8_t* xq, const float* xs, const int32_t* ids, const float* tw, const uint8_t* w13,
                            const float* s13, const uint8_t* w2, const float* s2, uint16_t* out, uint8_t* out_q,
                            float* out_s, int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk, void* ws,
                            hipStream_t stream) {
  const dim3 blocks((unsigned)((T * ((H + 127) / 128) + 15) / 16));  // of 16 blocks of the output
  if (block_few(T, E, topk)) {
    float* const h = static_cast<float*>(ws);
    float* const y = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align256(T * topk * I * 4));
    const BlockFewArgs f{xq, xs, ids, tw, w13, w2, s13, s2, h, y, (int)T, (int)H, (int)I, (int)E, (int)topk,
                         (int)(T * topk), T * topk <= E ? 1 : 0};
    if (block_small(T, I, topk)) {
      const hipError_t e = launch_block_few(f, out, stream);
      return e != hipSuccess || out_q == nullptr ? e : launch_quantize_blocks(out, T, H, out_q, out_s, stream);
    }
    const hipError_t e = launch_block_few(f, nullptr, stream);
    if (e != hipSuccess) return e;
    if (out_q == nullptr) return launch_combine(y, ids, nullptr, T, topk, E, H, out, stream);
    hipLaunchKernelGGL(combine_block_quant, blocks, dim3(256), 0, stream, y, ids, T, (int)topk, (int)E, (int)H, out, out_q,
                       out_s);
    return hipGetLastError();
  }
  const BlockMoeLayout L = block_moe_layout(T, H, I, E, topk);
  uint8_t* b = static_cast<uint8_t*>(ws);
  const int64_t n = T * topk;
  int32_t* const slot_row = reinterpret_cast<int32_t*>(b + L.slot_row);
  uint16_t* const y = reinterpret_cast<uint16_t*>(b + L.y);
  float* const ys = reinterpret_cast<float*>(b + L.ys);
  RouteArgs r{};
  r.ids = ids;
  r.tw = tw;
  r.tok = reinterpret_cast<int32_t*>(b + L.tok);
  r.w = reinterpret_cast<float*>(b + L.w);
  r.slot_row = slot_row;
  for (int i = 0; i < 2; ++i) r.tiles[i] = reinterpret_cast<int4*>(b + L.tiles[i]);
  r.n = (int)n;
  r.E = (int)E;
  r.topk = (int)topk;
  r.bm[0] = gate_rows(T, E, topk);
  r.bm[1] = down_rows(T, E, topk);
  const dim3 chunks((unsigned)((n + kRouteThreads - 1) / kRouteThreads));
  hipError_t err = hipSuccess;
  if (route_one(n, E)) {
    hipLaunchKernelGGL(block_route, chunks, dim3(kRouteThreads), (size_t)E * (5 + kRouteWaves) * 4, stream, r);
    err = hipGetLastError();
  } else {
    uint8_t* at = b + L.route;
    int32_t* const counts = reinterpret_cast<int32_t*>(at);
    int32_t* const offsets = reinterpret_cast<int32_t*>(at += align256(E * 4));
    int32_t* const perm = reinterpret_cast<int32_t*>(at += align256((E + 1) * 4));
    err = launch_route(ids, T, topk, E, 0, counts, offsets, perm, slot_row, at + align256(n * 4), stream);
    if (err == hipSuccess) {
      hipLaunchKernelGGL(block_route_rest, chunks, dim3(kRouteThreads), 0, stream, r, offsets, perm);
      err = hipGetLastError();
    }
  }
  if (err != hipSuccess) return err;
  BlockArgs p{};
  p.A = xq;
  p.sA = xs;
  p.a_rows = T;
  p.B = w13;
  p.sB = s13;
  p.tiles = r.tiles[0];
  p.tok = r.tok;
  p.hq = b + L.hq;
  p.hs = reinterpret_cast<float*>(b + L.hs);
  p.topk = (int)topk;
  p.N = (int)(2 * I);
  p.K = (int)H;
  int64_t tiles = max_tiles(n, E, r.bm[0]);
  err = r.bm[0] == 32 ? run_tiled<32, 256, 1, 4, kGateUp, 3, 1, true>(p, tiles, stream)
                      : run_tiled<64, 256, 1, 4, kGateUp, 3, 1>(p, tiles, stream);
  if (err != hipSuccess) return err;
  BlockArgs d{};
  d.A = p.hq;
  d.sA = p.hs;
  d.a_rows = n;
  d.B = w2;
  d.sB = s2;
  d.tiles = r.tiles[1];
  d.tw = r.w;
  d.y16 = y;
  d.ys = ys;
  d.N = (int)H;
  d.K = (int)I;
  tiles = max_tiles(n, E, r.bm[1]);
  err = r.bm[1] == 32   ? run_tiled<32, 256, 1, 4, kDown, 4, 1>(d, tiles, stream)
        : r.bm[1] == 64 ? run_tiled<64, 128, 2, 2, kDown, 4, 1>(d, tiles, stream)
                        : run_tiled<128, 128, 2, 2, kDown, 3, 1>(d, tiles, stream);
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(combine_half, blocks, dim3(256), 0, stream, y, ys, ids, slot_row, T, (int)topk, (int)E, (int)H, out,
                     out_q, out_s);
  return hipGetLastError();
}

}  // namespace w8a8
