// FP8 e4m3 product with a scale for each block of 128: activations [M, K]
// carry one scale per token and 128 features, weights [N, K] one per block of
// 128 rows x 128 features:
//     y[m,n] = sum_j S_x[j,m] S_w[n / 128, j] sum_{k in j} e4m3(xq[m,k]) e4m3(wq[n,k])  (+ b[n])
// Each block's inner sum is one chain of MFMAs started at zero, multiplied by
// its scale in fp32 and added to the fp32 accumulator.
#include "q8_device.hpp"
#include "q8_kv.hpp"

namespace q8 {
namespace {

constexpr int kThreads = 256;

template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t off, float* v) {
  if constexpr (DT == DT_F32) {
    const v4i* p = (const v4i*)((const float*)base + off);
    Chunk<DT>::decode(p[0], v);
    Chunk<DT>::decode(p[1], v + 4);
  } else {
    Chunk<DT>::decode(*(const v4i*)((const uint16_t*)base + off), v);
  }
}

// e4m3 codes of 8 values, x / s rounded as the correctly rounded quotient is
// (16-bit inputs: two FMAs on RN(1/s), the same codes over that whole domain)
template <int DT>
__device__ __forceinline__ v2i codes8(const float* v, float s) {
  const float r = 1.0f / s;
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = DT == DT_F32 ? v[e] / s : __builtin_copysignf(quot_fma(v[e], s, r), v[e]);
    q[e] = fminf(fmaxf(y, -kFp8Max), kFp8Max);
  }
  return v2i{(int)pack4_e4m3(q[0], q[1], q[2], q[3]), (int)pack4_e4m3(q[4], q[5], q[6], q[7])};
}

// One 16-lane row of a wave per group of 128 features of one token.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_quant_act_block(const void* __restrict__ x, int64_t M, int64_t K, int groups,
                                                              uint8_t* __restrict__ xq, float* __restrict__ x_scale) {
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
  if (i >= M * groups) return;                                 // whole 16-lane rows leave together
  const int64_t m = i / groups;
  const int j = (int)(i - m * groups), k = j * kScaleBlock + 8 * (threadIdx.x & 15);
  float v[8] = {};
  if (k < K) load8<DT>(x, m * K + k, v);
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
  amax = __int_as_float(dpp_row_reduce(__float_as_int(amax), [](int a, int b) {
    return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
  }));
  float s = amax / kFp8Max;
  s = s < kEps ? kEps : s;
  if (k < K) *(v2i*)(xq + m * K + k) = codes8<DT>(v, s);
  if ((threadIdx.x & 15) == 0) x_scale[(int64_t)j * M + m] = s;
}

// One workgroup per 128 x 128 block of the weights (offline).
template <int DT>
__global__ __launch_bounds__(kThreads) void k_quant_weight_block(const void* __restrict__ w, int64_t N, int64_t K,
                                                                 uint8_t* __restrict__ wq, float* __restrict__ w_scale) {
  __shared__ float red[kThreads / 64];
  const int cols = (int)((K + kScaleBlock - 1) / kScaleBlock);
  const int64_t n0 = (int64_t)(blockIdx.x / cols) * kScaleBlock;
  const int k = (int)(blockIdx.x % cols) * kScaleBlock + 8 * (threadIdx.x & 15);
  const int r0 = threadIdx.x >> 4;
  float amax = 0.0f;
  for (int r = r0; r < kScaleBlock; r += kThreads / 16) {
    if (n0 + r >= N || k >= K) continue;
    float v[8];
    load8<DT>(w, (n0 + r) * K + k, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
  }
  amax = block_max<kThreads / 64>(amax, red);
  float s = amax / kFp8Max;
  s = s < kEps ? kEps : s;
  for (int r = r0; r < kScaleBlock; r += kThreads / 16) {
    if (n0 + r >= N || k >= K) continue;
    float v[8];
    load8<DT>(w, (n0 + r) * K + k, v);
    *(v2i*)(wq + (n0 + r) * K + k) = codes8<DT_F32>(v, s);
  }
  if (threadIdx.x == 0) w_scale[blockIdx.x] = s;
}

// One wave per 16 x 16 outputs, straight from memory.
template <int YDT>
__global__ __launch_bounds__(kThreads) void k_gemm_block(const uint8_t* __restrict__ xq, const float* __restrict__ x_scale,
                                                         int M, int K, const uint8_t* __restrict__ wq,
                                                         const float* __restrict__ w_scale, int N,
                                                         const float* __restrict__ bias, void* __restrict__ y) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, lg = lane >> 4;
  const int across = (N + 63) / 64;
  const int n0 = ((blockIdx.x % across) * (kThreads / 64) + wave) * 16, m0 = (blockIdx.x / across) * 16;
  if (n0 >= N) return;
  const int groups = (K + kScaleBlock - 1) / kScaleBlock;
  const int wr = n0 + lr < N ? n0 + lr : N - 1, xr = m0 + lr < M ? m0 + lr : M - 1;
  const uint8_t* wp = wq + (int64_t)wr * K;
  const uint8_t* xp = xq + (int64_t)xr * K;
  v4f acc = {0, 0, 0, 0};
  for (int j = 0; j < groups; ++j) {
    v8i a, b;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = j * kScaleBlock + 32 * lg + 16 * h;
      const v4i u = k < K ? *(const v4i*)(wp + k) : v4i{0, 0, 0, 0};
      const v4i w = k < K ? *(const v4i*)(xp + k) : v4i{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) { a[4 * h + i] = u[i]; b[4 * h + i] = w[i]; }
    }
    const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
    const float sc = x_scale[(int64_t)j * M + xr] * w_scale[(int64_t)(n0 / kScaleBlock) * groups + j];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += sc * part[i];
  }
  if (m0 + lr >= M) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + 4 * lg + i;
    if (n < N) store_out<YDT>(y, (int64_t)(m0 + lr) * N + n, acc[i] + (bias ? bias[n] : 0.0f));
  }
}

}  // namespace

hipError_t launch_quant_weight_block(const void* w, int dt, int64_t N, int64_t K, uint8_t* wq, float* w_scale,
                                     hipStream_t st) {
  const unsigned grid = (unsigned)(((K + kScaleBlock - 1) / kScaleBlock) * ((N + kScaleBlock - 1) / kScaleBlock));
  switch (dt) {
    case DT_F32: k_quant_weight_block<DT_F32><<<grid, kThreads, 0, st>>>(w, N, K, wq, w_scale); break;
    case DT_F16: k_quant_weight_block<DT_F16><<<grid, kThreads, 0, st>>>(w, N, K, wq, w_scale); break;
    default: k_quant_weight_block<DT_BF16><<<grid, kThreads, 0, st>>>(w, N, K, wq, w_scale); break;
  }
  return hipGetLastError();
}

hipError_t launch_quant_act_block(const void* x, int dt, int64_t M, int64_t K, uint8_t* xq, float* x_scale,
                                  hipStream_t st) {
  const int groups = (int)((K + kScaleBlock - 1) / kScaleBlock);
  const unsigned grid = (unsigned)((M * groups + kThreads / 16 - 1) / (kThreads / 16));
  switch (dt) {
    case DT_F32: k_quant_act_block<DT_F32><<<grid, kThreads, 0, st>>>(x, M, K, groups, xq, x_scale); break;
    case DT_F16: k_quant_act_block<DT_F16><<<grid, kThreads, 0, st>>>(x, M, K, groups, xq, x_scale); break;
    default: k_quant_act_block<DT_BF16><<<grid, kThreads, 0, st>>>(x, M, K, groups, xq, x_scale); break;
  }
  return hipGetLastError();
}

hipError_t launch_gemm_fp8_block(const uint8_t* xq, const float* x_scale, int64_t M, int64_t K, const uint8_t* wq,
                                 const float* w_scale, int64_t N, const float* bias, void* y, int ydt, hipStream_t st) {
  const unsigned grid = (unsigned)(((N + 63) / 64) * ((M + 15) / 16));
  if (ydt == DT_F16) k_gemm_block<DT_F16><<<grid, kThreads, 0, st>>>(xq, x_scale, (int)M, (int)K, wq, w_scale, (int)N, bias, y);
  else k_gemm_block<DT_BF16><<<grid, kThreads, 0, st>>>(xq, x_scale, (int)M, (int)K, wq, w_scale, (int)N, bias, y);
  return hipGetLastError();
}

}  // namespace q8
