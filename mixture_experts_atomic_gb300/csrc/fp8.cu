// Rows in 8-bit floating point (eight.cuh): quantising and widening.
#include "common.cuh"
#include "eight.cuh"

namespace moeblaze {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16x2(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 f = reinterpret_cast<const float4*>(p)[i];
    v[4 * i] = f.x;
    v[4 * i + 1] = f.y;
    v[4 * i + 2] = f.z;
    v[4 * i + 3] = f.w;
  }
}

// 8 columns a thread, 16 neighbouring lanes a block.  Reads every element once
// and writes its byte; bound by HBM.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) quantize_rows_kernel(const T* __restrict__ x, int64_t L, int d,
                                                                    uint8_t* __restrict__ q, float* __restrict__ s) {
  const int nb = blocks8(d), sub = threadIdx.x & 15;
  const int64_t total = L * nb;
  for (int64_t b0 = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) >> 4; b0 - (threadIdx.x >> 4 & 1) < total;
       b0 += (int64_t)gridDim.x * (kRowThreads / 16)) {
    const int64_t t = b0 / nb;
    const int blk = (int)(b0 - t * nb), c = blk * kBlock8 + sub * 8;
    const bool in = b0 < total && c < d;
    float v[8];
    uint32_t m = 0u;
    if (in) {
      load8(x + t * d + c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    }
#pragma unroll
    for (int k = 8; k > 0; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
    const Scale8 sc = scale8(m);
    if (in) {
      *reinterpret_cast<uint2*>(q + t * d + c) = make_uint2(e4m3x4(v, sc.inv), e4m3x4(v + 4, sc.inv));
      if (sub == 0) s[b0] = sc.s;
    }
  }
}

// 16 columns a thread
template <typename T>
__global__ void __launch_bounds__(kRowThreads) dequantize_rows_kernel(const uint8_t* __restrict__ q,
                                                                      const float* __restrict__ s, int64_t words, int d,
                                                                      T* __restrict__ x) {
  const int per_row = d / 16;
  for (int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; i < words;
       i += (int64_t)gridDim.x * kRowThreads) {
    const int64_t t = words <= 0xffffffffll ? (uint32_t)i / (uint32_t)per_row : i / per_row;
    const int c = (int)(i - t * per_row) * 16;
    const uint4 u = reinterpret_cast<const uint4*>(q)[i];
    const float sc = s[t * blocks8(d) + c / kBlock8];
    float v[16];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) e4m3_values(w[k], sc, v + 4 * k);
    if constexpr (sizeof(T) == 2) {
      uint4* o = reinterpret_cast<uint4*>(x) + 2 * i;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        o[k] = make_uint4(pack_bf16x2(v[8 * k], v[8 * k + 1]), pack_bf16x2(v[8 * k + 2], v[8 * k + 3]),
                          pack_bf16x2(v[8 * k + 4], v[8 * k + 5]), pack_bf16x2(v[8 * k + 6], v[8 * k + 7]));
    } else {
      float4* o = reinterpret_cast<float4*>(x) + 4 * i;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
  }
}

unsigned row_blocks(int64_t threads) {
  const int64_t need = (threads + kRowThreads - 1) / kRowThreads, most = (int64_t)sm_count() * 16;
  return (unsigned)(need < most ? need : most);
}

}  // namespace

moeblaze_status launch_fp8_quantize_rows(int64_t L, int d, int dtype, const void* x, void* q, float* scales,
                                         cudaStream_t st) {
  const unsigned g = row_blocks(L * blocks8(d) * 16);
  if (dtype == MOEBLAZE_BF16)
    quantize_rows_kernel<<<g, kRowThreads, 0, st>>>((const __nv_bfloat16*)x, L, d, (uint8_t*)q, scales);
  else
    quantize_rows_kernel<<<g, kRowThreads, 0, st>>>((const float*)x, L, d, (uint8_t*)q, scales);
  MB_CUDA(cudaGetLastError());
  count_launch();
  return MOEBLAZE_OK;
}

moeblaze_status launch_fp8_dequantize_rows(int64_t L, int d, int dtype, const void* q, const float* scales, void* x,
                                           cudaStream_t st) {
  const int64_t words = L * (d / 16);
  const unsigned g = row_blocks(words);
  if (dtype == MOEBLAZE_BF16)
    dequantize_rows_kernel<<<g, kRowThreads, 0, st>>>((const uint8_t*)q, scales, words, d, (__nv_bfloat16*)x);
  else
    dequantize_rows_kernel<<<g, kRowThreads, 0, st>>>((const uint8_t*)q, scales, words, d, (float*)x);
  MB_CUDA(cudaGetLastError());
  count_launch();
  return MOEBLAZE_OK;
}

}  // namespace moeblaze
