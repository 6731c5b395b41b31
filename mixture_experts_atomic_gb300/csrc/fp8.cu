// Rows and weights in 8-bit floating point (eight.cuh): quantising and
// widening; and the steps around the experts' products on them (fp8_tc.cu):
// which row each slot takes, the rows themselves, and the sum of a token's
// slots.
#include "common.cuh"
#include "eight.cuh"
#include "fp8.cuh"

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

// 16 columns a thread, 8 neighbouring lanes a block.  Reads every element once
// and writes its byte; bound by HBM: 32768 x 4096
// bf16 66 us, 6.1 TB/s (8 columns a thread: 82).
template <typename T>
__global__ void __launch_bounds__(kRowThreads) quantize_rows_kernel(const T* __restrict__ x, int64_t L, int d,
                                                                    uint8_t* __restrict__ q, float* __restrict__ s) {
  const int nb = blocks8(d), sub = threadIdx.x & 7;
  const int64_t total = L * nb;
  for (int64_t b0 = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) >> 3; b0 - (threadIdx.x >> 3 & 3) < total;
       b0 += (int64_t)gridDim.x * (kRowThreads / 8)) {
    // (64-bit division only where the blocks do not fit 32 bits)
    const int64_t t = total >> 32 ? b0 / nb : (uint32_t)b0 / (uint32_t)nb;
    const int blk = (int)(b0 - t * nb), c = blk * kBlock8 + sub * 16;
    const bool in = b0 < total && c < d;
    float v[16];
    uint32_t m = 0u;
    if (in) {
      load8(x + t * d + c, v);
      load8(x + t * d + c + 8, v + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, abs_bits(v[i]));
    }
#pragma unroll
    for (int k = 4; k > 0; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
    const Scale8 sc = scale8(m);
    if (in) {
      *reinterpret_cast<uint4*>(q + t * d + c) = make_uint4(e4m3x4(v, sc.inv), e4m3x4(v + 4, sc.inv),
                                                            e4m3x4(v + 8, sc.inv), e4m3x4(v + 12, sc.inv));
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
    uint32_t o[8];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
      store_sector(x + 16 * i, o);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(v[8 * h + k]);
        store_sector(x + 16 * i + 8 * h, o);
      }
    }
  }
}

// ------------------------------------------------------------------ weights
// A block of 128 x 128 of W (R,N), transposed to q (N,R): 512 threads read rows
// of it and write rows of its transpose, through shared memory in between.
// 8 of 4096 x 14336, bf16: 227 us (6.2 TB/s), and back 224 (6.3).
constexpr int kWThreads = 512, kWPitch = 132;
template <typename T>
__global__ void __launch_bounds__(kWThreads) quantize_weights_kernel(const T* __restrict__ W, int R, int N,
                                                                     uint8_t* __restrict__ q, float* __restrict__ s) {
  __shared__ uint32_t top;
  __shared__ __align__(16) uint8_t t8[kBlock8 * kWPitch];  // [column][row]
  const int r0 = blockIdx.x * kBlock8, n0 = blockIdx.y * kBlock8;
  const int64_t e = blockIdx.z, base = e * R * N;
  if (threadIdx.x == 0) top = 0u;
  __syncthreads();
  // thread: 8 columns of rows 4 ty + i
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float v[4][8];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    load8(W + base + (int64_t)(r0 + 4 * ty + i) * N + n0 + 8 * tx, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) atomicMax(&top, m);
  __syncthreads();
  const Scale8 sc = scale8(top);
#pragma unroll
  for (int j = 0; j < 8; ++j) {  // four neighbouring rows of a column are four neighbouring bytes
    const float c[4] = {v[0][j], v[1][j], v[2][j], v[3][j]};
    *reinterpret_cast<uint32_t*>(t8 + (8 * tx + j) * kWPitch + 4 * ty) = e4m3x4(c, sc.inv);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kBlock8 * kBlock8 / 4; i += kWThreads) {
    const int c = i >> 5, w = i & 31;
    *reinterpret_cast<uint32_t*>(q + base + (int64_t)(n0 + c) * R + r0 + 4 * w) =
        *reinterpret_cast<const uint32_t*>(t8 + c * kWPitch + 4 * w);
  }
  if (threadIdx.x == 0) s[(e * (N / kBlock8) + blockIdx.y) * (R / kBlock8) + blockIdx.x] = sc.s;
}

// The layout the products read: blocks of 128 x 128 one after the other, each
// output's 128 bytes side by side.  A CTA that walks along the reduction then
// reads 16 KB after 16 KB of neighbouring memory, in place of 128 bytes from each
// of 128 rows (one token, d 4096, h 14336: the down projection, whose rows are
// 14 KB apart, ran at 2.0 TB/s so).
__global__ void __launch_bounds__(256) pack_weights_kernel(const uint4* __restrict__ q, int R, int N,
                                                           uint4* __restrict__ out) {
  const int64_t e = blockIdx.z;
  const uint4* src = q + (e * N + (int64_t)blockIdx.y * kBlock8) * (R / 16) + blockIdx.x * (kBlock8 / 16);
  uint4* dst = out + ((e * (N / kBlock8) + blockIdx.y) * (R / kBlock8) + blockIdx.x) * (kBlock8 * kBlock8 / 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = threadIdx.x + 256 * i;
    dst[j] = src[(int64_t)(j >> 3) * (R / 16) + (j & 7)];
  }
}

// PACKED: of the layout above.  CTAs side by side write pieces of the same rows (of
// the same columns: 365 us; and a byte at a time out of shared memory: 384).
template <bool PACKED>
__global__ void __launch_bounds__(kWThreads) dequantize_weights_kernel(const uint8_t* __restrict__ q,
                                                                       const float* __restrict__ s, int R, int N,
                                                                       __nv_bfloat16* __restrict__ W) {
  __shared__ __align__(16) uint8_t t8[kBlock8 * kWPitch];  // [column][row]
  const int n0 = blockIdx.x * kBlock8, r0 = blockIdx.y * kBlock8;
  const int64_t e = blockIdx.z, base = e * R * N;
#pragma unroll
  for (int i = 0; i < kBlock8 * kBlock8 / 4; i += kWThreads) {
    const int c = (i + (int)threadIdx.x) >> 5, w = threadIdx.x & 31;
    const int64_t at = PACKED ? ((int64_t)(n0 * (R / kBlock8) + r0) + c) * kBlock8 + 4 * w : (int64_t)(n0 + c) * R + r0 + 4 * w;
    *reinterpret_cast<uint32_t*>(t8 + c * kWPitch + 4 * w) = *reinterpret_cast<const uint32_t*>(q + base + at);
  }
  __syncthreads();
  const float sc = s[(e * (N / kBlock8) + blockIdx.x) * (R / kBlock8) + blockIdx.y];
#pragma unroll
  for (int i = 0; i < kBlock8 * kBlock8 / 8; i += kWThreads) {  // two columns of four rows
    const int c = 2 * (threadIdx.x & 63), r = 4 * ((i + (int)threadIdx.x) >> 6);
    float v0[4], v1[4];
    e4m3_values(*reinterpret_cast<const uint32_t*>(t8 + c * kWPitch + r), sc, v0);
    e4m3_values(*reinterpret_cast<const uint32_t*>(t8 + (c + 1) * kWPitch + r), sc, v1);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<uint32_t*>(W + base + (int64_t)(r0 + r + k) * N + n0 + c) = pack_bf16x2(v0[k], v1[k]);
  }
}

// ------------------------------------------------------------------ routing
// Rows for the slots: an expert's slots take its rows in any order (what a row
// holds does not depend on its neighbours, and the sum of a token's slots goes
// by slot), an id outside [0,E) takes none.
constexpr int kChunkSlots = 4096, kRouteThreads = 512;

__device__ __forceinline__ void count_chunk(const int32_t* ids, int64_t n, int E, int chunk, int* hist) {
  for (int e = threadIdx.x; e < E; e += kRouteThreads) hist[e] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kChunkSlots / kRouteThreads; ++i) {
    const int64_t j = (int64_t)chunk * kChunkSlots + i * kRouteThreads + threadIdx.x;
    if (j < n && (unsigned)ids[j] < (unsigned)E) atomicAdd(&hist[ids[j]], 1);
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kRouteThreads) route_count_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                                    int32_t* __restrict__ cnt) {
  __shared__ int hist[kMaxE];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  count_chunk(ids, n, E, blockIdx.x, hist);
  for (int e = threadIdx.x; e < E; e += kRouteThreads) cnt[(int64_t)blockIdx.x * E + e] = hist[e];
}

// ONE: the slots are one chunk, counted here
template <bool ONE>
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                                    const int32_t* cnt, int chunks, int32_t* hdr,
                                                                    int32_t* tile_e, int32_t* pos) {
  static_assert(kMaxE <= kRouteThreads, "a thread an expert");
  __shared__ int hist[kMaxE];
  __shared__ int warp_sums[kRouteThreads / 32];
  const int e = threadIdx.x, lane = e & 31, wp = e >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (ONE) count_chunk(ids, n, E, 0, hist);
  else asm volatile("griddepcontrol.wait;" ::: "memory");
  int all = 0, before = 0;
  if (e < E) {
    if (ONE) {
      all = hist[e];
    } else {
#pragma unroll 8
      for (int c = 0; c < chunks; ++c) {
        const int v = cnt[(int64_t)c * E + e];
        all += v;
        before += c < (int)blockIdx.x ? v : 0;
      }
    }
  }
  // padded row offsets: an exclusive sum over the experts
  const int tiles = (all + 255) / 256;
  int sum = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) warp_sums[wp] = sum;
  __syncthreads();
  int base = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kRouteThreads / 32; ++i) {
    base += i < wp ? warp_sums[i] : 0;
    total += warp_sums[i];
  }
  const int first = base + sum - tiles;  // the expert's first row tile
  if (e < E) hist[e] = first * 256 + before;
  if (blockIdx.x == 0) {
    for (int i = 0; i < tiles; ++i) tile_e[first + i] = e;
    if (e == 0) {
      hdr[0] = 0;
      hdr[1] = total;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kChunkSlots; i += kRouteThreads) {
    const int64_t j = (int64_t)blockIdx.x * kChunkSlots + i;
    if (j >= n) break;
    const int id = ids[j];
    pos[j] = (unsigned)id < (unsigned)E ? atomicAdd(&hist[id], 1) : -1;
  }
}

// A token's row to the row of each of its slots, a warp a token; bf16 rows are
// quantised on the way (T = uint8_t: given in 8 bits, with scales sx).  Scales
// go to (d/128, rows), where the products' threads, a row each, read them side
// by side.
template <typename T>
__global__ void __launch_bounds__(256) gather_rows_kernel(const T* __restrict__ x, const float* __restrict__ sx,
                                                          const int32_t* pos, int64_t L, int d, int K, int64_t rows,
                                                          uint8_t* __restrict__ x8, float* __restrict__ s8) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= L) return;
  const int mine = lane < K ? pos[t * K + lane] : -1;
  if (!__any_sync(0xffffffffu, mine >= 0)) return;
  int to[kMaxK];
#pragma unroll
  for (int k = 0; k < kMaxK; ++k) to[k] = __shfl_sync(0xffffffffu, mine, k);  // -1 from K on
  if constexpr (sizeof(T) == 1) {
    const uint4* src = reinterpret_cast<const uint4*>(x + t * d);
    constexpr int U = 4;  // words of a lane on their way
    for (int c0 = lane; c0 < d / 16; c0 += 32 * U) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + 32 * u < d / 16) v[u] = src[c0 + 32 * u];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + 32 * u < d / 16) {
#pragma unroll
          for (int k = 0; k < kMaxK; ++k)
            if (to[k] >= 0) reinterpret_cast<uint4*>(x8 + (int64_t)to[k] * d)[c0 + 32 * u] = v[u];
        }
    }
    for (int b = lane; b < d / kBlock8; b += 32) {
      const float v = sx[t * (d / kBlock8) + b];
#pragma unroll
      for (int k = 0; k < kMaxK; ++k)
        if (to[k] >= 0) s8[b * rows + to[k]] = v;
    }
  } else {
    constexpr int U = 4;
    for (int c0 = 0; c0 < d / 8; c0 += 32 * U) {  // 8 columns a lane, 16 lanes a block
      float v[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + 32 * u + lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
        if (c < d / 8) load8(x + t * d + 8 * c, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + 32 * u + lane;
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[u][i]));
#pragma unroll
        for (int k = 8; k > 0; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
        const Scale8 sc = scale8(m);
        const uint2 o = make_uint2(e4m3x4(v[u], sc.inv), e4m3x4(v[u] + 4, sc.inv));
#pragma unroll
        for (int k = 0; k < kMaxK; ++k) {
          if (to[k] >= 0 && c < d / 8) {
            reinterpret_cast<uint2*>(x8 + (int64_t)to[k] * d)[c] = o;
            if ((lane & 15) == 0) s8[(int64_t)(c >> 4) * rows + to[k]] = sc.s;
          }
        }
      }
    }
  }
}

// y[t] = sum_k gates[t,k] Y[pos[t,k]], slot by slot; eight columns a thread.
// Y fp32, or fp16 with scales sy (d/128, rows).  NaN where the products gave up
// (hdr[0]).  KM: slots whose loads are in flight together (all of them).
// Bound by HBM: 8192 x 4096, 2 slots: 200 MB.
__device__ __forceinline__ void eight(const float* p, float* v) { load8(p, v); }
__device__ __forceinline__ void eight(const __half* p, float* v) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <typename T, int KM>
__global__ void __launch_bounds__(256) combine_rows_kernel(const T* Y, const float* sy, int64_t rows, const int32_t* hdr,
                                                           const int32_t* pos, const float* __restrict__ gates, int64_t L,
                                                           int d, int K, __nv_bfloat16* __restrict__ y) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per_row = d / 8;
  if (i >= L * per_row) return;
  const int64_t t = i <= 0xffffffffll ? (uint32_t)i / (uint32_t)per_row : i / per_row;
  const int c = (int)(i - t * per_row);
  float v[KM][8], g[KM];
  int r[KM];
#pragma unroll
  for (int k = 0; k < KM; ++k) r[k] = k < K ? pos[t * K + k] : -1;
#pragma unroll
  for (int k = 0; k < KM; ++k) {
    // (an empty slot reads row 0 and leaves it: branches around the loads would
    // put one behind the other, 221 in place of 85 us at 16000 x 2048, 6 slots)
    const int64_t row = max(r[k], 0);
    const float gate = k < K ? gates[t * K + k] : 0.f;
    const float scale = sizeof(T) == 2 ? sy[(int64_t)(c / (kBlock8 / 8)) * rows + row] : 1.f;
    eight(Y + row * d + 8 * c, v[k]);
    g[k] = r[k] >= 0 ? gate * scale : 0.f;
  }
#pragma unroll
  for (int k = 0; k < KM; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[k][j] = r[k] >= 0 ? v[k][j] : 0.f;
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < KM; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = fmaf(g[k], v[k][j], o[j]);
  if (hdr[0]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = __uint_as_float(0x7fffffffu);
  }
  reinterpret_cast<uint4*>(y)[i] = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                                              pack_bf16x2(o[6], o[7]));
}

unsigned row_blocks(int64_t threads) {
  const int64_t need = (threads + kRowThreads - 1) / kRowThreads, most = (int64_t)sm_count() * 16;
  return (unsigned)(need < most ? need : most);
}

// a launch that may start while the one before it still runs (it waits for its results itself)
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), int64_t grid, int threads, cudaStream_t st, A... a) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(a)...);
}

int64_t route_chunks(const moeblaze_shape& s) { return (s.L * s.K + kChunkSlots - 1) / kChunkSlots; }

// places of a call's scratch; bytes: how many it takes (base may be null)
Fp8Scratch scratch(const moeblaze_shape& s, void* base, size_t* bytes) {
  Fp8Scratch w;
  w.rows = max_padded_rows(s.L * s.K, s.E);
  size_t at = 0;
  auto take = [&](size_t n) {
    char* p = static_cast<char*>(base) + at;
    at += align_up(n, 256);
    return static_cast<void*>(p);
  };
  w.hdr = (int32_t*)take(256);
  w.cnt = (int32_t*)take(sizeof(int32_t) * route_chunks(s) * s.E);
  w.tile_e = (int32_t*)take(sizeof(int32_t) * (w.rows / 256));
  w.pos = (int32_t*)take(sizeof(int32_t) * s.L * s.K);
  w.x8 = (uint8_t*)take((size_t)w.rows * s.d);
  w.sx = (float*)take(sizeof(float) * w.rows * (s.d / kBlock8));
  w.h8 = (uint8_t*)take((size_t)w.rows * s.h);
  w.sh = (float*)take(sizeof(float) * w.rows * (s.h / kBlock8));
  w.y = (__half*)take(sizeof(__half) * w.rows * s.d);
  w.sy = (float*)take(sizeof(float) * w.rows * (s.d / kBlock8));
  *bytes = at;
  return w;
}

Fp8FewScratch few_scratch(const moeblaze_shape& s, void* base, size_t* bytes) {
  Fp8FewScratch w;
  w.rows = few_max_rows(s);
  size_t at = 0;
  auto take = [&](size_t n) {
    char* p = static_cast<char*>(base) + at;
    at += align_up(n, 256);
    return static_cast<void*>(p);
  };
  w.hdr = (int32_t*)take(256);
  w.entries = (int32_t*)take(16 * few_max_entries(s));
  w.cnt = (int32_t*)take(sizeof(int32_t) * few_max_entries(s) * (few_tiles_up(s) + few_tiles_down(s)));
  w.pos = (int32_t*)take(sizeof(int32_t) * s.L * s.K);
  w.x8 = (uint8_t*)take((size_t)w.rows * s.d);
  w.sx = (float*)take(sizeof(float) * w.rows * (s.d / kBlock8));
  w.h8 = (uint8_t*)take((size_t)w.rows * s.h);
  w.sh = (float*)take(sizeof(float) * w.rows * (s.h / kBlock8));
  w.y = (float*)take(sizeof(float) * w.rows * s.d);
  w.parts = (float*)take(sizeof(float) * sm_count() * 2 * 2 * few_part_tokens(s) * 128);
  *bytes = at;
  return w;
}

template <typename T>
auto combine_kernel(int K) {
  return K <= 2 ? combine_rows_kernel<T, 2> : K <= 4 ? combine_rows_kernel<T, 4>
       : K <= 6 ? combine_rows_kernel<T, 6> : combine_rows_kernel<T, kMaxK>;
}

// The most tokens a call of this shape takes the path for few tokens with, by
// slots an expert.  That path reads an expert's weights once for each 32 of its
// tokens, the prompts' once for each 256; it has more than 32 where the average is
// high or the routing uneven.  Both paths, us (few | prompts), slots drawn evenly,
// and with experts as unequal as exp of a normal number:
//   d 4096, h 14336, 2 of 8     16  263 | 350, 287 | 343   20  269 | 351, 285 | 317   24  281 | 351, 350 | 351
//   d 4096, h 1536, 8 of 128    16  454 | 657, 470 | 492   20  468 | 659, 502 | 515   24  485 | 666, 574 | 534
//   d 4096, h 14336, 2 of 8, SiLU  16  216 | 241, 222 | 234   20  221 | 241, 253 | 237   24  224 | 241, 263 | 241
//   d 2048, h 1408, 6 of 64     16  142 | 189, 145 | 153   20  148 | 188, 160 | 156   24  155 | 188, 174 | 159
//   d 2048, h 8192, 2 of 8      16  111 | 123, 120 | 122   20  114 | 124, 132 | 122   24  119 | 124, 130 | 112
//   d 1024, h 2816, 1 of 200     8  364 | 541, 269 | 252   12  397 | 543, 329 | 281   16  426 | 546, 399 | 303
//   d 1024, h 4096, 1 of 16      8   70 | 79,   69 | 66    12   74 | 79,   76 | 69    16   78 | 79,   78 | 70
//   d 1024, h 2048, 2 of 32      8   70 | 84,   69 | 68    12   75 | 84,   72 | 67    16   78 | 85,   81 | 75
//   d 512, h 512, 8 of 256       8   88 | 118,  86 | 77    12   98 | 119, 101 | 86    16  108 | 121, 114 | 92
//   d 256, h 512, 4 of 128       8   45 | 54,   44 | 41    12   50 | 55,   47 | 45    16   52 | 55,   53 | 42
// So up to where one routing loses as much as the other gains: 20, and 12 where a
// tile of the prompts' up projection has fewer than 16 blocks.  Where all slots fall
// on one of many experts the prompts' path is up to four times as fast (d 1024, h
// 2816, 1 of 200, 12 slots an expert: 187 | 48).
constexpr int kFewLong = 20, kFewShort = 12, kLongBlocks = 16;
// Layers so small that the prompts' path has few rounds of short tiles are its own
// with one token already: rounds of tiles over the pairs of SMs, by the blocks of a
// tile and three for its end, of both products (few | prompts at 2 and 8 slots):
//   18  d 512, h 1024, 2 of 8    23 | 22, 24 | 22      33  d 512, h 2048, 2 of 8    25 | 31, 26 | 32
//   22  d 1024, h 1024, 2 of 4   26 | 24, 27 | 24      33  d 2048, h 512, 2 of 16   31 | 37, 33 | 38
//   26  d 1024, h 1536, 2 of 4   27 | 26, 28 | 26      38  d 2048, h 2048, 1 of 1   27 | 32, 27 | 32
//   30  d 1536, h 1536, 1 of 2   26 | 28, 28 | 29      46  d 1024, h 4096, 1 of 1   27 | 33, 28 | 33
// SiLU, whose up projection has half as many tiles:
//   30  d 1024, h 2048, 2 of 8   37 | 32, 37 | 32      57  d 1024, h 4096, 2 of 8   48 | 45, 50 | 46
//   38  d 2048, h 2048, 1 of 2   35 | 34, 36 | 34      66  d 2048, h 1408, 4 of 16  58 | 56, 58 | 59
constexpr int64_t kSmallSwiglu = 28, kSmallSilu = 60;
int64_t few_tokens(const moeblaze_shape& s) {
  const bool sw = s.act == MOEBLAZE_SWIGLU;
  const int64_t pairs = sm_count() / 2;
  const int64_t up = (int64_t)s.E * (sw ? s.h / 128 : (s.h + 255) / 256), down = (int64_t)s.E * ((s.d + 255) / 256);
  const int64_t blocks = (up + pairs - 1) / pairs * (s.d / kBlock8 + 3) + (down + pairs - 1) / pairs * (s.h / kBlock8 + 3);
  if (blocks < (sw ? kSmallSwiglu : kSmallSilu)) return 0;
  const int64_t per = s.d / kBlock8 >= kLongBlocks ? kFewLong : kFewShort;
  const int64_t slots = per * s.E < kFewSlots ? per * s.E : kFewSlots;
  return slots / s.K;
}

}  // namespace

// of any call of at most s.L tokens
size_t fp8_ws_bytes(const moeblaze_shape& s) {
  size_t n = 0, m = 0;
  moeblaze_shape f = s;
  f.L = s.L < few_tokens(s) ? s.L : few_tokens(s);
  if (f.L > 0) few_scratch(f, nullptr, &n);
  if (s.L > few_tokens(s)) scratch(s, nullptr, &m);
  return n > m ? n : m;
}

moeblaze_status launch_fp8_forward(const moeblaze_shape& s, const void* x, const float* x_scales, const int32_t* ids,
                                   const float* gates, const moeblaze_fp8_experts& w, __nv_bfloat16* y, void* ws,
                                   cudaStream_t st) {
  if (s.L == 0) return MOEBLAZE_OK;
  size_t n = 0;
  const int64_t combine = (s.L * (s.d / 8) + 255) / 256;
  if (s.L <= few_tokens(s)) {
    const Fp8FewScratch sc = few_scratch(s, ws, &n);
    const moeblaze_status r = launch_fp8_few(s, x, x_scales, ids, w, sc, st);
    if (r != MOEBLAZE_OK) return r;
    MB_CUDA(launch_dependent(combine_kernel<float>(s.K), combine, 256, st, sc.y, (const float*)nullptr, sc.rows, sc.hdr,
                             sc.pos, gates, s.L, s.d, s.K, y));
    count_launch();
    return MOEBLAZE_OK;
  }
  const Fp8Scratch sc = scratch(s, ws, &n);
  const int64_t slots = s.L * s.K, chunks = route_chunks(s);
  if (chunks == 1) {
    route_place_kernel<true><<<1, kRouteThreads, 0, st>>>(ids, slots, s.E, sc.cnt, 1, sc.hdr, sc.tile_e, sc.pos);
    MB_CUDA(cudaGetLastError());
  } else {
    route_count_kernel<<<(unsigned)chunks, kRouteThreads, 0, st>>>(ids, slots, s.E, sc.cnt);
    MB_CUDA(cudaGetLastError());
    MB_CUDA(launch_dependent(route_place_kernel<false>, chunks, kRouteThreads, st, ids, slots, s.E, sc.cnt, (int)chunks,
                             sc.hdr, sc.tile_e, sc.pos));
    count_launch();
  }
  const int64_t warps = (s.L + 7) / 8;
  if (x_scales)
    MB_CUDA(launch_dependent(gather_rows_kernel<uint8_t>, warps, 256, st, (const uint8_t*)x, x_scales, sc.pos, s.L, s.d,
                             s.K, sc.rows, sc.x8, sc.sx));
  else
    MB_CUDA(launch_dependent(gather_rows_kernel<__nv_bfloat16>, warps, 256, st, (const __nv_bfloat16*)x, x_scales, sc.pos,
                             s.L, s.d, s.K, sc.rows, sc.x8, sc.sx));
  count_launch(2);
  const moeblaze_status r = launch_fp8_products(s, w, sc, st);
  if (r != MOEBLAZE_OK) return r;
  MB_CUDA(launch_dependent(combine_kernel<__half>(s.K), combine, 256, st, sc.y, sc.sy, sc.rows, sc.hdr, sc.pos, gates, s.L,
                           s.d, s.K, y));
  count_launch();
  return MOEBLAZE_OK;
}

moeblaze_status launch_fp8_quantize_weights(int E, int R, int N, int dtype, const void* W, void* q, float* scales,
                                            cudaStream_t st) {
  const dim3 g((unsigned)(R / kBlock8), (unsigned)(N / kBlock8), (unsigned)E);
  if (dtype == MOEBLAZE_BF16)
    quantize_weights_kernel<<<g, kWThreads, 0, st>>>((const __nv_bfloat16*)W, R, N, (uint8_t*)q, scales);
  else
    quantize_weights_kernel<<<g, kWThreads, 0, st>>>((const float*)W, R, N, (uint8_t*)q, scales);
  MB_CUDA(cudaGetLastError());
  count_launch();
  return MOEBLAZE_OK;
}

moeblaze_status launch_fp8_pack(int E, int R, int N, const void* q, void* packed, cudaStream_t st) {
  const dim3 g((unsigned)(R / kBlock8), (unsigned)(N / kBlock8), (unsigned)E);
  pack_weights_kernel<<<g, 256, 0, st>>>((const uint4*)q, R, N, (uint4*)packed);
  MB_CUDA(cudaGetLastError());
  count_launch();
  return MOEBLAZE_OK;
}

moeblaze_status launch_fp8_dequantize_weights(int E, int R, int N, const void* q, bool packed, const float* scales, void* W,
                                              cudaStream_t st) {
  const dim3 g((unsigned)(N / kBlock8), (unsigned)(R / kBlock8), (unsigned)E);
  auto kern = packed ? dequantize_weights_kernel<true> : dequantize_weights_kernel<false>;
  kern<<<g, kWThreads, 0, st>>>((const uint8_t*)q, scales, R, N, (__nv_bfloat16*)W);
  MB_CUDA(cudaGetLastError());
  count_launch();
  return MOEBLAZE_OK;
}

moeblaze_status launch_fp8_quantize_rows(int64_t L, int d, int dtype, const void* x, void* q, float* scales,
                                         cudaStream_t st) {
  const unsigned g = row_blocks(L * blocks8(d) * 8);
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
