// Norms with the residual sum fused, and their backward: the norm in front of
// an MoE layer (pre-norm block), over rows of d elements.  Layer norm (norm.cu):
//
//   s = x (+ residual)     mu = mean(s)     rstd = 1 / sqrt(var(s) + eps)
//   y = (s - mu) rstd w + b
//
//   g = dy w, xh = (s - mu) rstd
//   ds = rstd (g - mean(g) - xh mean(g xh)) (+ dsum)
//   dw = sum_t dy xh,  db = sum_t dy
//
// Root-mean-square norm (RMS, rmsnorm.cu): the same with mu = 0, without b, db
// and mean(g); and, with Q8, the rows once more in e4m3 with a scale for each
// 128 columns, as the 8-bit products read them.
//
// Everything is computed in fp32 and rounded once at the store.  Both passes
// read every input and write every output once: the row lives in registers
// between the statistics and the normalisation, and the variance is taken of
// the centred row (a second sum over registers, not E[s^2] - mu^2, which
// would cancel for rows with an offset).  Bound by HBM: 32768 x 4096 bf16,
// with residual and dsum 1.07 GB each way, takes 154 us forward (6.95 TB/s)
// and 178 us backward (6.0 TB/s, where the instructions of a row come to
// three fifths of the issue slots).  The RMS norm's backward has fewer of them:
// 165 us (6.5 TB/s).  Its forward with Q8 as well as y moves 1.21 GB in 171 us;
// a block's largest is taken across the 16 lanes (bf16) that hold it.
//
// A row is spread over TPR threads (one warp, or a whole CTA), NV 16-byte
// words of VEC elements per thread.
#pragma once

#include "common.cuh"
#include "eight.cuh"

namespace moeblaze {
namespace {

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
  T v[VEC];
};

__device__ __forceinline__ float ld_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float ld_f32(float v) { return v; }
__device__ __forceinline__ void st_t(__nv_bfloat16& o, float v) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void st_t(float& o, float v) { o = v; }

// a piece's elements as floats, and back; pairs of bf16 in one conversion
template <typename T, int VEC>
__device__ __forceinline__ void to_floats(const Vec<T, VEC>& p, float (&v)[VEC]) {
  if constexpr (sizeof(T) == 2 && VEC >= 2) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const float2 f = unpack_bf16x2(reinterpret_cast<const uint32_t*>(&p)[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = ld_f32(p.v[i]);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> from_floats(const float (&v)[VEC]) {
  Vec<T, VEC> p;
  if constexpr (sizeof(T) == 2 && VEC >= 2) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) reinterpret_cast<uint32_t*>(&p)[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) st_t(p.v[i], v[i]);
  }
  return p;
}

// fp32 pairs: each half an ordinary fp32 operation, one instruction for both
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// sum over the TPR threads of a row; `red` holds one float per warp of the
// row and is not shared with another reduction in flight
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += red[i];
  }
  return v;
}

// RMS: a mean of squares that fp32 does not hold, or holds with few digits (and
// no eps in front of it), is formed again of values times `sum`.  2^-80 leaves
// room for every row: squares below 2^96, 2^24 columns of them below 2^120; and
// 2^100 as well, for rows whose mean is below 2^-100: squares of fp32's smallest
// value are 2^-98, all of a row below 2^124.  The row itself goes on times `row`
// and `rstd` as 1 / sqrt(mean + eps) times rstd: neither it nor its elements
// leave the normal numbers where y does not (rstd alone is subnormal for values
// near fp32's largest, and infinite below 2^-128).
__device__ __forceinline__ bool out_of_range(float ms) { return !(ms <= 3.402823466e38f) || ms < 0x1p-100f; }
struct Range {
  float sum, row, rstd;  // sum = row rstd
};
__device__ __forceinline__ Range into_range(float ms) {
  return ms < 1.f ? Range{0x1p100f, 0x1p100f, 1.f} : Range{0x1p-80f, 0x1p-16f, 0x1p-64f};
}
// what the row times r.row is multiplied with; mean: of the squares of the row times r.sum
__device__ __forceinline__ float rstd_in_range(const Range& r, float mean, float eps) {
  return r.rstd / sqrtf(mean + eps * r.sum * r.sum);
}

constexpr int kNormWarps = 4;  // rows per CTA when a warp holds a row

template <int TPR>
constexpr int norm_threads() {
  return TPR == 32 ? 32 * kNormWarps : TPR;
}

// ------------------------------------------------------------------ forward
// SHIFT: rows that do not start on 16 bytes.  A thread still loads the whole
// words the row lies in, whose columns then begin `shift` before the row; the
// first and the last word are shared with its neighbours and masked.  (With
// pieces of one element instead: 290 us at 32768 x 1409 bf16.)  For the rows
// that norm_fwd_shift_kernel is not for.
//
// Q8: a block's 128 columns are 16 words of 8 bf16, or 32 of 4 fp32, and lie in
// as many neighbouring lanes, whose largest magnitude the shuffles find.
template <typename T, int TPR, int NV, bool SHIFT, bool RMS, bool Q8>
__global__ void __launch_bounds__(norm_threads<TPR>()) norm_fwd_kernel(const T* x, const T* res,
                                                                        const float* __restrict__ w,
                                                                        const float* __restrict__ b, int64_t L, int d,
                                                                        float eps, T* sum, T* y,
                                                                        float* __restrict__ mean_out,
                                                                        float* __restrict__ rstd_out, Rows8 q8) {
  static_assert(!Q8 || (RMS && !SHIFT), "8-bit rows: RMS norm, whole words");
  constexpr int VEC = 16 / (int)sizeof(T);
  using V = Vec<T, VEC>;
  __shared__ float red[2][32];
  const int lane = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t t = TPR == 32 ? (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (t >= L) return;  // a whole warp or a whole CTA
  const int shift = SHIFT ? (int)((t * d) % VEC) : 0;
  const int nvec = SHIFT ? (shift + d + VEC - 1) / VEC : d / VEC;
  const int64_t row = t * d - shift;  // element of the row's first word
  auto whole = [&](int c) {           // every element of word c is of the row
    return c * VEC >= shift && (c + 1) * VEC <= shift + d;
  };
  auto load = [&](const T* p, int c) {
    V v;
    if (!SHIFT || row + (int64_t)(c + 1) * VEC <= L * d) {
      v = *reinterpret_cast<const V*>(p + row + (int64_t)c * VEC);
    } else {  // the tensor ends inside this word
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (row + (int64_t)c * VEC + i < L * d) v.v[i] = p[row + (int64_t)c * VEC + i];
        else st_t(v.v[i], 0.f);
    }
    return v;
  };
  auto store = [&](T* p, int c, const float (&f)[VEC]) {
    if (!SHIFT || whole(c)) {
      *reinterpret_cast<V*>(p + row + (int64_t)c * VEC) = from_floats<T, VEC>(f);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if ((unsigned)(c * VEC + i - shift) < (unsigned)d) st_t(p[row + (int64_t)c * VEC + i], f[i]);
    }
  };
  float s[NV][VEC];
  V xv[NV], rv[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = lane + j * TPR;
    if (c < nvec) xv[j] = load(x, c);
  }
  if (res) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = lane + j * TPR;
      if (c < nvec) rv[j] = load(res, c);
    }
  }
  // elements outside the row are kept at zero
  auto clear_outside = [&](int j) {
    const int c = lane + j * TPR;
    if (SHIFT && c < nvec && !whole(c)) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if ((unsigned)(c * VEC + i - shift) >= (unsigned)d) s[j][i] = 0.f;
    }
  };
  float acc = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = lane + j * TPR;
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[j][i] = 0.f;
    if (c < nvec) {
      to_floats(xv[j], s[j]);
      if (res) {
        float r[VEC];
        to_floats(rv[j], r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[j][i] += r[i];
      }
    }
    clear_outside(j);
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc = RMS ? fmaf(s[j][i], s[j][i], acc) : acc + s[j][i];
  }
  if (sum) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = lane + j * TPR;
      if (c < nvec) store(sum, c, s[j]);
    }
  }
  const float inv_d = 1.f / (float)d;
  float mu = 0.f;
  if constexpr (!RMS) {
    mu = row_sum<TPR>(acc, red[0]) * inv_d;
    acc = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = lane + j * TPR < nvec;
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[j][i] -= mu;
      clear_outside(j);
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc = in ? fmaf(s[j][i], s[j][i], acc) : acc;
    }
  }
  const float ms = row_sum<TPR>(acc, red[1]) * inv_d + eps;
  float rstd = 1.f / sqrtf(ms), of_row = 1.f;
  if (RMS && out_of_range(ms)) {  // (the same for all of the row's threads)
    const Range r = into_range(ms);
    acc = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        acc = fmaf(s[j][i] * r.sum, s[j][i] * r.sum, acc);
        s[j][i] *= r.row;
      }
    rstd = rstd_in_range(r, row_sum<TPR>(acc, red[0]) * inv_d, eps);
    of_row = r.row;
  }
  if (lane == 0) {
    if (!RMS) mean_out[t] = mu;
    rstd_out[t] = rstd * of_row;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = lane + j * TPR;
    float o[VEC];
    if (c < nvec) {
      if constexpr (SHIFT) {
        const int k0 = c * VEC - shift, a0 = k0 & ~3;  // of the word's columns, and of w's and b's words around them
        if (VEC == 8 && whole(c) && a0 + 12 <= d) {
          // twelve elements in three 16-byte loads, of which the word's eight
          // begin at the row's k0 % 4 (lanes are 32 bytes apart: eight loads of
          // one element each would pass over the same lines eight times)
          float wb[2][12];
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            const float4 wv = reinterpret_cast<const float4*>(w + a0)[q];
            const float4 bv = b ? reinterpret_cast<const float4*>(b + a0)[q] : make_float4(0.f, 0.f, 0.f, 0.f);
            wb[0][4 * q] = wv.x; wb[0][4 * q + 1] = wv.y; wb[0][4 * q + 2] = wv.z; wb[0][4 * q + 3] = wv.w;
            wb[1][4 * q] = bv.x; wb[1][4 * q + 1] = bv.y; wb[1][4 * q + 2] = bv.z; wb[1][4 * q + 3] = bv.w;
          }
          const int r = k0 & 3;  // the same for the whole row
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float wv = r == 0 ? wb[0][i] : r == 1 ? wb[0][i + 1] : r == 2 ? wb[0][i + 2] : wb[0][i + 3];
            const float bv = r == 0 ? wb[1][i] : r == 1 ? wb[1][i + 1] : r == 2 ? wb[1][i + 2] : wb[1][i + 3];
            o[i] = fmaf(s[j][i] * rstd, wv, bv);
          }
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const int k = k0 + i;
            const bool in = (unsigned)k < (unsigned)d;
            o[i] = fmaf(s[j][i] * rstd, in ? w[k] : 0.f, in && b ? b[k] : 0.f);
          }
        }
      } else {
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q) {
          const float4 wv = reinterpret_cast<const float4*>(w)[c * (VEC / 4) + q];
          const float4 bv =
              b ? reinterpret_cast<const float4*>(b)[c * (VEC / 4) + q] : make_float4(0.f, 0.f, 0.f, 0.f);
          o[4 * q] = fmaf(s[j][4 * q] * rstd, wv.x, bv.x);
          o[4 * q + 1] = fmaf(s[j][4 * q + 1] * rstd, wv.y, bv.y);
          o[4 * q + 2] = fmaf(s[j][4 * q + 2] * rstd, wv.z, bv.z);
          o[4 * q + 3] = fmaf(s[j][4 * q + 3] * rstd, wv.w, bv.w);
        }
      }
      if (!Q8 || y) store(y, c, o);
    }
    if constexpr (Q8) {
      constexpr int LANES = kBlock8 / VEC;  // of a block
      uint32_t m = 0u;
      if (c < nvec) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = max(m, abs_bits(o[i]));
      }
#pragma unroll
      for (int k = LANES / 2; k > 0; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
      const Scale8 sc = scale8(m);
      if (c < nvec) {
        uint8_t* out = q8.q + t * d + (int64_t)c * VEC;
        if constexpr (VEC == 8) *reinterpret_cast<uint2*>(out) = make_uint2(e4m3x4(o, sc.inv), e4m3x4(o + 4, sc.inv));
        else *reinterpret_cast<uint32_t*>(out) = e4m3x4(o, sc.inv);
        if ((threadIdx.x & (LANES - 1)) == 0) q8.s[t * blocks8(d) + c / LANES] = sc.s;
      }
    }
  }
}

// rows wider than the register tiles: the row is read again for each of the
// three steps (the second and third time from L2).  Row t of `sum` may be
// row t of x or of the residual: it is written in the last step, by the
// thread that has just read the element for the last time.
template <typename T, bool RMS, bool Q8>
__global__ void __launch_bounds__(1024) norm_fwd_wide_kernel(const T* x, const T* res, const float* __restrict__ w,
                                                             const float* __restrict__ b, int64_t L, int d, float eps,
                                                             T* sum, T* y, float* __restrict__ mean_out,
                                                             float* __restrict__ rstd_out, Rows8 q8) {
  __shared__ float red[2][32];
  const int64_t o = (int64_t)blockIdx.x * d;
  auto at = [&](int c) { return ld_f32(x[o + c]) + (res ? ld_f32(res[o + c]) : 0.f); };
  float acc = 0.f, mu = 0.f;
  if constexpr (!RMS) {
    for (int c = threadIdx.x; c < d; c += 1024) acc += at(c);
    mu = row_sum<1024>(acc, red[0]) / (float)d;
    acc = 0.f;
  }
  for (int c = threadIdx.x; c < d; c += 1024) {
    const float v = at(c) - mu;
    acc = fmaf(v, v, acc);
  }
  const float ms = row_sum<1024>(acc, red[1]) / (float)d + eps;
  float rstd = 1.f / sqrtf(ms), of_row = 1.f;
  if (RMS && out_of_range(ms)) {
    const Range r = into_range(ms);
    acc = 0.f;
    for (int c = threadIdx.x; c < d; c += 1024) acc = fmaf(at(c) * r.sum, at(c) * r.sum, acc);
    rstd = rstd_in_range(r, row_sum<1024>(acc, red[0]) / (float)d, eps);
    of_row = r.row;
  }
  if constexpr (Q8) {  // a warp takes a block, a lane four neighbouring columns of it
    const int lane = threadIdx.x & 31;
    for (int blk = threadIdx.x >> 5; blk < blocks8(d); blk += 32) {
      const int c = blk * kBlock8 + 4 * lane;  // (d is a multiple of 16)
      float f[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t m = 0u;
      if (c < d) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = at(c + i);
          if (sum) st_t(sum[o + c + i], v);
          f[i] = v * of_row * rstd * w[c + i];
          if (y) st_t(y[o + c + i], f[i]);
          m = max(m, abs_bits(f[i]));
        }
      }
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
      const Scale8 sc = scale8(m);
      if (c < d) *reinterpret_cast<uint32_t*>(q8.q + o + c) = e4m3x4(f, sc.inv);
      if (lane == 0) q8.s[(int64_t)blockIdx.x * blocks8(d) + blk] = sc.s;
    }
  } else {
    for (int c = threadIdx.x; c < d; c += 1024) {
      const float v = at(c);
      if (sum) st_t(sum[o + c], v);
      st_t(y[o + c], fmaf((v - mu) * of_row * rstd, w[c], b ? b[c] : 0.f));
    }
  }
  if (threadIdx.x == 0) {
    if (!RMS) mean_out[blockIdx.x] = mu;
    rstd_out[blockIdx.x] = rstd * of_row;
  }
}

// ------------------------------------------------------------------ backward
// A persistent CTA walks over rows t = first, first + rows in flight, ...;
// a thread always holds the same columns, so the sums of dw and db over the
// CTA's rows stay in its registers.  The rows to come are copied ahead by
// cp.async into a ring in which every thread reads back only its own pieces
// (no barrier, no registers): 1024 threads x 192 bytes keep an SM's loads in
// flight while a row's two sums go through the CTA's one barrier.
// part[cta][0][c] and part[cta][1][c] are added up in a fixed order by
// norm_wgrad_kernel.
// the two sums of a warp, a in lanes 0-15 and b in lanes 16-31
__device__ __forceinline__ float warp_sum2(float a, float b) {
  const bool hi = threadIdx.x & 16;
  float v = (hi ? b : a) + __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// the first n of 16 bytes, the rest zeros (not read)
__device__ __forceinline__ void copy_part(void* dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(n)
               : "memory");
}
__device__ __forceinline__ void copy_ahead(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// Rows that do not start on 16 bytes, persistent: a CTA's (or a warp's) rows
// are a multiple of VEC apart, so that their words begin at the same `shift`
// before the row, and a thread keeps the w and b of its words' columns in
// registers.  The rows to come are copied ahead into a ring of each thread's
// own words.  Eight elements a thread; WARP: a row in a warp, four side by
// side; RES: with a residual.
// One CTA a row, which has to look its w and b up each time, against this, in
// bf16: 41261 x 1700 121 and 88 us, with residual 166 and 121 us; 32768 x 1409
// with residual 129 and 94 us; 131072 x 65 70 and 45 us.
template <typename T, bool RES>
constexpr int fwd_depth() {  // 192 KB of an SM's 1024 threads, at most six rows
  constexpr int room = 192 / (16 * (RES ? 2 : 1) * ((int)sizeof(T) / 2));
  return room < 6 ? room : 6;
}
template <typename T, bool RES>
constexpr size_t fwd_shift_smem(int threads) {
  return (size_t)fwd_depth<T, RES>() * (RES ? 2 : 1) * (sizeof(T) / 2) * 16 * threads;
}
template <typename T, bool WARP, bool RES, bool RMS>
__global__ void __launch_bounds__(WARP ? 32 * kNormWarps : 1024, WARP ? 8 : 1) norm_fwd_shift_kernel(
    const T* x, const T* res, const float* __restrict__ w, const float* __restrict__ b, int64_t L, int d, float eps,
    T* sum, T* y, float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  constexpr int VEC = 16 / (int)sizeof(T), NV = 8 / VEC, N = 8, ROWS = WARP ? kNormWarps : 1;
  constexpr int A = RES ? 2 : 1, D = fwd_depth<T, RES>();
  using V = Vec<T, VEC>;
  extern __shared__ __align__(16) uint8_t nsm[];
  uint4* ring = reinterpret_cast<uint4*>(nsm);  // [D][A][NV][threads]: x and, with RES, the residual
  __shared__ float red[2][32];
  const int tid = threadIdx.x, NT = WARP ? 32 * kNormWarps : (int)blockDim.x, TPR = WARP ? 32 : NT, lane = WARP ? (tid & 31) : tid;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  const int64_t first = (int64_t)blockIdx.x * ROWS + (WARP ? (tid >> 5) : 0);
  if (first >= L) return;  // a whole warp or a whole CTA
  const int shift = (int)((first * d) % VEC), nvec = (shift + d + VEC - 1) / VEC;
  const int64_t end = L * d;
  auto column = [&](int q) { return (lane + (q / VEC) * TPR) * VEC + q % VEC - shift; };  // of element q
  auto inside = [&](int q) { return (unsigned)column(q) < (unsigned)d; };
  float wv[N], bv[N];
  bool edge = false;  // a word is shared with a neighbouring row
#pragma unroll
  for (int q = 0; q < N; ++q) {
    wv[q] = inside(q) ? w[column(q)] : 0.f;
    bv[q] = inside(q) && b ? b[column(q)] : 0.f;
    edge = edge || (!inside(q) && lane + (q / VEC) * TPR < nvec);
  }
  int64_t o = first * d - shift + lane * VEC;  // the thread's first word in the row at work
  const int64_t stride = step * d;
  // pieces past the row's end stay zero
#pragma unroll
  for (int q = 0; q < D * A * NV; ++q) ring[q * NT + tid] = make_uint4(0u, 0u, 0u, 0u);
  int64_t ft = first, fo = o;  // the next row to copy
  auto fetch = [&](int at) {
    if (ft < L) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (lane + j * TPR < nvec) {
          const int64_t p = fo + j * TPR * VEC;
          uint4* dst = ring + (at * A * NV + j) * NT + tid;
          if (p + VEC > end) {  // the tensor ends inside this word
            const int n = (int)(end - p) * (int)sizeof(T);
            copy_part(dst, x + p, n);
            if (RES) copy_part(dst + NV * NT, res + p, n);
          } else {
            copy_ahead(dst, x + p);
            if (RES) copy_ahead(dst + NV * NT, res + p);
          }
        }
      }
    }
    ft += step;
    fo += stride;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto store = [&](T* p, const float (&f)[N]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float g[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) g[i] = f[j * VEC + i];
      if (edge) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (inside(j * VEC + i)) st_t(p[o + j * TPR * VEC + i], g[i]);
      } else if (lane + j * TPR < nvec) {
        *reinterpret_cast<V*>(p + o + j * TPR * VEC) = from_floats<T, VEC>(g);
      }
    }
  };
  const int warps = TPR / 32;
  auto row_sum = [&](float v, float* r) {
    v = warp_sum(v);
    if constexpr (!WARP) {
      if ((tid & 31) == 0) r[tid >> 5] = v;
      __syncthreads();
      v = warp_sum((tid & 31) < warps ? r[tid & 31] : 0.f);
    }
    return v;
  };
  const float inv_d = 1.f / (float)d;
#pragma unroll
  for (int i = 0; i < D; ++i) fetch(i);
  int slot = 0, turn = 0;
  for (int64_t t = first; t < L; t += step, o += stride) {
    float s[N];
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[VEC];
      const uint4* at = ring + (slot * A * NV + j) * NT + tid;
      const uint4 u = at[0];
      to_floats(*reinterpret_cast<const V*>(&u), f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[j * VEC + i] = f[i];
      if constexpr (RES) {
        const uint4 v = at[NV * NT];
        to_floats(*reinterpret_cast<const V*>(&v), f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[j * VEC + i] += f[i];
      }
    }
    fetch(slot);
    slot = slot == D - 1 ? 0 : slot + 1;
    // elements outside the row are kept at zero
    if (edge) {
#pragma unroll
      for (int q = 0; q < N; ++q) s[q] = inside(q) ? s[q] : 0.f;
    }
    if (sum) store(sum, s);
    float acc = 0.f;
    float mu = 0.f;
    if constexpr (!RMS) {
#pragma unroll
      for (int q = 0; q < N; ++q) acc += s[q];
      mu = row_sum(acc, red[0]) * inv_d;
      acc = 0.f;
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
      if constexpr (!RMS) {
        s[q] = lane + (q / VEC) * TPR < nvec ? s[q] - mu : 0.f;
        if (edge && !inside(q)) s[q] = 0.f;
      }
      acc = fmaf(s[q], s[q], acc);
    }
    // (RMS has one sum and one barrier a row: rows take the two places in turn, so that a place is written again only
    // behind the barrier that follows its readers)
    if (RMS) turn ^= 1;
    const float ms = row_sum(acc, red[RMS ? turn : 1]) * inv_d + eps;
    float rstd = 1.f / sqrtf(ms), of_row = 1.f;
    if (RMS && out_of_range(ms)) {
      const Range r = into_range(ms);
      acc = 0.f;
#pragma unroll
      for (int q = 0; q < N; ++q) {
        acc = fmaf(s[q] * r.sum, s[q] * r.sum, acc);
        s[q] *= r.row;
      }
      turn ^= 1;
      rstd = rstd_in_range(r, row_sum(acc, red[turn]) * inv_d, eps);
      of_row = r.row;
    }
    if (lane == 0) {
      if (!RMS) mean_out[t] = mu;
      rstd_out[t] = rstd * of_row;
    }
#pragma unroll
    for (int q = 0; q < N; ++q) s[q] = fmaf(s[q] * rstd, wv[q], bv[q]);
    store(y, s);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

constexpr int kBwdDepth = 4;
// sums of a CTA's rows for each column: dw and db, or dw alone
template <bool RMS>
__host__ __device__ constexpr int wgrad_sums() {
  return RMS ? 1 : 2;
}
// The backward's shapes.  WARP: four rows per CTA, a warp each; else a row per
// CTA, of as many threads as its words need.  BUDGET: threads of an SM, which
// set the registers a thread may have and the ring's depth (two rows at work,
// the others on their way; with two, a row is fetched as soon as its place is
// free).  RES: with a gradient dsum besides dy, a third array.
template <typename T, int NV, int BUDGET, bool RES>
constexpr int bwd_depth() {
  constexpr int row = (RES ? 3 : 2) * 16 * NV;  // bytes of a row a thread holds
  constexpr int room = 200 * 1024 / BUDGET / row;
  return room >= kBwdDepth ? kBwdDepth : room < 2 ? 2 : room;
}
template <typename T, int NV, int BUDGET, bool RES>
constexpr size_t bwd_smem(int threads) {
  return (size_t)bwd_depth<T, NV, BUDGET, RES>() * (RES ? 3 : 2) * 16 * NV * threads;
}

// Rows that do not start on 16 bytes (SHIFT): the 16-byte words of a dense
// matrix lie at the same places of every VEC-th row, and a CTA's rows are a
// multiple of VEC apart.  So a thread still holds whole words, whose columns
// begin `shift` before the row, the same for all of the CTA's rows; the first
// and the last word of a row are shared with its neighbours and masked.
// (Measured at 8191 x 1409 fp32 and 32768 x 1409 bf16 before: 41 and 248 us
// with pieces of one element, 50 and 161 us with rows copied whole and read
// by element.)
// THREADS: the CTA's threads where they are known here, 0 where not (the ring's
// and the sums' places then cost instructions: 182 us against 194 us at
// 32768 x 4096 bf16, 156 against 191 at 16384 x 6144).
template <typename T, int NV, bool WARP, int BUDGET, int THREADS, bool SHIFT, bool RES, bool RMS>
__global__ void __launch_bounds__(WARP ? 32 * kNormWarps : BUDGET, WARP ? 4 : 1) norm_bwd_kernel(
    const T* dy, const T* s, const float* __restrict__ mean, const float* __restrict__ rstd,
    const float* __restrict__ w, const T* dsum, int64_t L, int d, T* dx, float* __restrict__ part) {
  constexpr int VEC = 16 / (int)sizeof(T), ROWS = WARP ? kNormWarps : 1, A = RES ? 3 : 2,
                D = bwd_depth<T, NV, BUDGET, RES>();
  // D rows at a time, for constant places in the ring (32768 x 4096 bf16: 181
  // against 185 us, 155 against 169 without dsum); two words a thread: slower
  constexpr bool UNROLL = sizeof(T) == 2 && NV == 1;
  using V = Vec<T, VEC>;
  extern __shared__ __align__(16) uint8_t nsm[];
  uint4* ring = reinterpret_cast<uint4*>(nsm);  // [D][A][NV][threads]: dy, s and, with RES, dsum
  __shared__ float red[2][2][32];  // [buffer][sum][warp]
  const int tid = threadIdx.x, NT = WARP ? 32 * kNormWarps : THREADS ? THREADS : (int)blockDim.x, TPR = WARP ? 32 : NT;
  const int lane = WARP ? (tid & 31) : tid;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // norm_wgrad_kernel sets itself up meanwhile
  const int64_t step = (int64_t)gridDim.x * ROWS;
  const int64_t first = (int64_t)blockIdx.x * ROWS + (WARP ? (tid >> 5) : 0);
  // a word's columns: word c of a row holds columns c VEC - shift, ...
  const int shift = SHIFT ? (int)((first * d) % VEC) : 0;
  const int nvec = SHIFT ? (shift + d + VEC - 1) / VEC : d / VEC;
  const float inv_d = 1.f / (float)d;
  // sums and weights of this thread's columns, in pairs of elements
  constexpr int P = NV * VEC / 2;
  auto column = [&](int q) { return (lane + (q / VEC) * TPR) * VEC + q % VEC - shift; };  // of element q
  auto inside = [&](int c) { return SHIFT ? (unsigned)c < (unsigned)d : c < d; };
  float2 aw[P], ab[P], wv[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    aw[i] = ab[i] = both(0.f);
    wv[i].x = inside(column(2 * i)) ? w[column(2 * i)] : 0.f;
    wv[i].y = inside(column(2 * i + 1)) ? w[column(2 * i + 1)] : 0.f;
  }
  // the elements of this thread's words that belong to the row, as bits; and
  // whether one of the words is shared with a neighbouring row
  uint32_t keep[NV][4];
  bool edge = false;
  if constexpr (SHIFT) {
#pragma unroll
    for (int q = 0; q < NV * VEC; ++q) {
      constexpr int PER = 4 / (int)sizeof(T);  // elements of 32 bits
      const int j = q / VEC, i = q % VEC / PER;
      if (q % PER == 0) keep[j][i] = 0u;
      if (inside(column(q))) keep[j][i] |= PER == 1 ? 0xFFFFFFFFu : 0xFFFFu << (16 * (q % PER));
      else edge = edge || lane + j * TPR < nvec;
    }
  }
  // array a of ring slot `at`, as pairs; clean: the neighbours' elements as zeros
  auto read = [&](int at, int a, float2 (&v)[P], bool clean) {
    float f[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint4 u = ring[((at * A + a) * NV + j) * NT + tid];
      if (SHIFT && clean) {
        u.x &= keep[j][0];
        u.y &= keep[j][1];
        u.z &= keep[j][2];
        u.w &= keep[j][3];
      }
      to_floats(*reinterpret_cast<const V*>(&u), f[j]);
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
      v[i] = make_float2(f[2 * i / VEC][2 * i % VEC], f[(2 * i + 1) / VEC][(2 * i + 1) % VEC]);
  };
  // (the threads' words lie side by side: a part of the ring of its own for each
  // thread, whose places would be constants, measured 280 against 184 us)
  // pieces past the row's end stay zero
#pragma unroll
  for (int q = 0; q < D * A * NV; ++q) ring[q * NT + tid] = make_uint4(0u, 0u, 0u, 0u);
  // the first element of this thread's word in the next row to fetch (SHIFT),
  // kept from row to row; without SHIFT the place is formed anew for each row
  // (a register pair less: 187 against 193 us at 32768 x 4096 bf16)
  int64_t fo = first * d - shift + lane * VEC;
  const int64_t stride = step * d;
  auto fetch = [&](int64_t t, int at) {
    if (t < L) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (lane + j * TPR < nvec) {
          const int64_t o = SHIFT ? fo + j * TPR * VEC : t * d + (lane + j * TPR) * VEC;
          uint4* dst = ring + (at * A * NV + j) * NT + tid;
          if (SHIFT && o + VEC > L * d) {  // the tensor ends inside this word
            const int n = (int)(L * d - o) * (int)sizeof(T);
            copy_part(dst, dy + o, n);
            copy_part(dst + NV * NT, s + o, n);
            if (RES) copy_part(dst + 2 * NV * NT, dsum + o, n);
          } else {
            copy_ahead(dst, dy + o);
            copy_ahead(dst + NV * NT, s + o);
            if (RES) copy_ahead(dst + 2 * NV * NT, dsum + o);
          }
        }
      }
    }
    if (SHIFT) fo += stride;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // A row's two sums meet at the CTA's barrier.  They are formed one row
  // ahead: in one iteration the threads sum up row i + 1 and finish row i,
  // whose sums passed the barrier of the iteration before, so that neither
  // the barrier nor the shuffles stand in a row's way (all in one row's
  // order measured 187 us at 32768 x 4096 bf16, and 206 us with the
  // shuffles below in place of a read of all warps' sums).
#pragma unroll
  for (int i = 0; i < D; ++i) fetch(first + i * step, i);
  float mu = 0.f, rs = 0.f, nmu = 0.f, nrs = 0.f;  // of the row to sum up, and of the one after
  if (first < L) {
    if (!RMS) mu = mean[first];
    rs = rstd[first];
  }
  if (first + step < L) {
    if (!RMS) nmu = mean[first + step];
    nrs = rstd[first + step];
  }
  float2 mine = make_float2(0.f, 0.f);  // a warp's row: the sums of the row to finish
  // the sums of row t, in ring slot `at`, into red[buf] (or mine)
  auto sum_up = [&](int at, int buf) {
    const float2 rs2 = both(rs), nmu2 = both(-mu);
    float2 sg = both(0.f), sgx = both(0.f);
    float2 dv[P], sv[P];
    read(at, 0, dv, true);
    read(at, 1, sv, true);
    // a piece past the row's end: dy = 0 and w = 0 keep it out of the sums
#pragma unroll
    for (int i = 0; i < P; ++i) {
      // (s - mu first, as the forward does: s rs - mu rs loses |mu| rs half steps of
      // fp32; 178.6 against 178.3 us at 32768 x 4096 bf16, 49.4 against 47.5 at
      // 131072 x 65)
      const float2 xh = __fmul2_rn(RMS ? sv[i] : __fadd2_rn(sv[i], nmu2), rs2), g = __fmul2_rn(dv[i], wv[i]);
      aw[i] = __ffma2_rn(dv[i], xh, aw[i]);
      if constexpr (!RMS) {
        ab[i] = __fadd2_rn(ab[i], dv[i]);
        sg = __fadd2_rn(sg, g);
      }
      sgx = __ffma2_rn(g, xh, sgx);
    }
    if constexpr (RMS) {  // the one sum
      const float v = warp_sum(sgx.x + sgx.y);
      if constexpr (WARP) mine = make_float2(0.f, v);
      else if ((tid & 31) == 0) red[buf][1][tid >> 5] = v;
      return;
    }
    const float v = warp_sum2(sg.x + sg.y, sgx.x + sgx.y);
    if constexpr (!WARP) {
      if ((tid & 15) == 0) red[buf][(tid >> 4) & 1][tid >> 5] = v;
    } else {
      mine = make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
    }
  };
  // dx of the next row, in ring slot `at`, from its sums
  T* kept = dx + first * d - shift + lane * VEC;  // SHIFT: of the next row to finish
  auto finish = [&](int64_t t, int at, int buf, float rs, float mu, float2 sums) {
    if constexpr (!WARP && RMS) {
      const int nw = NT / 32, i = tid & 31;
      sums = make_float2(0.f, warp_sum(i < nw ? red[buf][1][i] : 0.f));
    } else if constexpr (!WARP) {
      // lanes 0-15 add up the first sum over the warps, lanes 16-31 the second
      const float* r = red[buf][(tid >> 4) & 1];
      float v;
      if constexpr (THREADS != 0 && (THREADS & (THREADS - 1)) == 0) {
        constexpr int W = THREADS / 32, H = W < 16 ? W : 16;
        v = r[tid & (H - 1)];
        if constexpr (W == 32) v += r[16 + (tid & 15)];
#pragma unroll
        for (int o = H / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      } else {
        const int i = tid & 15, nw = NT / 32;
        v = i < nw ? r[i] : 0.f;
        if (i + 16 < nw) v += r[i + 16];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      }
      sums = make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
    }
    // ds = rs (dy w - mg - (s - mu) rs mgx) + r
    const float mg = sums.x * inv_d, mgx = sums.y * inv_d;
    const float2 rs2 = both(rs), nmu2 = both(-mu), c0 = both(-mg), c1 = both(-rs * mgx);
    float2 dv[P], sv[P], rv[P];
    // (a neighbour's elements give results that are not stored)
    read(at, 0, dv, false);
    read(at, 1, sv, false);
    if constexpr (RES) read(at, 2, rv, false);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 u = RMS ? __ffma2_rn(sv[i], c1, __fmul2_rn(dv[i], wv[i]))
                           : __ffma2_rn(__fadd2_rn(sv[i], nmu2), c1, __ffma2_rn(dv[i], wv[i], c0));
      rv[i] = RES ? __ffma2_rn(rs2, u, rv[i]) : __fmul2_rn(rs2, u);
    }
    T* out = SHIFT ? kept : dx + t * d + lane * VEC;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = lane + j * TPR;
      float f[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = (j * VEC + i) % 2 ? rv[(j * VEC + i) / 2].y : rv[(j * VEC + i) / 2].x;
      if (SHIFT && edge) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (inside(c * VEC + i - shift)) st_t(out[j * TPR * VEC + i], f[i]);
      } else if (c < nvec) {
        *reinterpret_cast<V*>(out + j * TPR * VEC) = from_floats<T, VEC>(f);
      }
    }
    if (SHIFT) kept += stride;
  };
  asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
  if (first < L) sum_up(0, 0);  // (whole warps, and whole CTAs where a CTA holds a row)
  if constexpr (!WARP) __syncthreads();
  int buf = 0;
  int64_t t = first;
  auto row = [&](int slot, int next) {
    const float rs0 = rs, mu0 = mu;
    const float2 sums = mine;
    mu = nmu;
    rs = nrs;
    if (t + 2 * step < L) {
      if (!RMS) nmu = mean[t + 2 * step];
      nrs = rstd[t + 2 * step];
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory");
    if (t + step < L) sum_up(next, buf ^ 1);
    finish(t, slot, buf, rs0, mu0, sums);
    fetch(t + (int64_t)D * step, slot);
    if constexpr (!WARP) __syncthreads();
    t += step;
    buf ^= 1;
  };
  if constexpr (UNROLL) {
    while (t < L) {
#pragma unroll
      for (int slot = 0; slot < D; ++slot) {
        if (t >= L) break;
        row(slot, (slot + 1) % D);
      }
    }
  } else {
    for (int slot = 0; t < L;) {
      const int next = slot == D - 1 ? 0 : slot + 1;
      row(slot, next);
      slot = next;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  float* pw = part + (int64_t)blockIdx.x * wgrad_sums<RMS>() * d;
  if constexpr (!WARP) {
#pragma unroll
    for (int q = 0; q < 2 * P; ++q) {
      const int c = column(q);
      if (inside(c)) {
        pw[c] = q % 2 ? aw[q / 2].y : aw[q / 2].x;
        if (!RMS) pw[d + c] = q % 2 ? ab[q / 2].y : ab[q / 2].x;
      }
    }
  } else {
    // the CTA's warps hold rows of their own (and, with SHIFT, the columns
    // in places of their own): one warp after the other adds its sums
    __shared__ float csum[2][32 * NV * VEC];
    for (int r = 0; r < kNormWarps; ++r) {
      if ((tid >> 5) == r) {
#pragma unroll
        for (int q = 0; q < 2 * P; ++q) {
          const int c = column(q);
          if (inside(c)) {
            csum[0][c] = (r ? csum[0][c] : 0.f) + (q % 2 ? aw[q / 2].y : aw[q / 2].x);
            if (!RMS) csum[1][c] = (r ? csum[1][c] : 0.f) + (q % 2 ? ab[q / 2].y : ab[q / 2].x);
          }
        }
      }
      __syncthreads();
    }
    for (int c = tid; c < d; c += NT) {
      pw[c] = csum[0][c];
      if (!RMS) pw[d + c] = csum[1][c];
    }
  }
}

// dw and db from the CTAs' partial sums, in the order of the CTAs: 32 columns
// per block, warp i of its 32 takes partials i, i + 32, ...
constexpr int kWgradWarps = 32;
template <bool RMS>
__global__ void __launch_bounds__(32 * kWgradWarps) norm_wgrad_kernel(const float* part, int G, int d,
                                                         float* __restrict__ dw, float* __restrict__ db) {
  const int width = wgrad_sums<RMS>() * d;
  __shared__ float acc[kWgradWarps][32];
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;  // column of the row [dw | db] (RMS: dw alone)
  float a = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c < width) {
    // 16 in flight at a time, the last ones too
    for (int g0 = wp; g0 < G; g0 += 16 * kWgradWarps) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int g = g0 + i * kWgradWarps;
        v[i] = g < G ? part[(int64_t)g * width + c] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) a += v[i];
    }
  }
  acc[wp][lane] = a;
  __syncthreads();
  if (wp == 0 && c < width) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < kWgradWarps; ++i) a += acc[i][lane];
    if (c < d) dw[c] = a;
    else if (!RMS && db) db[c - d] = a;
  }
}

// rows wider than the register tiles
template <typename T, bool RMS>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(const T* dy, const T* s, const float* __restrict__ mean,
                                                             const float* __restrict__ rstd,
                                                             const float* __restrict__ w, const T* dsum, int d, T* dx) {
  __shared__ float red[2][32];
  const int64_t t = blockIdx.x, o = t * d;
  const float mu = RMS ? 0.f : mean[t], rs = rstd[t];
  float sg = 0.f, sgx = 0.f;
  for (int c = threadIdx.x; c < d; c += 1024) {
    const float g = ld_f32(dy[o + c]) * w[c];
    sg += g;
    sgx = fmaf(g, (ld_f32(s[o + c]) - mu) * rs, sgx);
  }
  const float mg = RMS ? 0.f : row_sum<1024>(sg, red[0]) / (float)d, mgx = row_sum<1024>(sgx, red[1]) / (float)d;
  for (int c = threadIdx.x; c < d; c += 1024) {
    const float g = ld_f32(dy[o + c]) * w[c], xh = (ld_f32(s[o + c]) - mu) * rs;
    st_t(dx[o + c], fmaf(rs, g - mg - xh * mgx, dsum ? ld_f32(dsum[o + c]) : 0.f));
  }
}

// partial dw and db of every `step`-th row, a thread per column
template <typename T, bool RMS>
__global__ void __launch_bounds__(256) norm_wide_wgrad_kernel(const T* dy, const T* s, const float* __restrict__ mean,
                                                              const float* __restrict__ rstd, int64_t L, int d,
                                                              float* __restrict__ part) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  float aw = 0.f, ab = 0.f;
#pragma unroll 4
  for (int64_t t = blockIdx.y; t < L; t += gridDim.y) {
    const float dv = ld_f32(dy[t * d + c]);
    aw = fmaf(dv, (ld_f32(s[t * d + c]) - (RMS ? 0.f : mean[t])) * rstd[t], aw);
    ab += dv;
  }
  part[(int64_t)blockIdx.y * wgrad_sums<RMS>() * d + c] = aw;
  if (!RMS) part[(int64_t)blockIdx.y * 2 * d + d + c] = ab;
}

constexpr int kWideSplits = 32;
constexpr int kMaxTileWords = 4096;  // widest register tile of the forward: 1024 threads of 4 words

// The backward's shape for a row of d elements: 8 elements a thread (their
// two sums and weights in registers), 16 in a lane of a warp that holds a
// short row, and where rows of just over half an SM's threads would leave the
// other half idle.  Wider rows than any: words = 0.
struct BwdShape {
  int words, nv, threads, budget, ctas;  // ctas: the resident ones, or as many as there are rows
  bool warp, shift;
};
BwdShape bwd_shape(const moeblaze_shape& s) {
  BwdShape b = {};
  const bool half = s.dtype == MOEBLAZE_BF16;
  const int vec = half ? 8 : 4;
  b.shift = s.d % vec != 0;
  const int words = b.shift ? (s.d + 2 * vec - 2) / vec : s.d / vec;
  b.words = words;
  auto wide = [&](int nv, int budget) {
    b.nv = nv;
    b.budget = budget;
    b.threads = ((words + nv - 1) / nv + 31) / 32 * 32;
  };
  if (words <= (half ? 64 : 128)) {
    b.warp = true;
    b.nv = words <= (half ? 32 : 64) ? (half ? 1 : 2) : (half ? 2 : 4);
    b.threads = 32 * kNormWarps;
    b.budget = 512;
  } else if (half) {
    if (words <= 512 || (words > 640 && words <= 1024)) {
      // the next of the thread counts that bwd_shaped has: as many CTAs an SM
      // as with whole warps only
      wide(1, 1024);
      for (int t : {96, 128, 160, 192, 224, 256, 320, 384, 448, 512, 768, 896, 1024})
        if (t >= b.threads) {
          b.threads = t;
          break;
        }
    } else if (words <= 640) wide(2, 640);
    else if (words <= 2048) wide(2, 1024);
    else b.words = 0;
  } else {
    if (words <= 1280) wide(2, 640);
    else if (words <= 2048) wide(2, 1024);
    else b.words = 0;
  }
  if (b.words == 0) return b;
  const int rows = b.warp ? kNormWarps : 1;
  int64_t g = (int64_t)(b.warp ? 4 : b.budget / b.threads) * sm_count();
  if (g > 8) g -= g % 8;  // a CTA's rows are a multiple of 8 apart (shift), unless each has one row
  const int64_t need = (s.L + rows - 1) / rows;
  b.ctas = (int)(g < need ? g : need);
  return b;
}

template <bool RMS>
moeblaze_status launch_wgrad(const float* part, int G, int d, float* dw, float* db, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((wgrad_sums<RMS>() * (int64_t)d + 31) / 32));
  cfg.blockDim = dim3(32 * kWgradWarps);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MB_CUDA(cudaLaunchKernelEx(&cfg, norm_wgrad_kernel<RMS>, part, G, d, dw, db));
  return MOEBLAZE_OK;
}

struct FwdArgs {
  const void *x, *res;
  const float *w, *b;
  float eps;
  void *sum, *y;
  float *mean, *rstd;
  Rows8 q8;  // RMS norm: q null for none
};
struct BwdArgs {
  const void *dy, *sum;
  const float *mean, *rstd, *w;
  const void* dsum;
  void* dx;
  float *dw, *db, *part;
};

template <typename T, int TPR, int NV, bool SHIFT, bool RMS, bool Q8>
moeblaze_status fwd_tile(const moeblaze_shape& s, const FwdArgs& a, cudaStream_t st) {
  const int rows = TPR == 32 ? kNormWarps : 1;
  norm_fwd_kernel<T, TPR, NV, SHIFT, RMS, Q8><<<(unsigned)((s.L + rows - 1) / rows), norm_threads<TPR>(), 0, st>>>(
      (const T*)a.x, (const T*)a.res, a.w, a.b, s.L, s.d, a.eps, (T*)a.sum, (T*)a.y, a.mean, a.rstd, a.q8);
  MB_CUDA(cudaGetLastError());
  count_launch();
  return MOEBLAZE_OK;
}

template <typename T, int NV, bool WARP, int BUDGET, int THREADS, bool SHIFT, bool RES, bool RMS>
moeblaze_status bwd_tile(const moeblaze_shape& s, const BwdShape& b, const BwdArgs& a, cudaStream_t st) {
  auto kern = norm_bwd_kernel<T, NV, WARP, BUDGET, THREADS, SHIFT, RES, RMS>;
  const size_t sm = bwd_smem<T, NV, BUDGET, RES>(b.threads);
  MB_CUDA(smem_limit(kern, bwd_smem<T, NV, BUDGET, RES>(WARP ? 32 * kNormWarps : THREADS ? THREADS : BUDGET)));
  kern<<<(unsigned)b.ctas, b.threads, sm, st>>>((const T*)a.dy, (const T*)a.sum, a.mean, a.rstd, a.w, (const T*)a.dsum,
                                                s.L, s.d, (T*)a.dx, a.part);
  MB_CUDA(cudaGetLastError());
  count_launch(2);
  return launch_wgrad<RMS>(a.part, b.ctas, s.d, a.dw, a.db, st);
}

// the forward's register tile of a row of n words
template <typename T, bool SHIFT, bool RMS, bool Q8>
moeblaze_status fwd_words(const moeblaze_shape& s, int n, const FwdArgs& a, cudaStream_t st) {
#define MB_CALL(TPR, NV) fwd_tile<T, TPR, NV, SHIFT, RMS, Q8>(s, a, st)
  constexpr bool half = sizeof(T) == 2;
  if constexpr (!SHIFT) {
    if (n <= 32) return MB_CALL(32, 1);
    if (n <= 64) return MB_CALL(32, 2);
  }
  if constexpr (!SHIFT || !half) {  // see fwd_t
    if (n <= 128) return MB_CALL(32, 4);
    if (n <= 256) return MB_CALL(128, 2);
    if (n <= 384) return MB_CALL(128, 3);
    // (without a residual twice the words a thread, for as many loads in flight:
    // 105 us instead of 117 at 32768 x 4096 bf16)
    if (n <= 512) return a.res ? MB_CALL(256, 2) : MB_CALL(128, 4);
    if (n <= 768) return MB_CALL(256, 3);
    if (n <= 1024) return MB_CALL(512, 2);
  }
  if constexpr (!SHIFT || half)
    if (n <= 2048) return MB_CALL(1024, 2);
  return MB_CALL(1024, 4);
#undef MB_CALL
}

template <typename T, bool SHIFT, bool RES, bool RMS>
moeblaze_status bwd_shaped(const moeblaze_shape& s, const BwdShape& b, const BwdArgs& a, cudaStream_t st) {
  constexpr bool half = sizeof(T) == 2;
#define MB_CALL(NV, WARP, BUDGET, THREADS) bwd_tile<T, NV, WARP, BUDGET, THREADS, SHIFT, RES, RMS>(s, b, a, st)
  if (b.warp)
    return b.nv == (half ? 1 : 2) ? MB_CALL((half ? 1 : 2), true, 512, 0) : MB_CALL((half ? 2 : 4), true, 512, 0);
  if constexpr (half) {
    if (b.nv == 1) {
      switch (b.threads) {
        case 96: return MB_CALL(1, false, 1024, 96);
        case 128: return MB_CALL(1, false, 1024, 128);
        case 160: return MB_CALL(1, false, 1024, 160);
        case 192: return MB_CALL(1, false, 1024, 192);
        case 224: return MB_CALL(1, false, 1024, 224);
        case 256: return MB_CALL(1, false, 1024, 256);
        case 320: return MB_CALL(1, false, 1024, 320);
        case 384: return MB_CALL(1, false, 1024, 384);
        case 448: return MB_CALL(1, false, 1024, 448);
        case 512: return MB_CALL(1, false, 1024, 512);
        case 768: return MB_CALL(1, false, 1024, 768);
        case 896: return MB_CALL(1, false, 1024, 896);
      }
      return MB_CALL(1, false, 1024, 1024);
    }
  }
  return b.budget == 640 ? MB_CALL(2, false, 640, 0) : MB_CALL(2, false, 1024, 0);
#undef MB_CALL
}

// rows that do not start on 16 bytes, of up to 8192 elements
template <typename T, bool RMS>
moeblaze_status fwd_shift(const moeblaze_shape& s, int words, const FwdArgs& a, cudaStream_t st) {
  constexpr int nv = (int)sizeof(T) / 2;  // words of a thread: 8 elements
  const int threads = ((words + nv - 1) / nv + 31) / 32 * 32;
  const bool warp = threads == 32, res = a.res != nullptr;
  const int64_t need = warp ? (s.L + kNormWarps - 1) / kNormWarps : s.L;
  // (two CTAs of 545 to 576 threads still have their registers and rings)
  int64_t g = (int64_t)(warp ? 8 : threads > 512 && threads <= 576 ? 2 : 1024 / threads) * sm_count();
  g -= g % 8;  // a CTA's rows are a multiple of 8 apart (shift), unless each has one row
  if (g > need) g = need;
  auto kern = warp ? (res ? norm_fwd_shift_kernel<T, true, true, RMS> : norm_fwd_shift_kernel<T, true, false, RMS>)
                   : (res ? norm_fwd_shift_kernel<T, false, true, RMS> : norm_fwd_shift_kernel<T, false, false, RMS>);
  const int nt = warp ? 32 * kNormWarps : threads;
  const size_t sm = res ? fwd_shift_smem<T, true>(nt) : fwd_shift_smem<T, false>(nt);
  const int most = warp ? nt : 1024;
  MB_CUDA(smem_limit(kern, res ? fwd_shift_smem<T, true>(most) : fwd_shift_smem<T, false>(most)));
  kern<<<(unsigned)g, nt, sm, st>>>((const T*)a.x, (const T*)a.res, a.w, a.b, s.L, s.d, a.eps, (T*)a.sum, (T*)a.y,
                                    a.mean, a.rstd);
  MB_CUDA(cudaGetLastError());
  count_launch();
  return MOEBLAZE_OK;
}

template <typename T, bool RMS>
moeblaze_status fwd_t(const moeblaze_shape& s, const FwdArgs& a, cudaStream_t st) {
  constexpr int vec = 16 / (int)sizeof(T);
  const bool shift = s.d % vec != 0;
  const int words = shift ? (s.d + 2 * vec - 2) / vec : s.d / vec;
  if (words > kMaxTileWords) {
    auto kern = norm_fwd_wide_kernel<T, RMS, false>;
    if constexpr (RMS)
      if (a.q8.q) kern = norm_fwd_wide_kernel<T, RMS, true>;
    kern<<<(unsigned)s.L, 1024, 0, st>>>((const T*)a.x, (const T*)a.res, a.w, a.b, s.L, s.d, a.eps, (T*)a.sum, (T*)a.y,
                                         a.mean, a.rstd, a.q8);
    MB_CUDA(cudaGetLastError());
    count_launch();
    return MOEBLAZE_OK;
  }
  if constexpr (RMS)
    if (a.q8.q) return fwd_words<T, false, true, true>(s, words, a, st);  // (d is a multiple of 16)
  // fp32 rows of 65 to 1024 words are as fast or faster with a CTA a row
  // (20000 x 1001 with residual: 55 against 68 us; 8000 x 5001: 137 against 129)
  constexpr bool half = sizeof(T) == 2;
  if (shift && (half ? words <= 1024 : words <= 64 || (words > 1024 && words <= 2048)))
    return fwd_shift<T, RMS>(s, words, a, st);
  return shift ? fwd_words<T, true, RMS, false>(s, words, a, st) : fwd_words<T, false, RMS, false>(s, words, a, st);
}

template <typename T, bool RMS>
moeblaze_status bwd_t(const moeblaze_shape& s, const BwdArgs& a, cudaStream_t st) {
  const BwdShape b = bwd_shape(s);
  if (b.words == 0) {
    norm_bwd_wide_kernel<T, RMS><<<(unsigned)s.L, 1024, 0, st>>>((const T*)a.dy, (const T*)a.sum, a.mean, a.rstd, a.w,
                                                                 (const T*)a.dsum, s.d, (T*)a.dx);
    MB_CUDA(cudaGetLastError());
    const int64_t G = s.L < kWideSplits ? s.L : kWideSplits;
    norm_wide_wgrad_kernel<T, RMS><<<dim3((unsigned)((s.d + 255) / 256), (unsigned)G), 256, 0, st>>>(
        (const T*)a.dy, (const T*)a.sum, a.mean, a.rstd, s.L, s.d, a.part);
    MB_CUDA(cudaGetLastError());
    count_launch(3);
    return launch_wgrad<RMS>(a.part, (int)G, s.d, a.dw, a.db, st);
  }
  auto run = b.shift ? (a.dsum ? bwd_shaped<T, true, true, RMS> : bwd_shaped<T, true, false, RMS>)
                     : (a.dsum ? bwd_shaped<T, false, true, RMS> : bwd_shaped<T, false, false, RMS>);
  return run(s, b, a, st);
}

template <bool RMS>
moeblaze_status norm_forward(const moeblaze_shape& s, const FwdArgs& a, cudaStream_t st) {
  if (s.L == 0) return MOEBLAZE_OK;
  return s.dtype == MOEBLAZE_BF16 ? fwd_t<__nv_bfloat16, RMS>(s, a, st) : fwd_t<float, RMS>(s, a, st);
}

template <bool RMS>
moeblaze_status norm_backward(const moeblaze_shape& s, const BwdArgs& a, cudaStream_t st) {
  if (s.L == 0) {
    MB_CUDA(cudaMemsetAsync(a.dw, 0, sizeof(float) * s.d, st));
    if (a.db) MB_CUDA(cudaMemsetAsync(a.db, 0, sizeof(float) * s.d, st));
    return MOEBLAZE_OK;
  }
  return s.dtype == MOEBLAZE_BF16 ? bwd_t<__nv_bfloat16, RMS>(s, a, st) : bwd_t<float, RMS>(s, a, st);
}

template <bool RMS>
size_t norm_scratch(const moeblaze_shape& s) {
  if (s.L == 0) return 0;
  const BwdShape b = bwd_shape(s);
  const int64_t G = b.words == 0 ? (s.L < kWideSplits ? s.L : kWideSplits) : b.ctas;
  return (size_t)G * wgrad_sums<RMS>() * s.d * sizeof(float);
}

}  // namespace
}  // namespace moeblaze
