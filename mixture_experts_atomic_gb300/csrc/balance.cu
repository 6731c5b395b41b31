// The router's auxiliary losses on its logits, the tokens per expert, and the
// gradient of the logits.
//
//   a token is active when valid (if given) is nonzero and one of its logits
//   is above -inf; N = active tokens
//   lse_t = log sum_e exp(l_te),  p_te = exp(l_te - lse_t)
//   count_e = slots of active tokens that name expert e,  f_e = count_e/(N K)
//   P_e = sum_t p_te / N
//   balance = E sum_e f_e P_e        z = sum_t lse_t^2 / N
//
//   dl_te = a E/N p_te (f_e - sum_j f_j p_tj) + 2 b/N lse_t p_te
//           (a, b the gradients of the two losses; the counts are piecewise
//           constant) and, with the gates' gradients, on a token's chosen
//           experts + g_k (dg_k - sum_j g_j dg_j)
//   rows of tokens that are not active are zero.
//
// f_e - sum_j f_j p_tj cancels when the load is even; both sides are taken
// relative to the mean load (sum_j p_tj = 1 leaves the difference as it is).
//
// A token's row of logits lies in TE lanes of a warp, EPT vectors of VEC
// experts each; P_e is summed in a lane's registers over the CTA's tokens,
// then over the warps and (balance_losses_kernel, in double) over the CTAs,
// always in the same order: repeatable to the bit.
#include "common.cuh"

namespace moeblaze {
namespace {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;

// floats of one CTA's partial sums: P[E], z, counts[E] (int), active (int)
__host__ __device__ inline int bal_cols(int E) { return 2 * E + 2; }

template <int VEC>
struct alignas(4 * VEC) FVec {
  float v[VEC];
};

// reductions over the TE lanes (consecutive, TE a power of two) of a token
template <int TE>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = TE / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int TE>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = TE / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int VEC, int TE, int EPT>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int te, bool on, float (&l)[EPT][VEC]) {
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const int e = (j * TE + te) * VEC;
    FVec<VEC> v;
    const bool in = on && e < E;  // E is a multiple of VEC
    if (in) v = *reinterpret_cast<const FVec<VEC>*>(row + e);
#pragma unroll
    for (int i = 0; i < VEC; ++i) l[j][i] = in ? v.v[i] : -INFINITY;
  }
}

template <int VEC, int TE, int EPT, int U>
__global__ void __launch_bounds__(kBalThreads) balance_fwd_kernel(const float* __restrict__ logits,
                                                                  const int32_t* __restrict__ ids,
                                                                  const uint8_t* __restrict__ valid, int64_t L, int E,
                                                                  int K, float* __restrict__ lse_out,
                                                                  float* __restrict__ part) {
  constexpr int GROUPS = kBalThreads / TE;  // tokens side by side in the CTA
  extern __shared__ float sm[];
  float* ps = sm;                                               // [warps][E]
  int* cs = reinterpret_cast<int*>(sm + kBalWarps * E);         // [E]
  float* zs = reinterpret_cast<float*>(cs + E);                 // [warps]
  int* as = reinterpret_cast<int*>(zs + kBalWarps);             // [warps]
  const int tid = threadIdx.x, te = tid % TE, grp = tid / TE, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < E; e += kBalThreads) cs[e] = 0;
  __syncthreads();
  float pa[EPT][VEC];
#pragma unroll
  for (int j = 0; j < EPT; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) pa[j][i] = 0.f;
  float za = 0.f;
  int na = 0;
  // every lane of a warp runs the same number of passes: the shuffles below are warp-wide
  for (int64_t t0 = (int64_t)blockIdx.x * GROUPS * U; t0 < L; t0 += (int64_t)gridDim.x * GROUPS * U) {
    float l[U][EPT][VEC];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * GROUPS + grp;
      on[u] = t < L && (!valid || valid[t]);
      load_row<VEC, TE, EPT>(logits + t * E, E, te, on[u], l[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * GROUPS + grp;
      float m = -INFINITY;
      bool some = false;  // a logit above -inf (or NaN, which the sum then carries)
#pragma unroll
      for (int j = 0; j < EPT; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          m = fmaxf(m, l[u][j][i]);
          some = some || !(l[u][j][i] == -INFINITY);
        }
      m = group_max<TE>(m);
      const bool act = group_max<TE>(some ? 1.f : 0.f) > 0.f;
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < EPT; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          l[u][j][i] = expf(l[u][j][i] - m);
          s += l[u][j][i];
        }
      s = group_sum<TE>(s);
      const float lse = m + logf(s), inv = 1.f / s;
      if (act) {
#pragma unroll
        for (int j = 0; j < EPT; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) pa[j][i] = fmaf(l[u][j][i], inv, pa[j][i]);
        for (int k = te; k < K; k += TE) {
          const int e = ids[t * K + k];
          if ((unsigned)e < (unsigned)E) atomicAdd(&cs[e], 1);
        }
        if (te == 0) {
          za = fmaf(lse, lse, za);
          ++na;
        }
      }
      if (te == 0 && t < L) lse_out[t] = act ? lse : -INFINITY;
    }
  }
  // over the warp's groups, then over the warps
#pragma unroll
  for (int j = 0; j < EPT; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
      for (int o = TE; o < 32; o <<= 1) pa[j][i] += __shfl_xor_sync(0xffffffffu, pa[j][i], o);
      const int e = (j * TE + te) * VEC + i;
      if (lane < TE && e < E) ps[warp * E + e] = pa[j][i];
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    za += __shfl_xor_sync(0xffffffffu, za, o);
    na += __shfl_xor_sync(0xffffffffu, na, o);
  }
  if (lane == 0) {
    zs[warp] = za;
    as[warp] = na;
  }
  __syncthreads();
  float* dst = part + (int64_t)blockIdx.x * bal_cols(E);
  for (int e = tid; e < E; e += kBalThreads) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < kBalWarps; ++w) a += ps[w * E + e];
    dst[e] = a;
    reinterpret_cast<int*>(dst)[E + 1 + e] = cs[e];
  }
  if (tid == 0) {
    float z = 0.f;
    int n = 0;
#pragma unroll
    for (int w = 0; w < kBalWarps; ++w) {
      z += zs[w];
      n += as[w];
    }
    dst[E] = z;
    reinterpret_cast<int*>(dst)[2 * E + 1] = n;
  }
}

// One CTA adds the G partial rows up (double, in a fixed order) and forms the
// two losses and the counts (the last one: the active tokens).
constexpr int kLossThreads = 1024;
__global__ void __launch_bounds__(kLossThreads) balance_losses_kernel(const float* __restrict__ part, int G, int E,
                                                                      int K, float* __restrict__ losses,
                                                                      int32_t* __restrict__ counts) {
  extern __shared__ double dsm[];
  const int C = bal_cols(E);           // at most 1026 columns
  const int tid = threadIdx.x;
  const int rows = C >= kLossThreads ? 1 : kLossThreads / C;  // threads side by side on a column
  double* col = dsm;                   // [rows][C]
  for (int i = tid; i < rows * C; i += kLossThreads) {
    const int c = i % C, r = i / C;
    const bool is_int = c > E;
    double a = 0.0;
#pragma unroll 8
    for (int g = r; g < G; g += rows) {
      const float v = part[(int64_t)g * C + c];
      a += is_int ? (double)__float_as_int(v) : (double)v;
    }
    col[r * C + c] = a;
  }
  __syncthreads();
  for (int c = tid; c < C; c += kLossThreads) {
    double a = col[c];
    for (int r = 1; r < rows; ++r) a += col[r * C + c];
    col[c] = a;
  }
  __syncthreads();
  const double n = col[2 * E + 1], inv = n > 0.0 ? 1.0 / n : 0.0;
  for (int e = tid; e < E; e += kLossThreads) counts[e] = (int32_t)col[E + 1 + e];
  if (tid == 0) counts[E] = (int32_t)n;
  if (tid < 32) {
    double b = 0.0;
    for (int e = tid; e < E; e += 32) b += (col[E + 1 + e] * inv / K) * (col[e] * inv);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
    if (tid == 0) {
      losses[0] = (float)(E * b);
      losses[1] = (float)(col[E] * inv);
    }
  }
}

template <int VEC, int TE, int EPT, int U>
__global__ void __launch_bounds__(kBalThreads) balance_bwd_kernel(
    const float* __restrict__ logits, const float* __restrict__ lse_in, const int32_t* __restrict__ counts,
    const float* __restrict__ dloss, const int32_t* __restrict__ ids, const float* __restrict__ gates,
    const float* __restrict__ dgates, int64_t L, int E, int K, float* __restrict__ dlogits) {
  constexpr int GROUPS = kBalThreads / TE;
  const int tid = threadIdx.x, te = tid % TE, grp = tid / TE;
  const int n = counts[E];
  const float inv_n = n > 0 ? 1.f / (float)n : 0.f;
  const float A = dloss[0] * (float)E * inv_n, Z = 2.f * dloss[1] * inv_n;
  // loads relative to the mean load, exact until the last product: E count_e - sum of counts
  __shared__ int total_s;
  if (tid < 32) {
    int a = 0;
    for (int e = tid; e < E; e += 32) a += counts[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (tid == 0) total_s = a;
  }
  __syncthreads();
  const double scale = n > 0 ? 1.0 / ((double)n * K * E) : 0.0;
  float f[EPT][VEC];
#pragma unroll
  for (int j = 0; j < EPT; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int e = (j * TE + te) * VEC + i;
      f[j][i] = e < E ? (float)((double)((int64_t)E * counts[e] - total_s) * scale) : 0.f;
    }
  for (int64_t t0 = (int64_t)blockIdx.x * GROUPS * U; t0 < L; t0 += (int64_t)gridDim.x * GROUPS * U) {
    float l[U][EPT][VEC], lse[U];
    bool act[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * GROUPS + grp;
      lse[u] = t < L ? lse_in[t] : -INFINITY;
      act[u] = !(lse[u] == -INFINITY);
      load_row<VEC, TE, EPT>(logits + t * E, E, te, act[u], l[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * GROUPS + grp;
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < EPT; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          l[u][j][i] = expf(l[u][j][i] - lse[u]);
          dot = fmaf(l[u][j][i], f[j][i], dot);
        }
      dot = group_sum<TE>(dot);
      const float zl = Z * lse[u];
#pragma unroll
      for (int j = 0; j < EPT; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) l[u][j][i] *= fmaf(A, f[j][i] - dot, zl);
      if (gates && act[u]) {
        float g[kMaxK], dg[kMaxK], sd = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxK; ++k) {
          g[k] = k < K ? gates[t * K + k] : 0.f;
          dg[k] = k < K ? dgates[t * K + k] : 0.f;
          sd = fmaf(g[k], dg[k], sd);
        }
#pragma unroll
        for (int k = 0; k < kMaxK; ++k) {
          const int e = k < K ? ids[t * K + k] : -1;
          const float v = g[k] * (dg[k] - sd);
#pragma unroll
          for (int j = 0; j < EPT; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (e == (j * TE + te) * VEC + i) l[u][j][i] += v;
        }
      }
      if (t < L) {
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
          const int e = (j * TE + te) * VEC;
          FVec<VEC> o;
#pragma unroll
          for (int i = 0; i < VEC; ++i) o.v[i] = act[u] ? l[u][j][i] : 0.f;
          if (e < E) *reinterpret_cast<FVec<VEC>*>(dlogits + t * E + e) = o;
        }
      }
    }
  }
}

// tokens of one pass of a CTA
template <int TE, int U>
constexpr int pass_tokens() {
  return kBalThreads / TE * U;
}

int64_t bal_ctas(int64_t L, int tokens, int per_sm) {
  const int64_t need = (L + tokens - 1) / tokens, most = (int64_t)per_sm * sm_count();
  return need < most ? need : most;
}

// The forward's CTAs: one partial row each, which one CTA adds up.
constexpr int kFwdPerSm = 1;
constexpr int kBwdPerSm = 4;

// the layout of a row of E experts: f(VEC, TE, EPT, U) as integral constants.
// 16-byte vectors when every row starts on one, single floats otherwise.
#define MB_BAL_LAYOUT(E, CALL)                            \
  do {                                                    \
    if ((E) % 4 == 0) {                                   \
      if ((E) <= 8) return CALL(4, 2, 1, 4);              \
      if ((E) <= 16) return CALL(4, 4, 1, 4);             \
      if ((E) <= 32) return CALL(4, 8, 1, 4);             \
      if ((E) <= 64) return CALL(4, 8, 2, 2);             \
      if ((E) <= 128) return CALL(4, 16, 2, 2);           \
      if ((E) <= 256) return CALL(4, 16, 4, 1);           \
      return CALL(4, 32, 4, 1);                           \
    }                                                     \
    if ((E) <= 8) return CALL(1, 8, 1, 4);                \
    if ((E) <= 16) return CALL(1, 16, 1, 4);              \
    if ((E) <= 32) return CALL(1, 32, 1, 4);              \
    if ((E) <= 64) return CALL(1, 32, 2, 4);              \
    if ((E) <= 128) return CALL(1, 32, 4, 2);             \
    if ((E) <= 256) return CALL(1, 32, 8, 1);             \
    return CALL(1, 32, 16, 1);                            \
  } while (0)

template <int VEC, int TE, int EPT, int U>
moeblaze_status fwd_layout(const moeblaze_shape& s, const float* logits, const int32_t* ids, const uint8_t* valid,
                           float* losses, int32_t* counts, float* lse, float* part, cudaStream_t st) {
  const int64_t G = bal_ctas(s.L, pass_tokens<TE, U>(), kFwdPerSm);
  const size_t sm = sizeof(float) * ((size_t)kBalWarps * s.E + s.E + 2 * kBalWarps);
  balance_fwd_kernel<VEC, TE, EPT, U><<<(unsigned)G, kBalThreads, sm, st>>>(logits, ids, valid, s.L, s.E, s.K, lse, part);
  MB_CUDA(cudaGetLastError());
  const int C = bal_cols(s.E), rows = C >= kLossThreads ? 1 : kLossThreads / C;
  balance_losses_kernel<<<1, kLossThreads, sizeof(double) * rows * C, st>>>(part, (int)G, s.E, s.K, losses, counts);
  MB_CUDA(cudaGetLastError());
  count_launch(2);
  return MOEBLAZE_OK;
}

template <int VEC, int TE, int EPT, int U>
moeblaze_status bwd_layout(const moeblaze_shape& s, const float* logits, const float* lse, const int32_t* counts,
                           const float* dloss, const int32_t* ids, const float* gates, const float* dgates,
                           float* dlogits, cudaStream_t st) {
  const int64_t G = bal_ctas(s.L, pass_tokens<TE, U>(), kBwdPerSm);
  balance_bwd_kernel<VEC, TE, EPT, U><<<(unsigned)G, kBalThreads, 0, st>>>(logits, lse, counts, dloss, ids, gates,
                                                                           dgates, s.L, s.E, s.K, dlogits);
  MB_CUDA(cudaGetLastError());
  count_launch();
  return MOEBLAZE_OK;
}

}  // namespace

size_t balance_ws_bytes(const moeblaze_shape& s) {
  return sizeof(float) * (size_t)kFwdPerSm * sm_count() * bal_cols(s.E);
}

moeblaze_status launch_balance_forward(const moeblaze_shape& s, const float* logits, const int32_t* ids,
                                       const uint8_t* valid, float* losses, int32_t* counts, float* lse, void* ws,
                                       cudaStream_t st) {
  if (s.L == 0) {
    MB_CUDA(cudaMemsetAsync(losses, 0, 2 * sizeof(float), st));
    MB_CUDA(cudaMemsetAsync(counts, 0, sizeof(int32_t) * (s.E + 1), st));
    return MOEBLAZE_OK;
  }
#define MB_CALL(VEC, TE, EPT, U) \
  fwd_layout<VEC, TE, EPT, U>(s, logits, ids, valid, losses, counts, lse, (float*)ws, st)
  MB_BAL_LAYOUT(s.E, MB_CALL);
#undef MB_CALL
}

moeblaze_status launch_balance_backward(const moeblaze_shape& s, const float* logits, const float* lse,
                                        const int32_t* counts, const float* dloss, const int32_t* ids,
                                        const float* gates, const float* dgates, float* dlogits, cudaStream_t st) {
  if (s.L == 0) return MOEBLAZE_OK;
#define MB_CALL(VEC, TE, EPT, U) \
  bwd_layout<VEC, TE, EPT, U>(s, logits, lse, counts, dloss, ids, gates, dgates, dlogits, st)
  MB_BAL_LAYOUT(s.E, MB_CALL);
#undef MB_CALL
}

}  // namespace moeblaze
