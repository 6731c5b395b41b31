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
//   rows of tokens that are not active are zero, or have the gates' share
//   alone (the mask is the losses': a token it leaves out is still routed).
//
// f_e - sum_j f_j p_tj cancels when the load is even; both sides are taken
// relative to the mean load (sum_j p_tj = 1 leaves the difference as it is).
//
// A token's row of logits lies in TE lanes of a warp, EPT vectors of VEC
// experts each; P_e is summed in a lane's registers over the CTA's tokens,
// then over the warps and (balance_losses_kernel) over the CTAs, always in
// the same order: repeatable to the bit.
//
// The bytes would take 3 and 5 us at 65536 x 64; what counts is the chain of
// launch, first loads and last sums: 9.5 us forward, 3 us for the losses and
// 11 us backward there, loss and gradient together 24 us.
#include "common.cuh"

namespace moeblaze {
namespace {

constexpr int kBalThreads = 1024;  // forward: one CTA an SM, few partial sums
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBwdThreads = 256;

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
__device__ __forceinline__ void load_row(const float* row, int E, int te, bool on, float (&l)[EPT][VEC]) {
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

// The losses from the sums, by one warp: n active tokens, count[e] slots and
// P[e] = sum_t p_te of E experts, z = sum_t lse_t^2
__device__ __forceinline__ void write_losses(int E, int K, int n, const int* count, const float* P, float z,
                                             float* __restrict__ losses) {
  const int lane = threadIdx.x & 31;
  float b = 0.f;  // sum_e count_e P_e
  for (int e = lane; e < E; e += 32) b = fmaf((float)count[e], P[e], b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
  if (lane == 0) {
    const float inv = n > 0 ? 1.f / (float)n : 0.f;
    losses[0] = ((float)E / (float)K) * (b * inv) * inv;
    losses[1] = inv * z;
  }
}

template <int VEC, int TE, int EPT, int U>
__global__ void __launch_bounds__(kBalThreads) balance_fwd_kernel(const float* __restrict__ logits,
                                                                  const int32_t* __restrict__ ids,
                                                                  const uint8_t* __restrict__ valid, int64_t L, int E,
                                                                  int K, float* __restrict__ lse_out,
                                                                  float* __restrict__ part,
                                                                  float* __restrict__ losses,
                                                                  int32_t* __restrict__ counts) {
  constexpr int GROUPS = kBalThreads / TE;  // tokens side by side in the CTA
  constexpr int KL = (kMaxK + TE - 1) / TE;  // slots a lane counts
  extern __shared__ float sm[];
  float* ps = sm;                                               // [warps][E]
  int* cs = reinterpret_cast<int*>(sm + kBalWarps * E);         // [E]
  float* zs = reinterpret_cast<float*>(cs + E);                 // [warps]
  int* as = reinterpret_cast<int*>(zs + kBalWarps);             // [warps]
  const int tid = threadIdx.x, te = tid % TE, grp = tid / TE, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
    int id[U][KL];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * GROUPS + grp;
      on[u] = t < L && (!valid || valid[t]);
#pragma unroll
      for (int q = 0; q < KL; ++q) id[u][q] = q * TE + te < K && t < L ? ids[t * K + q * TE + te] : -1;
      load_row<VEC, TE, EPT>(logits + t * E, E, te, on[u], l[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * GROUPS + grp;
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < EPT; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = fmaxf(m, l[u][j][i]);
      m = group_max<TE>(m);
      bool act = m > -INFINITY;
      if (__any_sync(0xffffffffu, on[u] && !act)) {
        // the maximum leaves NaN out: a row of NaN (and -inf) is active, and its sum NaN
        bool nan = false;
#pragma unroll
        for (int j = 0; j < EPT; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) nan = nan || l[u][j][i] != l[u][j][i];
        const float any_nan = group_max<TE>(nan ? 1.f : 0.f);  // by every lane: a shuffle
        if (any_nan > 0.f) act = true;
      }
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
#pragma unroll
        for (int q = 0; q < KL; ++q)
          if ((unsigned)id[u][q] < (unsigned)E) atomicAdd(&cs[id[u][q]], 1);
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
  // a CTA's own sums: to the workspace, or, when it is the only one, on to the losses
  const bool only = gridDim.x == 1;
  float* dst = part + (int64_t)blockIdx.x * bal_cols(E);
  for (int e = tid; e < E; e += kBalThreads) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < kBalWarps; ++w) a += ps[w * E + e];
    if (only) {
      ps[e] = a;  // (column e is this thread's alone)
      counts[e] = cs[e];
    } else {
      dst[e] = a;
      reinterpret_cast<int*>(dst)[E + 1 + e] = cs[e];
    }
  }
  if (only) __syncthreads();
  if (tid < 32) {
    float z = zs[tid];
    int n = as[tid];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      z += __shfl_xor_sync(0xffffffffu, z, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (only) {
      if (tid == 0) counts[E] = n;
      write_losses(E, K, n, cs, ps, z, losses);
    } else if (tid == 0) {
      dst[E] = z;
      reinterpret_cast<int*>(dst)[2 * E + 1] = n;
    }
  }
}

// One cluster adds the G partial rows up, each of its CTAs an equal range of
// them, and its first CTA, in whose shared memory the others put their sums,
// forms the two losses and the counts (the last one: the active tokens).
// Sums of positive fp32 numbers in trees of a few levels.
constexpr int kLossThreads = 512;
constexpr int kLossCluster = 8;
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__global__ void __launch_bounds__(kLossThreads) balance_losses_kernel(const float* part, int G, int E,
                                                                      int K, float* __restrict__ losses,
                                                                      int32_t* __restrict__ counts) {
  extern __shared__ float fsm[];
  const int C = bal_cols(E);           // at most 1026 columns
  const int tid = threadIdx.x;
  const int rows = C >= kLossThreads ? 1 : kLossThreads / C;  // threads side by side on a column
  float* all = fsm;                    // [kLossCluster][C] in the first CTA: every CTA's sums; then the whole sums
  float* col = fsm + kLossCluster * C; // [rows][C]; the integer columns hold int bits
  int rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int g0 = G * rank / kLossCluster, g1 = G * (rank + 1) / kLossCluster;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  cluster_sync();  // the first CTA runs: its shared memory may be written
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = tid; i < rows * C; i += kLossThreads) {
    const int c = i % C, r = i / C;
    float a = 0.f;
    int n = 0;
    // eight in flight at a time, the last ones too
    for (int g = g0 + r; g < g1; g += 8 * rows) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = g + u * rows < g1 ? part[(int64_t)(g + u * rows) * C + c] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (c > E) n += __float_as_int(v[u]);
        else a += v[u];
      }
    }
    col[i] = c > E ? __int_as_float(n) : a;
  }
  // column c over n values, ld floats apart; integer columns as integers
  auto add_up = [&](const float* p, int c, int n, int ld) {
    float a = 0.f;
    int k = 0;
#pragma unroll 4
    for (int r = 0; r < n; ++r) {
      const float v = p[r * ld];
      if (c > E) k += __float_as_int(v);
      else a += v;
    }
    return c > E ? __int_as_float(k) : a;
  };
  __syncthreads();
  for (int c = tid; c < C; c += kLossThreads) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
                 : "=r"(at)
                 : "r"((uint32_t)__cvta_generic_to_shared(all + rank * C + c)));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(add_up(col + c, c, rows, C)) : "memory");
  }
  __syncthreads();
  cluster_sync();
  if (rank != 0) return;
  for (int c = tid; c < C; c += kLossThreads) {
    const float v = add_up(all + c, c, kLossCluster, C);
    all[c] = v;  // (column c is this thread's alone)
    if (c > E) counts[c - E - 1] = __float_as_int(v);  // counts[E] is the active tokens
  }
  __syncthreads();
  if (tid < 32)
    write_losses(E, K, __float_as_int(all[2 * E + 1]), reinterpret_cast<const int*>(all) + E + 1, all, all[E], losses);
}

// MASK: 1 with a mask of its own, 2 (with or without one) with the gates' share
// of tokens that are out of the losses (variants of their own: 2 takes 0.6 us
// more at 65536 x 64)
template <int VEC, int TE, int EPT, int U, int MASK>
__global__ void __launch_bounds__(kBwdThreads) balance_bwd_kernel(
    const float* logits, const float* lse_in, const int32_t* counts, const float* dloss, const int32_t* ids,
    const float* gates, const float* dgates, const uint8_t* valid, int64_t L, int E, int K, float* dlogits) {
  // (no __restrict__: what the kernel before has written must not be read ahead of the wait)
  constexpr int GROUPS = kBwdThreads / TE;
  constexpr int KL = (kMaxK + TE - 1) / TE;  // slots a lane holds
  constexpr int ROW = EPT * TE * VEC + 4;    // a group's row in shared memory (rows 4 banks apart)
  __shared__ __align__(16) float rows[GROUPS * ROW];
  const int tid = threadIdx.x, te = tid % TE, grp = tid / TE;
  float* row = rows + grp * ROW;
  float l[U][EPT][VEC], lse[U], g[U][KL], dg[U][KL];
  int id[U][KL];
  bool act[U], on[U];
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * GROUPS + grp;
      lse[u] = t < L ? lse_in[t] : -INFINITY;
      if (MASK) on[u] = !valid || (t < L && valid[t]);
      // (the logits of a token that is not active are loaded and not used)
      load_row<VEC, TE, EPT>(logits + t * E, E, te, t < L, l[u]);
#pragma unroll
      for (int q = 0; q < KL; ++q) {
        const int k = q * TE + te;
        const bool in = gates && k < K && t < L;
        g[u][q] = in ? gates[t * K + k] : 0.f;
        dg[u][q] = in ? dgates[t * K + k] : 0.f;
        id[u][q] = in ? ids[t * K + k] : -1;
      }
    }
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the first tokens are on their way while the loads are looked up
  fetch((int64_t)blockIdx.x * GROUPS * U);
  const int n = counts[E];
  const float inv_n = n > 0 ? 1.f / (float)n : 0.f;
  const float A = dloss[0] * (float)E * inv_n, Z = 2.f * dloss[1] * inv_n;
  // loads relative to the mean load: the integer part of the difference is
  // exact (in fp32 and integers: fp64 runs at 1/64 of its rate, and this is
  // every CTA's start)
  int total = 0;  // by every warp for itself
  for (int e = tid & 31; e < E; e += 32) total += counts[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int mean = total / E;
  const float rest = (float)(total % E) / (float)E, scale = n > 0 ? 1.f / ((float)n * (float)K) : 0.f;
  float f[EPT][VEC];
#pragma unroll
  for (int j = 0; j < EPT; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int e = (j * TE + te) * VEC + i;
      f[j][i] = e < E ? ((float)(counts[e] - mean) - rest) * scale : 0.f;
    }
  const int64_t step = (int64_t)gridDim.x * GROUPS * U;
  for (int64_t t0 = (int64_t)blockIdx.x * GROUPS * U; t0 < L; t0 += step) {
    if (t0 >= step) fetch(t0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * GROUPS + grp;
      act[u] = !(lse[u] == -INFINITY) && (!MASK || on[u]);
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
        for (int i = 0; i < VEC; ++i) {
          l[u][j][i] *= fmaf(A, f[j][i] - dot, zl);
          if (MASK == 2 && !act[u]) l[u][j][i] = 0.f;
        }
      if (gates) {
        // the chosen experts' share: the row goes through shared memory,
        // where the lane that holds a slot adds to that slot's expert, slot
        // after slot (an expert named twice gets both, in their order)
        float sd = 0.f;
#pragma unroll
        for (int q = 0; q < KL; ++q) sd = fmaf(g[u][q], dg[u][q], sd);
        sd = group_sum<TE>(sd);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
          FVec<VEC> o;
#pragma unroll
          for (int i = 0; i < VEC; ++i) o.v[i] = l[u][j][i];
          *reinterpret_cast<FVec<VEC>*>(row + (j * TE + te) * VEC) = o;
        }
#pragma unroll
        for (int k = 0; k < kMaxK; ++k) {
          if (k < K) {
            __syncwarp();
            const int e = id[u][k / TE];
            if (te == k % TE && (unsigned)e < (unsigned)E) row[e] += g[u][k / TE] * (dg[u][k / TE] - sd);
          }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
          const FVec<VEC> o = *reinterpret_cast<const FVec<VEC>*>(row + (j * TE + te) * VEC);
#pragma unroll
          for (int i = 0; i < VEC; ++i) l[u][j][i] = o.v[i];
        }
      }
      if (t < L) {
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
          const int e = (j * TE + te) * VEC;
          FVec<VEC> o;
#pragma unroll
          for (int i = 0; i < VEC; ++i) o.v[i] = MASK == 2 || act[u] ? l[u][j][i] : 0.f;
          if (e < E) *reinterpret_cast<FVec<VEC>*>(dlogits + t * E + e) = o;
        }
      }
    }
  }
}

// tokens of one pass of a CTA
template <int THREADS, int TE, int U>
constexpr int pass_tokens() {
  return THREADS / TE * U;
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
      if ((E) <= 8) return CALL(4, 2, 1, 2);              \
      if ((E) <= 16) return CALL(4, 4, 1, 2);             \
      if ((E) <= 32) return CALL(4, 8, 1, 2);             \
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

constexpr size_t fwd_smem(int E) { return sizeof(float) * ((size_t)kBalWarps * E + E + 2 * kBalWarps); }

template <int VEC, int TE, int EPT, int U>
moeblaze_status fwd_layout(const moeblaze_shape& s, const float* logits, const int32_t* ids, const uint8_t* valid,
                           float* losses, int32_t* counts, float* lse, float* part, cudaStream_t st) {
  const int64_t G = bal_ctas(s.L, pass_tokens<kBalThreads, TE, U>(), kFwdPerSm);
  const size_t sm = fwd_smem(s.E);
  auto kern = balance_fwd_kernel<VEC, TE, EPT, U>;
  if (sm > 48 * 1024) MB_CUDA(smem_limit(kern, fwd_smem(kMaxE)));
  kern<<<(unsigned)G, kBalThreads, sm, st>>>(logits, ids, valid, s.L, s.E, s.K, lse, part, losses, counts);
  MB_CUDA(cudaGetLastError());
  count_launch();
  if (G == 1) return MOEBLAZE_OK;
  const int C = bal_cols(s.E), rows = C >= kLossThreads ? 1 : kLossThreads / C;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kLossCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(kLossCluster);
  cfg.blockDim = dim3(kLossThreads);
  cfg.dynamicSmemBytes = sizeof(float) * (kLossCluster + rows) * C;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  MB_CUDA(cudaLaunchKernelEx(&cfg, balance_losses_kernel, (const float*)part, (int)G, (int)s.E, (int)s.K, losses,
                             counts));
  count_launch();
  return MOEBLAZE_OK;
}

template <int VEC, int TE, int EPT, int U>
moeblaze_status bwd_layout(const moeblaze_shape& s, const float* logits, const float* lse, const int32_t* counts,
                           const float* dloss, const int32_t* ids, const float* gates, const float* dgates,
                           const uint8_t* valid, bool gates_of_all, float* dlogits, cudaStream_t st) {
  const int64_t G = bal_ctas(s.L, pass_tokens<kBwdThreads, TE, U>(), kBwdPerSm);
  // it may be set up while the kernel before it runs (and waits for its end)
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)G);
  cfg.blockDim = dim3(kBwdThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = gates_of_all ? balance_bwd_kernel<VEC, TE, EPT, U, 2>
              : valid      ? balance_bwd_kernel<VEC, TE, EPT, U, 1>
                           : balance_bwd_kernel<VEC, TE, EPT, U, 0>;
  MB_CUDA(cudaLaunchKernelEx(&cfg, kern, logits, lse, counts, dloss, ids, gates, dgates,
                             valid, (int64_t)s.L, (int)s.E, (int)s.K, dlogits));
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
                                        const float* gates, const float* dgates, const uint8_t* valid,
                                        bool gates_of_all, float* dlogits, cudaStream_t st) {
  if (s.L == 0) return MOEBLAZE_OK;
#define MB_CALL(VEC, TE, EPT, U) \
  bwd_layout<VEC, TE, EPT, U>(s, logits, lse, counts, dloss, ids, gates, dgates, valid, gates_of_all, dlogits, st)
  MB_BAL_LAYOUT(s.E, MB_CALL);
#undef MB_CALL
}

}  // namespace moeblaze
