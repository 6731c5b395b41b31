// The router's gradients from a dense gradient of its logits, on the tensor
// cores (bf16 x, up to 128 experts):
//
//   dWr = x^T dl,  dx = dl Wr^T,  dbias = sum_t dl[t]
//
// Both products have the expert count as their small extent and are bound by
// HBM: dWr reads x once, dx is written once.  dl and Wr are fp32.  They are
// split into bf16 parts, v = hi + mid + lo (each the rounding of what the
// parts before it leave), so that every product of two parts is exact and
// the sums are fp32 in TMEM:
//   dWr: x . hi + x . mid + x . lo              (dWr is fp32: 24 bits of dl)
//   dx:  hi . Whi + hi . Wmid + mid . Whi       (dx is bf16: 16 bits of each)
//
// split_kernel writes dl's parts as rows [hi | mid | lo] of EP columns each
// (EP = 16, 32 or 64 experts, padded to whole 64-column blocks), Wr's as
// [hi | mid], and the CTAs' sums of dl for dbias.  More than 64 experts are
// two groups of 64, a group's parts side by side.
//
// dwr_kernel: a CTA owns 256 columns of x and a range of tokens; TMA brings
// 64 tokens x (256 columns of x, the parts of dl) per stage, both operands
// MN-major (tokens are the reduction); two M = 128 MMAs share the dl tile.
// The tensor cores' fp32 sums are truncated, not rounded, at every step: over
// thousands of tokens the error is six times a rounded sum's (4.2e-6 of the
// norm at 3,640 tokens).  So the accumulator is emptied every 512 tokens
// into fp32 sums in the epilogue warps' registers, two accumulators in turn,
// and stored at the end as the range's partial dWr.  65536 x 2048, 64 experts:
// 55 us, 4.9 TB/s of x; an SM takes in about 35 bytes a clock, here 24 KB of
// dl's parts for every 32 KB of x (one load of dl for pairs of CTAs: 57 us,
// the same bytes arrive).  32768 x 4096, 8 experts: 42 us, 6.4 TB/s.
//
// dx_kernel: a CTA owns 256 columns of dx, whose rows of Wr stay in shared
// memory, and walks over 128-token tiles, two TMEM accumulators in turn, so
// that the epilogue (round, stage, TMA store) of one tile runs under the MMAs
// of the next: 48 and 43 us for the same sizes, 5.6 and 6.2 TB/s of stores.
// grad_reduce_kernel adds the partial sums up in a fixed order.
#include <algorithm>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace moeblaze {
namespace tc {
namespace {

constexpr int kGThreads = 320;  // warp 0 TMA, warp 1 MMA, warps 2-9 epilogue
constexpr int kGCols = 256;     // columns of x (dx) of a CTA
constexpr int kDxTokens = 128;
constexpr int kDxStages = 3;
constexpr int kDwStages = 4;
constexpr int kDwTokens = 64;
constexpr int kDwFlush = 8;     // stages summed in TMEM before the registers take over

constexpr int dl_width(int ep) { return (3 * ep + 63) / 64 * 64; }
constexpr int wr_width(int ep) { return (2 * ep + 63) / 64 * 64; }
constexpr int dx_blocks(int ep) { return wr_width(ep) / 64; }   // 64-column blocks of hi | mid
constexpr int dw_atoms(int ep) { return dl_width(ep) / 64; }
// columns of dx of a CTA: two groups' rows of Wr leave room for half as many
constexpr int dx_cols(int groups) { return groups == 2 ? kGCols / 2 : kGCols; }
constexpr int dx_smem(int ep, int groups) {  // Wr | token tiles | store staging | barriers | alignment
  return groups * dx_blocks(ep) * dx_cols(groups) * 128 + kDxStages * dx_blocks(ep) * kDxTokens * 128 + 8 * 2 * 4096 + 256 + 1024;
}
constexpr int dw_stage(int ep) { return (kGCols / 64 + dw_atoms(ep)) * 8192; }
constexpr int dw_smem(int ep) { return kDwStages * dw_stage(ep) + 256 + 1024; }

// ------------------------------------------------------------------ parts
// rows of dl (L x E fp32) -> [hi | mid | lo], V columns a thread (one 16-byte
// load where every row starts on one, else single floats), all of a thread's
// rows in flight together; part_b[block][e] = the block's tokens' sum.
// Blocks past the tokens' split Wr (d x E) -> [hi | mid].  blockIdx.y: the group
// of experts, gridDim.y of them.
// (65536 x 64: 8.4 us, against 10.6 us with two columns and four rows.)
__device__ __forceinline__ void allow_dependents();
constexpr int kSplitThreads = 256;
__device__ __forceinline__ void parts(float v, float& hi, float& mid, float& lo) {
  hi = __bfloat162float(__float2bfloat16_rn(v));
  const float r = v - hi;  // exact
  mid = __bfloat162float(__float2bfloat16_rn(r));
  lo = r - mid;  // exact; rounded when stored
}
template <int V>
__device__ __forceinline__ void split_load(const float* row, int c, int E, bool on, float (&v)[V]) {
  if constexpr (V == 4) {
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on && c < E) f = *reinterpret_cast<const float4*>(row + c);  // E is a multiple of 4, as the whole row's
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = on && c + i < E ? row[c + i] : 0.f;
  }
}
template <int V>
__device__ __forceinline__ void split_store(__nv_bfloat16* o, const float (&v)[V]) {
  if constexpr (V == 4) *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  else *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(v[0], v[1]);
}
template <int EP, int V>
__global__ void __launch_bounds__(kSplitThreads, 3) split_kernel(const float* __restrict__ dl, const float* __restrict__ Wr,
                                                              int64_t L, int d, int E, int64_t rows, int tblocks,
                                                              __nv_bfloat16* __restrict__ dls,
                                                              __nv_bfloat16* __restrict__ ws,
                                                              float* __restrict__ part_b, int32_t* __restrict__ err) {
  constexpr int PR = EP / V, SIDE = kSplitThreads / PR;  // threads of a row, rows side by side
  constexpr int U = EP / 8;                              // rows of a thread in flight
  const int tid = threadIdx.x, c = (tid % PR) * V, r0 = tid / PR;
  const int g0 = 64 * (int)blockIdx.y, EG = min(EP, E - g0);  // the group's first expert, its experts
  const float zero[V] = {};
  allow_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *err = 0;
  if ((int)blockIdx.x < tblocks) {
    constexpr int W = dl_width(EP);
    dls += blockIdx.y * W;
    const int64_t t0 = blockIdx.x * rows, t1 = min(L, t0 + rows);
    float sum[V] = {};
    for (int64_t t = t0 + r0; t < t1; t += SIDE * U) {
      float v[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u) split_load<V>(dl + (t + u * SIDE) * E + g0, c, EG, t + u * SIDE < t1, v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u * SIDE < t1) {
          float hi[V], mid[V], lo[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            sum[i] += v[u][i];
            parts(v[u][i], hi[i], mid[i], lo[i]);
          }
          __nv_bfloat16* o = dls + (t + u * SIDE) * (gridDim.y * W) + c;
          split_store<V>(o, hi);
          split_store<V>(o + EP, mid);
          split_store<V>(o + 2 * EP, lo);
          if (W > 3 * EP) split_store<V>(o + 3 * EP, zero);  // (W - 3 EP is EP or 0)
        }
      }
    }
    __shared__ float acc[SIDE][EP];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[r0][c + i] = sum[i];
    __syncthreads();
    if (tid < EG) {
      float a = 0.f;
#pragma unroll 8
      for (int i = 0; i < SIDE; ++i) a += acc[i][tid];
      part_b[(int64_t)blockIdx.x * E + g0 + tid] = a;
    }
  } else {
    constexpr int W = wr_width(EP);
    ws += blockIdx.y * W;
    const int wblocks = (int)gridDim.x - tblocks;
    for (int j = ((int)blockIdx.x - tblocks) * SIDE + r0; j < d; j += wblocks * SIDE) {
      float v[V], hi[V], mid[V], lo[V];
      split_load<V>(Wr + (int64_t)j * E + g0, c, EG, true, v);
#pragma unroll
      for (int i = 0; i < V; ++i) parts(v[i], hi[i], mid[i], lo[i]);
      __nv_bfloat16* o = ws + (int64_t)j * (gridDim.y * W) + c;
      split_store<V>(o, hi);
      split_store<V>(o + EP, mid);
      if (W > 2 * EP) {  // EP = 16: 64 columns
        split_store<V>(o + 2 * EP, zero);
        split_store<V>(o + 3 * EP, zero);
      }
    }
  }
}

struct GParams {
  CUtensorMap tmA, tmB, tmO;  // dx: dl parts, Wr parts, dx;  dwr: x, dl parts
  int64_t L;
  int d, E, tiles, splits;    // tiles of columns; splits: CTAs per tile (and group)
  int groups;                 // dwr: groups of 64 experts
  int64_t chunks;             // dwr: 64-token chunks of a split
  int add;                    // dx: added to what is there
  float* part;
  int32_t* err;
  uint64_t wait_ns;
};

// programmatic dependents: the next kernel of the call may set itself up on
// SMs this one has left, and waits for it before it reads anything
__device__ __forceinline__ void allow_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_prior() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void tmem_alloc_512(uint32_t slot) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_512(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base) : "memory");
}

// a tile added to the one in memory (bf16 sums, rounded to nearest, in L2)
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}

// ------------------------------------------------------------------ dx
// A ring stage is one group's parts of a token tile; the groups of a tile
// follow one another in the ring and add up in its accumulator.
template <int EP, int GROUPS>
__global__ void __launch_bounds__(kGThreads, 1) dx_kernel(const __grid_constant__ GParams p) {
  constexpr int NB = dx_blocks(EP), COLS = dx_cols(GROUPS);
  constexpr int SA = NB * kDxTokens * 128, SG = NB * COLS * 128, SW = GROUPS * SG;
  extern __shared__ uint8_t g_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(g_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sw = smem;                             // Wr: [group][block][COLS rows][128 bytes]
  uint8_t* sa = sw + SW;                          // ring: [stage][block][128 tokens][128 bytes]
  uint8_t* so = sa + kDxStages * SA;              // [warp][2][32 rows][128 bytes]
  uint64_t* bars = reinterpret_cast<uint64_t*>(so + 8 * 2 * 4096);
  // full[3], empty[3], wfull, dfull[2], dempty[2], done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 12);
  volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + 3 + s); };
  const uint32_t wfull = smem_u32(bars + 6), done = smem_u32(bars + 11);
  auto dfull = [&](int b) { return smem_u32(bars + 7 + b); };
  auto dempty = [&](int b) { return smem_u32(bars + 9 + b); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n0 = (int)(blockIdx.x % p.tiles) * COLS, split = (int)(blockIdx.x / p.tiles);
  const int nw = min(COLS, p.d - n0);  // a multiple of 64
  const int64_t tblocks = (p.L + kDxTokens - 1) / kDxTokens;
  const uint64_t lim = p.wait_ns;
  allow_dependents();

  if (tid == 0) {
    for (int s = 0; s < kDxStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(wfull, 1);
    mbar_init(done, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(dfull(b), 1);
      mbar_init(dempty(b), 8);
    }
    *abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc_512(smem_u32(tmem_slot));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_prior();

  if (warp == 0) {
    // ============================================================ TMA producer
    if (lane == 0) {
      mbar_expect_tx(wfull, (uint32_t)SW);
      for (int b = 0; b < GROUPS * NB; ++b)
        for (int r = 0; r < COLS; r += 128)  // rows past d are filled with zeros
          tma_load_2d(smem_u32(sw + b * COLS * 128 + r * 128), &p.tmB, b * 64, n0 + r, wfull);
      int s = 0;
      uint32_t ph = 0, armed = 0, armed_par = 0;
      bool ok = true;
      for (int64_t t = split; ok && t < tblocks; t += p.splits) {
        for (int g = 0; g < GROUPS; ++g) {
          ok = wait_bounded(empty(s), ph ^ 1u, abort_s, p.err, lim);
          if (!ok) break;
          mbar_expect_tx(full(s), (uint32_t)SA);
          for (int b = 0; b < NB; ++b)  // (a group's lo columns are not read)
            tma_load_2d(smem_u32(sa + s * SA + b * kDxTokens * 128), &p.tmA, g * dl_width(EP) + b * 64,
                        (int)(t * kDxTokens), full(s));
          armed |= 1u << s;
          armed_par = (armed_par & ~(1u << s)) | (ph << s);
          if (++s == kDxStages) { s = 0; ph ^= 1u; }
        }
      }
      // a CTA that gave up lets its copies in flight land before it exits
      if (*abort_s) {
        wait_bounded(wfull, 0u, nullptr, nullptr, kDrainNs);
        for (int i = 0; i < kDxStages; ++i)
          if ((armed >> i) & 1u) wait_bounded(full(i), (armed_par >> i) & 1u, nullptr, nullptr, kDrainNs);
      }
    }
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = instr_desc(nw, false, false);
      const uint32_t w0 = smem_u32(sw);
      int s = 0, b = 0;
      uint32_t ph = 0, dph = 0;
      bool ok = wait_bounded(wfull, 0u, abort_s, p.err, lim);
      for (int64_t t = split; ok && t < tblocks; t += p.splits) {
        ok = wait_bounded(dempty(b), dph ^ 1u, abort_s, p.err, lim);
        for (int g = 0; ok && g < GROUPS; ++g) {
          ok = wait_bounded(full(s), ph, abort_s, p.err, lim);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a0 = smem_u32(sa + s * SA), wg = w0 + g * SG;
          // slice q (16 experts) of part h: 64-column block (h EP / 16 + q) / 4
          auto da = [&](int h, int q) {
            const int i = h * (EP / 16) + q;
            return smem_desc(a0 + (i / 4) * kDxTokens * 128 + (i % 4) * 32, 16, 1024);
          };
          auto dw = [&](int h, int q) {
            const int i = h * (EP / 16) + q;
            return smem_desc(wg + (i / 4) * COLS * 128 + (i % 4) * 32, 16, 1024);
          };
          const uint32_t acc = tmem + b * 256;
#pragma unroll
          for (int q = 0; q < EP / 16; ++q) {
            mma_bf16(acc, da(0, q), dw(0, q), idesc, g > 0 || q > 0);
            mma_bf16(acc, da(0, q), dw(1, q), idesc, 1u);
            mma_bf16(acc, da(1, q), dw(0, q), idesc, 1u);
          }
          mma_commit(empty(s));
          if (++s == kDxStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        mma_commit(dfull(b));
        b ^= 1;
        if (b == 0) dph ^= 1u;
      }
      mma_commit(done);  // every MMA issued retires before TMEM is freed
      wait_bounded(done, 0u, nullptr, nullptr, *abort_s ? kDrainNs : lim);
    }
    __syncwarp();
  } else {
    // ============================================================ epilogue
    // warp: 32 tokens (its quarter of the TMEM lanes) x half of the columns,
    // 64 at a time through two staging buffers of its own
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    uint8_t* buf = so + (warp - 2) * 2 * 4096;
    int b = 0, q = 0;
    uint32_t dph = 0;
    for (int64_t t = split; t < tblocks; t += p.splits) {
      // warp-uniform: the TMEM loads below are warp-collective
      if (!__all_sync(0xffffffffu, wait_bounded(dfull(b), dph, abort_s, p.err, lim))) break;
      tc_fence_after();
      const int64_t row0 = t * kDxTokens + quarter * 32;
      for (int c = half * (COLS / 2); c < (half + 1) * (COLS / 2); c += 64) {
        if (c >= nw) break;
        uint32_t v[64];
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(b * 256 + c);
        MB_TMEM_LD32(at, v);
        {
          uint32_t* v2 = v + 32;
          MB_TMEM_LD32(at + 32, v2);
        }
        tmem_wait_ld();
        if (lane == 0) bulk_wait_read<1>();  // the store from this buffer two steps ago has been read
        __syncwarp();
        const uint32_t dst = smem_u32(buf + q * 4096) + lane * 128;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint4 o;
          o.x = pack_bf16x2(__uint_as_float(v[8 * i]), __uint_as_float(v[8 * i + 1]));
          o.y = pack_bf16x2(__uint_as_float(v[8 * i + 2]), __uint_as_float(v[8 * i + 3]));
          o.z = pack_bf16x2(__uint_as_float(v[8 * i + 4]), __uint_as_float(v[8 * i + 5]));
          o.w = pack_bf16x2(__uint_as_float(v[8 * i + 6]), __uint_as_float(v[8 * i + 7]));
          st_shared_v4(dst + ((i ^ (lane & 7)) << 4), o);  // the 128-byte swizzle of the store's map
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0 && row0 < p.L) {
          if (p.add) tma_add_2d(&p.tmO, smem_u32(buf + q * 4096), n0 + c, (int)row0);
          else tma_store_2d(&p.tmO, smem_u32(buf + q * 4096), n0 + c, (int)row0);
        }
        if (lane == 0) bulk_commit();
        q ^= 1;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dempty(b));
      b ^= 1;
      if (b == 0) dph ^= 1u;
    }
    if (lane == 0) bulk_wait<0>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free_512(tmem);
}

// ------------------------------------------------------------------ dWr
template <int EP>
__global__ void __launch_bounds__(kGThreads, 1) dwr_kernel(const __grid_constant__ GParams p) {
  // The parts of dl side by side: N = 3 EP columns, an accumulator for each
  // 128-column half of the tile.  EP = 16, 32: two of each, in turn.  EP = 64:
  // one (two of 2 x 192 columns do not fit), and a half's sums are taken
  // while the other half's products run.
  constexpr int NA = kGCols / 64, NB = dw_atoms(EP), SB = dw_stage(EP), N = 3 * EP, BUFS = EP == 64 ? 1 : 2;
  extern __shared__ uint8_t g_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(g_raw) + 1023) & ~uintptr_t(1023));
  // full[4], empty[4], done, dfull[2][2], dempty[2][2] (buffer, half)
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kDwStages * SB);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kDwStages + 9);
  volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + kDwStages + s); };
  const uint32_t done = smem_u32(bars + 2 * kDwStages);
  auto dfull = [&](int b, int h) { return smem_u32(bars + 2 * kDwStages + 1 + 2 * b + h); };
  auto dempty = [&](int b, int h) { return smem_u32(bars + 2 * kDwStages + 5 + 2 * b + h); };
  auto acc_col = [](int b, int h) { return EP == 64 ? h * N : b * 256 + h * 128; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the groups of a tile and split side by side: the second finds x in L2
  const int m0 = (int)(blockIdx.x % p.tiles) * kGCols, group = (int)(blockIdx.x / p.tiles) % p.groups;
  const int split = (int)(blockIdx.x / p.tiles) / p.groups;
  const int64_t all = (p.L + kDwTokens - 1) / kDwTokens;
  const int64_t c0 = split * p.chunks, c1 = min(all, c0 + p.chunks);  // at least one: the host makes no empty split
  const uint64_t lim = p.wait_ns;
  allow_dependents();
  if (tid == 0) {
    for (int s = 0; s < kDwStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    for (int b = 0; b < 2; ++b)
      for (int h = 0; h < 2; ++h) {
        mbar_init(dfull(b, h), 1);
        mbar_init(dempty(b, h), 4);
      }
    *abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc_512(smem_u32(tmem_slot));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_prior();

  if (warp == 0) {
    // ============================================================ TMA producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, armed = 0, armed_par = 0;
      for (int64_t c = c0; c < c1; ++c) {
        if (!wait_bounded(empty(s), ph ^ 1u, abort_s, p.err, lim)) break;
        mbar_expect_tx(full(s), (uint32_t)SB);
        const uint32_t at = smem_u32(smem + s * SB);
        // tokens past L and columns past d are filled with zeros
        for (int a = 0; a < NA; ++a) tma_load_2d(at + a * 8192, &p.tmA, m0 + a * 64, (int)(c * kDwTokens), full(s));
        for (int a = 0; a < NB; ++a) tma_load_2d(at + (NA + a) * 8192, &p.tmB, (group * NB + a) * 64, (int)(c * kDwTokens), full(s));
        armed |= 1u << s;
        armed_par = (armed_par & ~(1u << s)) | (ph << s);
        if (++s == kDwStages) { s = 0; ph ^= 1u; }
      }
      if (*abort_s)
        for (int i = 0; i < kDwStages; ++i)
          if ((armed >> i) & 1u) wait_bounded(full(i), (armed_par >> i) & 1u, nullptr, nullptr, kDrainNs);
    }
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = instr_desc(N, true, true);
      int s = 0, b = 0;
      uint32_t ph = 0, dph = 0;
      bool ok = true;
      for (int64_t g = c0; ok && g < c1; g += kDwFlush) {
        const int64_t g1 = min(c1, g + kDwFlush);
        for (int64_t c = g; ok && c < g1; ++c) {
          ok = wait_bounded(full(s), ph, abort_s, p.err, lim);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sA = smem_u32(smem + s * SB), sB = sA + NA * 8192;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // columns 0-127 and 128-255 of the tile
            if (c == g) {
              ok = ok && wait_bounded(dempty(b, h), dph ^ 1u, abort_s, p.err, lim);
              if (!ok) break;
              tc_fence_after();
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16(tmem + acc_col(b, h), smem_desc(sA + h * 16384 + kk * 2048, 8192, 1024),
                       smem_desc(sB + kk * 2048, 8192, 1024), idesc, (c > g || kk > 0) ? 1u : 0u);
            if (c == g1 - 1) mma_commit(dfull(b, h));
          }
          if (!ok) break;
          mma_commit(empty(s));
          if (++s == kDwStages) { s = 0; ph ^= 1u; }
        }
        if (++b == BUFS) { b = 0; dph ^= 1u; }
      }
      mma_commit(done);
      wait_bounded(done, 0u, nullptr, nullptr, *abort_s ? kDrainNs : lim);
    }
    __syncwarp();
  } else {
    // ============================================================ sums
    // warp: 32 columns of x (its quarter of the TMEM lanes) of one 128-column half
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    float sum[EP];
#pragma unroll
    for (int e = 0; e < EP; ++e) sum[e] = 0.f;
    int b = 0;
    uint32_t dph = 0;
    for (int64_t g = c0; g < c1; g += kDwFlush) {
      if (!__all_sync(0xffffffffu, wait_bounded(dfull(b, half), dph, abort_s, p.err, lim))) break;
      tc_fence_after();
      const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)acc_col(b, half);
      if constexpr (EP == 16) {  // columns hi 0-15, mid 16-31, lo 32-47 (48-63: not used)
        uint32_t v[32], v2[32];
        MB_TMEM_LD32(at, v);
        MB_TMEM_LD32(at + 32, v2);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sum[i] += __uint_as_float(v[i]) + (__uint_as_float(v[16 + i]) + __uint_as_float(v2[i]));
      } else {
#pragma unroll
        for (int e0 = 0; e0 < EP; e0 += 32) {
          uint32_t v[32], v2[32];
          MB_TMEM_LD32(at + EP + e0, v);
          MB_TMEM_LD32(at + 2 * EP + e0, v2);
          tmem_wait_ld();
          float small[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) small[i] = __uint_as_float(v[i]) + __uint_as_float(v2[i]);
          MB_TMEM_LD32(at + e0, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[e0 + i] += __uint_as_float(v[i]) + small[i];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dempty(b, half));
      if (++b == BUFS) { b = 0; dph ^= 1u; }
    }
    const int m = m0 + half * 128 + quarter * 32 + lane;
    if (m < p.d) {
      float* dst = p.part + ((int64_t)split * p.d + m) * p.E + group * 64;
      const int n = min(EP, p.E - group * 64);
#pragma unroll
      for (int e = 0; e < EP; ++e)
        if (e < n) dst[e] = sum[e];
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free_512(tmem);
}

// dWr and dbias: the partial sums in their order.  A block takes 128 values
// of dWr (four a lane; d E is a multiple of 64), its warp i partials i, i + 8,
// ...; the last blocks take dbias, a lane a value.  A wait that ran out in the
// kernels before leaves NaN, not a number that looks like a gradient.
constexpr int kGrWarps = 8;
__global__ void __launch_bounds__(32 * kGrWarps) grad_reduce_kernel(const float* part, const float* part_b, int64_t n, int E,
                                                                    int S, int SB, const int32_t* err,
                                                                    float* __restrict__ dWr,
                                                                    float* __restrict__ dbias) {
  __shared__ float4 acc[kGrWarps][32];
  wait_for_prior();
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int64_t blocks = (n + 127) / 128;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool weights = blockIdx.x < blocks;
  const int64_t i = weights ? ((int64_t)blockIdx.x * 32 + lane) * 4 : ((int64_t)blockIdx.x - blocks) * 32 + lane;
  if (weights) {
    if (i < n) {
      // four in flight at a time, the last ones too
      for (int s0 = wp; s0 < S; s0 += 4 * kGrWarps) {
        float4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int s = s0 + u * kGrWarps;
          v[u] = s < S ? *reinterpret_cast<const float4*>(part + s * n + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          a.x += v[u].x; a.y += v[u].y; a.z += v[u].z; a.w += v[u].w;
        }
      }
    }
  } else if (i < E) {
#pragma unroll 8
    for (int s = wp; s < SB; s += kGrWarps) a.x += part_b[(int64_t)s * E + i];
  }
  acc[wp][lane] = a;
  __syncthreads();
  if (wp != 0 || i >= (weights ? n : E)) return;
  a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int q = 0; q < kGrWarps; ++q) {
    const float4 v = acc[q][lane];
    a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
  }
  if (*err) a.x = a.y = a.z = a.w = __int_as_float(0x7fc00000);
  if (!weights) {
    if (dbias) dbias[i] = a.x;
  } else {  // dWr itself may start on any float
    dWr[i] = a.x;
    dWr[i + 1] = a.y;
    dWr[i + 2] = a.z;
    dWr[i + 3] = a.w;
  }
}

int padded(int E) { return E <= 16 ? 16 : E <= 32 ? 32 : 64; }  // of a group
int groups_of(int E) { return E <= 64 ? 1 : 2; }

struct Plan {
  int groups, tiles, dw_splits, dx_tiles, dx_splits, tblocks;
  int64_t chunks, rows;  // chunks of a dWr split; tokens of a split_kernel block
  size_t dls, ws, part, part_b, err, bytes;  // offsets in the workspace
};
Plan plan_of(const moeblaze_shape& s) {
  Plan p;
  const int ep = padded(s.E);
  p.groups = groups_of(s.E);
  p.tiles = (s.d + kGCols - 1) / kGCols;
  const int64_t all = (s.L + kDwTokens - 1) / kDwTokens;
  int64_t S = std::max<int64_t>(1, sm_count() / (p.tiles * p.groups));
  S = std::min(S, all);
  p.chunks = (all + S - 1) / S;
  p.dw_splits = (int)((all + p.chunks - 1) / p.chunks);
  const int64_t tb = (s.L + kDxTokens - 1) / kDxTokens;
  p.dx_tiles = (s.d + dx_cols(p.groups) - 1) / dx_cols(p.groups);
  p.dx_splits = (int)std::min<int64_t>(std::max<int64_t>(1, sm_count() / p.dx_tiles), tb);
  p.rows = std::max<int64_t>(64, (s.L + 4 * sm_count() - 1) / (4 * sm_count()));
  p.tblocks = (int)((s.L + p.rows - 1) / p.rows);
  size_t o = 0;
  auto take = [&](size_t n) {
    const size_t at = o;
    o += align_up(n, 256);
    return at;
  };
  p.dls = take((size_t)s.L * p.groups * dl_width(ep) * 2);
  p.ws = take((size_t)s.d * p.groups * wr_width(ep) * 2);
  p.part = take((size_t)p.dw_splits * s.d * s.E * sizeof(float));
  p.part_b = take((size_t)p.tblocks * s.E * sizeof(float));
  p.err = take(sizeof(int32_t));
  p.bytes = o;
  return p;
}

template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kern)(Params...), int64_t grid, int block, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

template <int EP, int GROUPS>
moeblaze_status launch_ep(const moeblaze_shape& s, const void* x, const float* Wr, const float* dl, float* dWr,
                          float* dbias, void* dx, bool add, void* ws, cudaStream_t st) {
  const Plan pl = plan_of(s);
  char* w = static_cast<char*>(ws);
  auto* dls = reinterpret_cast<__nv_bfloat16*>(w + pl.dls);
  auto* wsp = reinterpret_cast<__nv_bfloat16*>(w + pl.ws);
  float* part_b = reinterpret_cast<float*>(w + pl.part_b);
  GParams p;
  memset(&p, 0, sizeof(p));
  p.L = s.L;
  p.d = s.d;
  p.E = s.E;
  p.groups = GROUPS;
  p.part = reinterpret_cast<float*>(w + pl.part);
  p.err = reinterpret_cast<int32_t*>(w + pl.err);
  int withhold = 0;
  fault_injection(&p.wait_ns, &withhold);
  if (p.wait_ns == 0) p.wait_ns = kTimeoutNs;

  const int wblocks = dx ? std::max(1, std::min(sm_count(), s.d / 16)) : 0;
  auto split = s.E % 4 == 0 && ((uintptr_t)Wr & 15) == 0 ? split_kernel<EP, 4> : split_kernel<EP, 2>;
  split<<<dim3((unsigned)(pl.tblocks + wblocks), GROUPS), kSplitThreads, 0, st>>>(dl, Wr, s.L, s.d, s.E, pl.rows, pl.tblocks, dls, wsp,
                                                                    part_b, p.err);
  MB_CUDA(cudaGetLastError());
  count_launch();
  if (dx) {
    if (!make_map(&p.tmA, dls, GROUPS * dl_width(EP), (uint64_t)s.L, 64, kDxTokens) ||
        !make_map(&p.tmB, wsp, GROUPS * wr_width(EP), (uint64_t)s.d, 64, 128) ||
        !make_map(&p.tmO, dx, (uint64_t)s.d, (uint64_t)s.L, 64, 32))
      return MOEBLAZE_ERR_CUDA;
    p.tiles = pl.dx_tiles;
    p.splits = pl.dx_splits;
    p.add = add ? 1 : 0;
    auto kern = dx_kernel<EP, GROUPS>;
    constexpr int smem = dx_smem(EP, GROUPS);
    MB_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    MB_CUDA(launch_after(kern, (int64_t)pl.dx_tiles * pl.dx_splits, kGThreads, smem, st, p));
    count_launch();
  }
  if (!make_map(&p.tmA, x, (uint64_t)s.d, (uint64_t)s.L, 64, kDwTokens) ||
      !make_map(&p.tmB, dls, GROUPS * dl_width(EP), (uint64_t)s.L, 64, kDwTokens))
    return MOEBLAZE_ERR_CUDA;
  p.tiles = pl.tiles;
  p.splits = pl.dw_splits;
  p.chunks = pl.chunks;
  MB_CUDA(cudaFuncSetAttribute(dwr_kernel<EP>, cudaFuncAttributeMaxDynamicSharedMemorySize, dw_smem(EP)));
  MB_CUDA(launch_after(dwr_kernel<EP>, (int64_t)pl.tiles * GROUPS * pl.dw_splits, kGThreads, dw_smem(EP), st, p));
  const int64_t n = (int64_t)s.d * s.E;
  MB_CUDA(launch_after(grad_reduce_kernel, (n + 127) / 128 + (s.E + 31) / 32, 32 * kGrWarps, 0, st, (const float*)p.part,
                       (const float*)part_b, n, (int)s.E, pl.dw_splits, pl.tblocks, (const int32_t*)p.err, dWr, dbias));
  count_launch(2);
  return MOEBLAZE_OK;
}

}  // namespace
}  // namespace tc

bool router_grad_tc(const moeblaze_shape& s) { return s.dtype == MOEBLAZE_BF16 && s.E <= 128 && s.L > 0; }

size_t router_grad_tc_ws_bytes(const moeblaze_shape& s) { return tc::plan_of(s).bytes; }

moeblaze_status launch_router_grad_tc(const moeblaze_shape& s, const void* x, const float* Wr, const float* dl, float* dWr,
                                      float* dbias, void* dx, bool add, void* ws, cudaStream_t st) {
  if (tc::groups_of(s.E) == 2) return tc::launch_ep<64, 2>(s, x, Wr, dl, dWr, dbias, dx, add, ws, st);
  switch (tc::padded(s.E)) {
    case 16: return tc::launch_ep<16, 1>(s, x, Wr, dl, dWr, dbias, dx, add, ws, st);
    case 32: return tc::launch_ep<32, 1>(s, x, Wr, dl, dWr, dbias, dx, add, ws, st);
  }
  return tc::launch_ep<64, 1>(s, x, Wr, dl, dWr, dbias, dx, add, ws, st);
}

}  // namespace moeblaze
