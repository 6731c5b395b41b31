// Expert products on 4-bit weights with group scales, for few tokens (the
// serving form of the layer): every used expert's weights are read once.
//
//   w[r][n] = q[r][n] s[r / group][n],  q in -8..7, s bf16
//   h[t,k]  = SiLU(x[t] W1_e) (* x[t] W2_e),  e = ids[t,k]
//   y[t]    = sum_k g[t,k] h[t,k] W3_e        (ids outside [0,E): empty slots)
//
// Bound by the HBM reads of the weights (0.5 + 2/group bytes each).  The
// products run on mma.sync m16n8k16 (bf16, fp32 accumulate): 16 output
// columns of the weights are the M rows, up to 8 tokens the N columns, so a
// weight is converted once for 8 tokens, in registers.  tcgen05 takes its
// operands from shared memory or TMEM: the converted weights would make a
// round trip of four times their packed size there for a product whose N is
// a handful of tokens.
//
// Packed layout of a matrix (E,R,N): tiles of 16 columns n, chunks of 64
// reduction rows r; a chunk is 512 bytes, 16 per lane, one 32-bit word per
// k16 step of the MMA.  Lane (g = lane / 4, t = lane % 4) holds columns g and
// g + 8 and, in step i, rows r0 = 32 (i / 2) + 8 t + 4 (i % 2) to r0 + 3 of
// the chunk (the MMA's reduction order is free as long as both operands use
// it): two steps cover 32 consecutive rows, the smallest group, and a lane's
// x fragment of them is 16 consecutive bytes.  In a word, nibbles i and i + 4
// are the halves of the i-th A register (rows r0, r0 + 1 of column g; the
// same of g + 8; rows r0 + 2, r0 + 3 of g; of g + 8), biased by 8: masked and
// or-ed with 0x4300 they are the bf16 numbers 128 + q + 8, exactly.  The sum
// over a group starts at -136 sum x (formed once per token and group when
// the token rows are staged), which takes the bias of all its terms off
// again: one accumulator start instead of a subtraction per weight.  The
// group's sum is fp32, and the scale is applied to it in fp32.
//
// h is rounded to bf16 between the two products, as the layer's own is: y is
// then off by 2.3e-3 of its norm, by 1.7e-3 with h exact.  Both ways to keep
// more of it were slower at 1, 16 and 61 tokens (42.8, 128 and 66.5 us): fp16
// operands with rows scaled by powers of two (45, 147, 85 us), and h as two
// bf16 parts in two MMAs (45, 147, 74 us).
//
// Scales: [E][N/16][R/128][8][128/group][2] bf16: column g's and g + 8's
// scales of 128 rows, the piece a warp reads at a time.
#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace moeblaze {
namespace {

constexpr int kQThreads = 512;
constexpr int kQWarps = kQThreads / 32;
// warps that share a unit's reduction rows: 4, or 1 where a unit has few (see team_of)
constexpr int kQTeam = 4;
// token columns of a pass, at most: two MMA column tiles (fewer where as many
// rows of the reduction's length do not fit shared memory: 12 at d 4096, group
// 128).  An expert with more pairs is passed over again, its weights read once
// more (from L2, where they fit):
// three or four tiles at once spill (64 tokens at d 4096, h 14336, 8 experts:
// 273 us against 263; 61 over 64 fine-grained experts 82 against 76).
constexpr int kQCols = 16;
constexpr int kQMaxTokens = 64;                    // tokens of one launch
constexpr int kQMaxPairs = kQMaxTokens * kMaxK;    // (token, slot) pairs of one launch
constexpr int kQSlices = 64;                       // slices of the down projection's reduction axis, at most
// What a launch computes.  A unit is two tiles, so that a token fragment
// serves two weight tiles: the same tile of W1 and W2 (GATED), or two
// neighbouring tiles of one matrix (SINGLE: SiLU experts' W1; DOWN: W3).
enum QMode : int { GATED = 0, SINGLE = 1, DOWN = 2 };
constexpr int kQDepth = 3;                         // entries of a warp's ring, each a 128-row piece of a unit
constexpr size_t kQSmem = 227 * 1024;
// list, counts, offsets, pass and weight prefixes, scan totals
constexpr size_t kQIntBytes = 4 * (kQMaxPairs + 4 * kMaxE + 2 + 3 * kQWarps);

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 4, 8 or 16 bytes
template <int BYTES>
__device__ __forceinline__ void cp_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the A registers of one k16 step from a packed word: 136 + q.  One
// three-input logic operation takes a nibble pair (left to itself the
// compiler makes it two, and the ALU pipe is what the products wait for).
__device__ __forceinline__ void unpack_word(uint32_t w, uint32_t (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(a[i]) : "r"(w >> (4 * i)), "r"(0x000F000Fu), "r"(0x43004300u));
}

// the last i < n with table[i] <= v (table[0] <= v).  Not inlined, as loops of
// the kernel's start are not unrolled: its code is read once, and from L2
__device__ __noinline__ int last_at_most(const int* table, int n, int v) {
  int lo = 0;
  while (n - lo > 1) {
    const int m = (lo + n) >> 1;
    if (table[m] <= v) lo = m;
    else n = m;
  }
  return lo;
}

// relative time of a unit whose segment has n token columns: one MMA column
// tile is hidden behind the weights' loads, two are not quite
__host__ __device__ __forceinline__ int pass_weight(int n) { return n <= 8 ? 10 : 13; }

// barrier of one team of warps (barrier 0 is the CTA's)
template <int TEAM>
__device__ __forceinline__ void team_sync(int team) {
  if constexpr (TEAM == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(TEAM * 32) : "memory");
}

// ------------------------------------------------------------------ layouts
template <typename T>
__global__ void int4_quantize_kernel(const T* __restrict__ W, int64_t EG, int group, int N, int8_t* __restrict__ q,
                                     __nv_bfloat16* __restrict__ scales) {
  // one thread per (expert, group, column); EG = E R / group
  const int64_t total = EG * N;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t eg = i / N, n = i % N, base = eg * group * N + n;
    float m = 0.f;
    for (int r = 0; r < group; ++r) {
      const float a = fabsf((float)W[base + (int64_t)r * N]);
      m = a > m || a != a ? a : m;  // a NaN stays: no number is above it
    }
    const __nv_bfloat16 sb = __float2bfloat16_rn(m / 7.f);
    const float s = __bfloat162float(sb);
    scales[i] = sb;
    for (int r = 0; r < group; ++r) {
      const float v = s > 0.f && s < INFINITY ? rintf((float)W[base + (int64_t)r * N] / s) : 0.f;
      q[base + (int64_t)r * N] = (int8_t)fminf(fmaxf(v, -8.f), 7.f);
    }
  }
}

// word i of the packed matrix: [E][N/16][R/64][32 lanes][4 steps]
__global__ void int4_pack_kernel(const int8_t* __restrict__ q, int64_t words, int R, int N,
                                 uint32_t* __restrict__ packed) {
  const int kc = R / 64, nt = N / 16;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < words; i += (int64_t)gridDim.x * blockDim.x) {
    const int step = (int)(i & 3), lane = (int)((i >> 2) & 31);
    int64_t r = i >> 7;
    const int chunk = (int)(r % kc);
    r /= kc;
    const int tile = (int)(r % nt);
    const int64_t e = r / nt;
    const int g = lane >> 2, t = lane & 3;
    const int8_t* src = q + (e * R + chunk * 64 + 32 * (step >> 1) + 8 * t + 4 * (step & 1)) * (int64_t)N + tile * 16 + g;
    uint32_t w = 0;
#pragma unroll
    for (int a = 0; a < 4; ++a)    // register a: rows 2 (a / 2), + 1 of column g + 8 (a % 2)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int v = src[(int64_t)(2 * (a >> 1) + b) * N + 8 * (a & 1)] + 8;
        w |= (uint32_t)(v & 15) << (4 * a + 16 * b);
      }
    packed[i] = w;
  }
}

// element i of the packed scales: [E][N/16][R/128][8][128/group][2]
__global__ void int4_pack_scales_kernel(const __nv_bfloat16* __restrict__ s, int64_t total, int RG, int N, int group,
                                        __nv_bfloat16* __restrict__ packed) {
  const int nt = N / 16, per = 128 / group;  // groups of a piece
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int hi = (int)(i & 1), j = (int)((i >> 1) % per), g = (int)(i / (2 * per)) & 7;
    int64_t r = i / (16 * per);
    const int piece = (int)(r % (RG / per));
    r /= RG / per;
    const int tile = (int)(r % nt);
    const int64_t e = r / nt;
    packed[i] = s[(e * RG + piece * per + j) * N + tile * 16 + g + 8 * hi];
  }
}

__global__ void int4_dequantize_kernel(const uint32_t* __restrict__ packed, const __nv_bfloat16* __restrict__ ps,
                                       int64_t total, int R, int N, int group, __nv_bfloat16* __restrict__ W) {
  const int kc = R / 64, nt = N / 16;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int n = (int)(i % N);
    const int64_t er = i / N;
    const int r = (int)(er % R);
    const int64_t e = er / R;
    const int tile = n >> 4, c = n & 15, g = c & 7, hi = c >> 3;
    const int chunk = r >> 6, t = (r >> 3) & 3, step = 2 * ((r >> 5) & 1) + ((r >> 2) & 1), a = 2 * ((r >> 1) & 1) + hi, b = r & 1;
    const uint32_t w = packed[((((e * nt + tile) * kc + chunk) * 32) + g * 4 + t) * 4 + step];
    const int q = (int)((w >> (4 * a + 16 * b)) & 15u) - 8;
    const int per = 128 / group;
    const float s = __bfloat162float(ps[(((e * nt + tile) * (int64_t)(R / 128) + (r >> 7)) * 8 + g) * 2 * per +
                                        2 * ((r & 127) / group) + hi]);
    W[i] = __float2bfloat16_rn((float)q * s);
  }
}

// ------------------------------------------------------------------ products
struct QParams {
  const __nv_bfloat16* src;  // rows of the token operand: x (row = pair / K) or h (row = pair)
  int64_t src_ld;
  const uint8_t* w[2];       // packed weights of the branches
  const uint8_t* s[2];       // their packed scales
  const int32_t* ids;
  int pairs, E, K;
  int R, N;                  // reduction length and output columns of the matrices
  int slices;                // slices of the reduction axis (DOWN; else 1), at most kQSlices
  int per, more;             // 128-row pieces of a slice: per + 1 in the first `more` slices, per in the others
  int cap;                   // token columns of one pass, and token rows that shared memory holds
  float inv_grid, inv_full, inv_nt;  // 1 / gridDim, 1 / the weight of a full pass, 1 / units of a segment
  __nv_bfloat16* H;          // GATED, SINGLE: h (pairs x N)
  float* part;               // DOWN: (slices x pairs x N)
};

// Work: segments (expert in use, pass of `cap` of its pairs, slice), each
// with N / 16 tiles of a pair of matrices or N / 32 pairs of tiles; the units
// are split by weight, contiguously, over the CTAs, and a CTA's units go round
// its teams of TEAM warps, which share a unit's reduction rows: with four a
// CTA's last round costs a quarter of a unit's time, and few units still keep
// every warp loading; with one no unit is too short to share.  A
// segment's token rows are staged in shared memory; the packed weights
// stream through a ring of cp.async pieces per warp, of which every lane
// reads back only the bytes it copied itself (no barrier), and which runs on
// across units and segments.  The team's sums meet in shared memory, in the
// order of its warps.
template <int MODE, int NTL, int GROUP, int TEAM>
__global__ void __launch_bounds__(kQThreads, 1) int4_product_kernel(const QParams p) {
  constexpr int PIECES = kQDepth, NB = 2;
  constexpr int SW = 128 / GROUP;                   // groups, and scale words of a column pair, in a piece
  constexpr int BRANCH = 1024 + 32 * SW;            // ring bytes of a piece of one tile: weights, scale words
  constexpr int ENTRY = NB * BRANCH;
  extern __shared__ __align__(16) uint8_t qsm[];
  int* list = reinterpret_cast<int*>(qsm + (size_t)kQWarps * PIECES * ENTRY);  // [pairs] by expert, ascending
  int* cnt = list + kQMaxPairs;                                                // [E]
  int* off = cnt + kMaxE;                                                      // [E]
  int* pre = off + kMaxE;                                                      // [E + 1] passes before expert e
  int* wpre = pre + kMaxE + 1;                                                 // [E + 1] the passes' weights before e
  int* tot = wpre + kMaxE + 1;                                                 // warp totals of the scans [3][16]
  float* swap = reinterpret_cast<float*>(qsm + (((size_t)kQWarps * PIECES * ENTRY + kQIntBytes + 15) & ~(size_t)15));
  uint8_t* xs = reinterpret_cast<uint8_t*>(swap + kQWarps * NB * 128);         // swap: [warps][NB][4][32]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tq = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the next kernel's CTAs may take freed SMs

  // ---- pairs by expert: thread i ranks pair i among its warp's pairs of the
  // same expert; per-warp counts (in the ring, which is still empty) order the warps
  {
    uint16_t* tbl = reinterpret_cast<uint16_t*>(qsm);  // [warps][E]
    for (int i = tid; i < kQWarps * p.E / 2; i += kQThreads) reinterpret_cast<uint32_t*>(tbl)[i] = 0u;
    int id = tid < p.pairs ? p.ids[tid] : -1;
    if ((unsigned)id >= (unsigned)p.E) id = -1;
    __syncthreads();
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (id >= 0 && rank == 0) tbl[warp * p.E + id] = (uint16_t)__popc(same);
    __syncthreads();
    int c = 0;
    if (tid < p.E) {
#pragma unroll 4
      for (int w = 0; w < kQWarps; ++w) {
        const int v = tbl[w * p.E + tid];
        tbl[w * p.E + tid] = (uint16_t)c;
        c += v;
      }
    }
    // inclusive scans over the experts of pairs, passes and the passes' weights
    const int full = c / p.cap, rest = c % p.cap;
    const int passes = full + (rest > 0), weight = full * pass_weight(p.cap) + (rest > 0 ? pass_weight(rest) : 0);
    int a = c, b = passes, q = weight;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ua = __shfl_up_sync(0xffffffffu, a, o), ub = __shfl_up_sync(0xffffffffu, b, o);
      const int uq = __shfl_up_sync(0xffffffffu, q, o);
      if (lane >= o) {
        a += ua;
        b += ub;
        q += uq;
      }
    }
    if (lane == 31) {
      tot[warp] = a;
      tot[kQWarps + warp] = b;
      tot[2 * kQWarps + warp] = q;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
      a += tot[w];
      b += tot[kQWarps + w];
      q += tot[2 * kQWarps + w];
    }
    if (tid < p.E) {
      cnt[tid] = c;
      off[tid] = a - c;
      pre[tid] = b - passes;
      wpre[tid] = q - weight;
      if (tid == p.E - 1) {
        pre[p.E] = b;
        wpre[p.E] = q;
      }
    }
    __syncthreads();
    if (id >= 0) list[off[id] + tbl[warp * p.E + id] + rank] = tid;
    __syncthreads();
  }

  const int nt = p.N / (MODE == GATED ? 16 : 32);  // units of a segment
  const int allp = p.R / 128;
  const int per_pass = p.slices * nt;
  // slice sl's first piece, and how many it has
  auto first_piece = [&](int sl) { return MODE == DOWN ? sl * p.per + min(sl, p.more) : 0; };
  auto pieces_of = [&](int sl) { return MODE == DOWN ? p.per + (sl < p.more ? 1 : 0) : allp; };
  // A segment: pass `pi` of expert e, slice sl; its tiles are the CTA's units
  // [base, end), counted from the CTA's first unit (base < 0 where another CTA
  // has its first tiles).  Integer divisions are kept out of this start: they
  // and a search per unit were 1 us of it.
  struct Seg {
    int id, base, end;  // id: e, 9 bits; pi, 10 bits (512 pairs at most); sl, 7 bits (kQSlices)
    __device__ int e() const { return id & 511; }
    __device__ int pi() const { return (id >> 9) & 1023; }
    __device__ int sl() const { return id >> 19; }
  };
  auto next_segment = [&](Seg& s) {
    s.base = s.end;
    s.end += nt;
    int e = s.e(), pi = s.pi(), sl = s.sl() + 1;
    if (sl == p.slices) {
      sl = 0;
      if (++pi == pre[e + 1] - pre[e]) {
        pi = 0;
        do ++e;
        while (e + 1 < p.E && pre[e + 1] == pre[e]);
      }
    }
    s.id = e | (pi << 9) | (sl << 19);
  };
  // This CTA's units: an even share of the weights.  Lanes 0 and 1 map the
  // share's ends, blockIdx W / gridDim of the total weight W, to units; a
  // CTA's end and the next one's start are the same computation, which never
  // decreases from one to the next.
  Seg start;
  int units;
  {
    const int W = wpre[p.E];
    const float at = (float)W * ((float)(blockIdx.x + (lane & 1)) * p.inv_grid);
    const int q = (int)at;
    int e = p.E, pi = 0, off0 = 0, first = pre[p.E] * per_pass;
    if (blockIdx.x + (lane & 1) < gridDim.x && q < W) {
      e = last_at_most(wpre, p.E, q);
      pi = min((int)((float)(q - wpre[e]) * p.inv_full), pre[e + 1] - pre[e] - 1);
      const int n = min(p.cap, cnt[e] - pi * p.cap);
      const float in = (at - (float)(wpre[e] + pi * pass_weight(p.cap))) / (float)pass_weight(n);
      off0 = min(per_pass, max(0, (int)(in * (float)per_pass)));
      first = (pre[e] + pi) * per_pass + off0;
    }
    // the slice and tile of unit off0 of the pass
    int sl = (int)((float)off0 * p.inv_nt);
    if (sl * nt > off0) --sl;
    if ((sl + 1) * nt <= off0) ++sl;
    units = __shfl_sync(0xffffffffu, first, 1) - __shfl_sync(0xffffffffu, first, 0);
    e = __shfl_sync(0xffffffffu, e, 0);
    pi = __shfl_sync(0xffffffffu, pi, 0);
    sl = __shfl_sync(0xffffffffu, sl, 0);
    start.base = -(__shfl_sync(0xffffffffu, off0, 0) - sl * nt);
    start.end = start.base + nt;
    const bool over = sl == p.slices;  // the share begins with the next pass
    if (over) {
      --sl;
      start.end = start.base;
    }
    start.id = e | (pi << 9) | (sl << 19);
    if (over && units > 0) next_segment(start);
  }
  if (units <= 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  // ---- the fetch head of this warp: unit, pieces left of it, addresses
  const uint32_t ring = saddr(qsm) + warp * PIECES * ENTRY + lane * 16;
  const uint32_t ring_s = saddr(qsm) + warp * PIECES * ENTRY + 1024 + g * 4 * SW;
  constexpr int TEAMS = kQWarps / TEAM;
  const int team = warp / TEAM, mate = warp % TEAM;
  // this warp's pieces of a unit of kp pieces: [share(kp, mate), share(kp, mate + 1))
  auto share = [&](int kp, int m) { return (int)((unsigned)(kp * m) / TEAM); };
  int fu = team, left = 0;
  Seg fseg = start;
  uint32_t fslot = 0;  // byte offset of the ring entry to fill
  const uint8_t* fw[NB];
  const uint8_t* fs[NB];
  auto fetch_unit = [&]() {
    int k0;
    // (a warp may have no piece of a short slice's units)
    for (;; fu += TEAMS) {
      if (fu >= units) return;
      while (fu >= fseg.end) next_segment(fseg);
      const int kp = pieces_of(fseg.sl());
      k0 = share(kp, mate);
      left = share(kp, mate + 1) - k0;
      if (left > 0) break;
    }
    const int tile = fu - fseg.base;
#pragma unroll
    for (int br = 0; br < NB; ++br) {
      const int64_t row = MODE == GATED ? (int64_t)fseg.e() * nt + tile : ((int64_t)fseg.e() * nt + tile) * 2 + br;
      const int64_t at = row * allp + first_piece(fseg.sl()) + k0;
      fw[br] = p.w[MODE == GATED ? br : 0] + at * 1024 + lane * 16;
      fs[br] = p.s[MODE == GATED ? br : 0] + at * (32 * SW) + g * (4 * SW);
    }
  };
  auto fetch = [&]() {
    if (left > 0) {
#pragma unroll
      for (int br = 0; br < NB; ++br) {
        cp16(ring + fslot + br * BRANCH, fw[br]);
        cp16(ring + fslot + br * BRANCH + 512, fw[br] + 512);
        if (tq == 0) cp_small<4 * SW>(ring_s + fslot + br * BRANCH, fs[br]);  // one lane of the column pair's four
        fw[br] += 1024;
        fs[br] += 32 * SW;
      }
      if (--left == 0) {
        fu += TEAMS;
        fetch_unit();
      }
    }
    cp_commit();
    fslot = fslot == (PIECES - 1) * ENTRY ? 0u : fslot + ENTRY;
  };
  fetch_unit();
#pragma unroll 1
  for (int i = 0; i < PIECES - 1; ++i) fetch();
  // everything so far reads the routing and the weights, which the caller
  // provides; the rows staged below are the kernel before's (the down
  // projection's: h)
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- segments
  // rows of the longest slice, 16 banks apart: 2 rows x 64 bytes of a fragment load do not conflict
  const int pitch = pieces_of(0) * 256 + 64;
  float* nsx = reinterpret_cast<float*>(xs + (size_t)p.cap * pitch);  // [groups][8 NTL]: -136 sum x
  uint32_t slot = 0;
  int u = team;
  for (Seg seg = start;; next_segment(seg)) {
    const int e = seg.e(), sl = seg.sl(), first = off[e] + seg.pi() * p.cap;
    const int n = min(p.cap, cnt[e] - seg.pi() * p.cap), kp = pieces_of(sl);
    const int k0 = share(kp, mate), k1 = share(kp, mate + 1);
    __syncthreads();  // every warp is done with the previous segment's rows
    // a warp per 1024 elements of a row: 8 elements a lane, four times, all
    // in flight together; their sums meet over the GROUP / 8 lanes of a group
    {
      const int m = kp * 16, parts = (m + 127) / 128;  // m is a multiple of 16
#pragma unroll 1
      for (int i = warp; i < n * parts; i += kQWarps) {
        const int r = i / parts, c0 = (i - r * parts) * 128;
        const int pair = list[first + r];
        const int64_t row = MODE == DOWN ? pair : pair / p.K;
        const uint4* src = reinterpret_cast<const uint4*>(p.src + row * p.src_ld + (int64_t)first_piece(sl) * 128);
        uint4* dst = reinterpret_cast<uint4*>(xs + (size_t)r * pitch);
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = c0 + 32 * j + lane;
          v[j] = c < m ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = c0 + 32 * j + lane;
          const float2 a0 = unpack_bf16x2(v[j].x), a1 = unpack_bf16x2(v[j].y), a2 = unpack_bf16x2(v[j].z),
                       a3 = unpack_bf16x2(v[j].w);
          float t = ((a0.x + a0.y) + (a1.x + a1.y)) + ((a2.x + a2.y) + (a3.x + a3.y));
#pragma unroll
          for (int o = 1; o < GROUP / 8; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
          if (c < m) {
            dst[c] = v[j];
            if (lane % (GROUP / 8) == 0) nsx[(c / (GROUP / 8)) * (8 * NTL) + r] = -136.f * t;
          }
        }
      }
    }
    __syncthreads();
    const int send = min(seg.end, units);
    // the segment's units of this team, for T tiles of 8 token columns
    auto run_units = [&](auto tiles) {
      constexpr int T = decltype(tiles)::value;
      // fragment rows; columns past n repeat the last token: no column of the
      // product sees another, and those are not stored
      const uint8_t* xrow[T];
#pragma unroll
      for (int i = 0; i < T; ++i) xrow[i] = xs + (size_t)min(8 * i + g, n - 1) * pitch + tq * 16;
      const float* sums = nsx + 2 * tq;
      for (; u < send; u += TEAMS) {
        float acc[NB][T][4];
#pragma unroll
        for (int br = 0; br < NB; ++br)
#pragma unroll
          for (int i = 0; i < T; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[br][i][v] = 0.f;
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
          cp_wait<PIECES - 2>();
          __syncwarp();  // the scales are another lane's copies
          uint4 wv[NB][2];
          uint32_t sc[NB][SW];
#pragma unroll
          for (int br = 0; br < NB; ++br) {
            const uint8_t* at = qsm + warp * PIECES * ENTRY + slot + br * BRANCH;
            wv[br][0] = *reinterpret_cast<const uint4*>(at + lane * 16);
            wv[br][1] = *reinterpret_cast<const uint4*>(at + 512 + lane * 16);
#pragma unroll
            for (int j = 0; j < SW; ++j) sc[br][j] = reinterpret_cast<const uint32_t*>(at + 1024)[g * SW + j];
          }
          slot = slot == (PIECES - 1) * ENTRY ? 0u : slot + ENTRY;
          fetch();
          float part[NB][T][4];
#pragma unroll
          for (int hw = 0; hw < 4; ++hw) {  // 32 rows: two words of a lane, 16 bytes of a token
            if ((hw * 32) % GROUP == 0) {
#pragma unroll
              for (int i = 0; i < T; ++i) {
                const float2 s2 =
                    *reinterpret_cast<const float2*>(sums + (k * SW + hw * 32 / GROUP) * (8 * NTL) + 8 * i);
#pragma unroll
                for (int br = 0; br < NB; ++br) {
                  part[br][i][0] = part[br][i][2] = s2.x;
                  part[br][i][1] = part[br][i][3] = s2.y;
                }
              }
            }
            uint4 xv[T];
#pragma unroll
            for (int i = 0; i < T; ++i) xv[i] = *reinterpret_cast<const uint4*>(xrow[i] + k * 256 + hw * 64);
#pragma unroll
            for (int br = 0; br < NB; ++br) {
              const uint4 w4 = wv[br][hw >> 1];
              uint32_t A[4];
              unpack_word((hw & 1) ? w4.z : w4.x, A);
#pragma unroll
              for (int i = 0; i < T; ++i) mma16816(part[br][i], A, xv[i].x, xv[i].y);
              unpack_word((hw & 1) ? w4.w : w4.y, A);
#pragma unroll
              for (int i = 0; i < T; ++i) mma16816(part[br][i], A, xv[i].z, xv[i].w);
              if (((hw + 1) * 32) % GROUP == 0) {
                const float2 s = unpack_bf16x2(sc[br][hw * 32 / GROUP]);
#pragma unroll
                for (int i = 0; i < T; ++i) {
                  acc[br][i][0] = fmaf(part[br][i][0], s.x, acc[br][i][0]);
                  acc[br][i][1] = fmaf(part[br][i][1], s.x, acc[br][i][1]);
                  acc[br][i][2] = fmaf(part[br][i][2], s.y, acc[br][i][2]);
                  acc[br][i][3] = fmaf(part[br][i][3], s.y, acc[br][i][3]);
                }
              }
            }
          }
        }
        // ---- the team's sums of 8 token columns at a time: accumulator v of
        // a lane is column n = 16 tile + g + 8 (v / 2), token 8 i + 2 tq + v % 2;
        // warp v of the team adds up and stores accumulator v (one warp: all four)
#pragma unroll
        for (int i = 0; i < T; ++i) {
          if (i > 0) team_sync<TEAM>(team);  // the tile before is read
#pragma unroll
          for (int br = 0; br < NB; ++br)
#pragma unroll
            for (int v = 0; v < 4; ++v) swap[((warp * NB + br) * 4 + v) * 32 + lane] = acc[br][i][v];
          team_sync<TEAM>(team);
#pragma unroll
          for (int v = mate; v < 4; v += TEAM) {
            float sum[NB];
#pragma unroll
            for (int br = 0; br < NB; ++br) {
              sum[br] = 0.f;
#pragma unroll
              for (int w = 0; w < TEAM; ++w) sum[br] += swap[(((team * TEAM + w) * NB + br) * 4 + v) * 32 + lane];
            }
            const int tk = 8 * i + 2 * tq + (v & 1), unit = u - seg.base;
            if (tk >= n) continue;
            const int pair = list[first + tk];
            const int64_t at = (int64_t)(MODE == DOWN ? sl * p.pairs + pair : pair) * p.N;
            if constexpr (MODE == GATED) {
              const float hv = sum[0] / (1.f + expf(-sum[0])) * sum[1];
              p.H[at + unit * 16 + g + 8 * (v >> 1)] = __float2bfloat16_rn(hv);
            } else {
#pragma unroll
              for (int br = 0; br < NB; ++br) {
                const int64_t o = at + (unit * 2 + br) * 16 + g + 8 * (v >> 1);
                if constexpr (MODE == SINGLE) p.H[o] = __float2bfloat16_rn(sum[br] / (1.f + expf(-sum[br])));
                else p.part[o] = sum[br];
              }
            }
          }
        }
        team_sync<TEAM>(team);  // the last tile is read before the next unit's sums overwrite it
      }
    };
    if (NTL == 1 || n <= 8) run_units(std::integral_constant<int, 1>());
    else run_units(std::integral_constant<int, NTL>());
    if (seg.end >= units) break;
  }
  cp_wait<0>();
}

// y[t] = sum_k g[t,k] sum_slices part, in that order; KM slots (K <= KM) of
// kMaxK / KM slices in flight together
template <int KM>
__global__ void int4_combine_kernel(const float* part, const int32_t* __restrict__ ids,
                                    const float* __restrict__ gates, int L, int d, int E, int K, int slices,
                                    __nv_bfloat16* __restrict__ y) {
  constexpr int U = kMaxK / KM;
  const int64_t total = (int64_t)L * d / 4;
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int t = (int)(i / (d / 4)), c = (int)(i % (d / 4)) * 4;
  // the routing is the caller's: read while the products still run
  float g[KM];
  bool on[KM];
#pragma unroll
  for (int k = 0; k < KM; ++k) {
    on[k] = i < total && k < K && (unsigned)ids[t * K + k] < (unsigned)E;
    g[k] = on[k] ? gates[t * K + k] : 0.f;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (i >= total) return;
  float4 v[KM];
#pragma unroll
  for (int k = 0; k < KM; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* src = part + (int64_t)t * K * d + c;
  const int64_t slice = (int64_t)L * K * d;
  for (int s = 0; s < slices; s += U, src += U * slice) {
    float4 q[U][KM];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < KM; ++k) {
        q[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on[k] && s + u < slices) q[u][k] = *reinterpret_cast<const float4*>(src + u * slice + (int64_t)k * d);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < KM; ++k) {
        v[k].x += q[u][k].x; v[k].y += q[u][k].y; v[k].z += q[u][k].z; v[k].w += q[u][k].w;
      }
  }
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < KM; ++k) {
    if (!on[k]) continue;  // (an empty slot's gate may be anything)
    o.x = fmaf(g[k], v[k].x, o.x); o.y = fmaf(g[k], v[k].y, o.y);
    o.z = fmaf(g[k], v[k].z, o.z); o.w = fmaf(g[k], v[k].w, o.w);
  }
  *reinterpret_cast<uint2*>(y + (int64_t)t * d + c) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}

// shared memory besides the token rows: ring, routing, the teams' sums
size_t fixed_bytes(int group) {
  return align_up((size_t)kQWarps * kQDepth * 2 * (1024 + 32 * (128 / group)) + kQIntBytes, 16) +
         (size_t)kQWarps * 2 * 128 * sizeof(float);
}
// token columns are padded to whole MMAs in the table of group sums
int pad_cols(int cols) { return cols <= 8 ? 8 : 16; }
size_t token_bytes(int64_t len, int group, int rows) {
  return (size_t)rows * (len * 2 + 64) + (size_t)(len / group) * pad_cols(rows) * sizeof(float);
}

// token columns of one pass over an expert: up to 16, as many rows of `len`
// elements as shared memory holds
int pass_cap(int64_t len, int group) {
  int rows = kQCols;
  while (rows > 0 && fixed_bytes(group) + token_bytes(len, group, rows) > kQSmem) --rows;
  return rows;
}

// The time of `units` units of `pieces` 128-row pieces on the GPU, in pieces,
// with teams of `team` warps: a CTA's rounds, each a warp's pieces and about
// one more for its start and end.
int64_t team_cost(int64_t units, int pieces, int team) {
  const int64_t per_cta = (units + sm_count() - 1) / sm_count(), teams = kQWarps / team;
  return (per_cta + teams - 1) / teams * ((pieces + team - 1) / team + 1);
}
// One warp a unit where that is reckoned a fifth faster and has two rounds at
// least: units of a few pieces, which four warps cannot share evenly.  (d 640,
// h 11520, 47 experts, 42 tokens: 134 against 167 us; d 128, h 14336: 52 against
// 79.  Everywhere: 134 against 118 us at d 4096, h 14336, 16 tokens.)
int team_of(int64_t units, int pieces) {
  return units >= 2 * kQWarps * sm_count() && 5 * team_cost(units, pieces, 1) < 4 * team_cost(units, pieces, kQTeam)
             ? 1
             : kQTeam;
}

// Slices of the down projection's reduction axis (whole 128-row pieces): the
// teams' rounds times a warp's pieces of a unit, plus about a piece's time a
// round for its start and end; slices whose token rows fit shared memory for
// the usual load (16 tokens of an expert) only, unless the most there may be do
// not.  Slices of one length, but where these come to more than kQEven (h / 128
// has no divisor that fits) the first slices have a piece more than the others:
// d 4096, 8 experts, K 2, 16 tokens, h 11008 in 4 slices against 43 of two pieces
// 105 and 133 us, h 13696 in 7 against 107 of one 127 and 214 us.
constexpr int kQEven = 16;
int most_slices(const moeblaze_shape& s) { return std::min(s.h / 128, kQSlices); }
int64_t slice_len(const moeblaze_shape& s, int n) { return 128 * (int64_t)((s.h / 128 + n - 1) / n); }
int down_slices(const moeblaze_shape& s, int group, int tokens) {
  const int most = most_slices(s);
  const int64_t used = std::min<int64_t>(s.E, (int64_t)tokens * s.K);
  int best = most;
  int64_t least = INT64_MAX;
  auto look = [&](int n) {
    const int64_t len = slice_len(s, n);
    if (n < most && pass_cap(len, group) < std::min(tokens, 16)) return;
    const int64_t cost = team_cost(used * (s.d / 32) * n, (int)(len / 128), kQTeam);
    if (cost < least) {
      least = cost;
      best = n;
    }
  };
  for (int n = 1; n <= most; ++n)
    if (s.h / 128 % n == 0) look(n);
  if (best > kQEven)
    for (int n = 1; n <= most; ++n) look(n);
  return best;
}

size_t h_bytes(const moeblaze_shape& s, int tokens) {
  return align_up((size_t)tokens * s.K * s.h * 2, 256);
}

// `early`: the kernel may start while the one before it in the stream ends
// (it waits for it, griddepcontrol.wait, before it touches its results)
template <typename... Params, typename... Args>
cudaError_t launch_q(void (*kern)(Params...), unsigned grid, unsigned block, size_t smem, bool early, cudaStream_t st,
                     Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

template <int MODE, int GROUP>
moeblaze_status launch_product_g(QParams p, int tokens, cudaStream_t st) {
  const int pieces = p.R / 128;
  p.per = pieces / p.slices;
  p.more = pieces % p.slices;
  const int64_t len = 128 * (int64_t)(p.per + (p.more > 0));  // of the longest slice
  // (no more columns than tokens, although a token that names an expert twice
  // gives it more pairs than there are tokens: the rest is another pass)
  p.cap = std::min(pass_cap(len, GROUP), tokens);
  p.inv_grid = 1.f / (float)sm_count();
  p.inv_full = 1.f / (float)pass_weight(p.cap);
  p.inv_nt = 1.f / (float)(p.N / (MODE == GATED ? 16 : 32));
  const int team = team_of(std::min<int64_t>(p.E, p.pairs) * p.slices * (p.N / (MODE == GATED ? 16 : 32)), (int)(len / 128));
  const size_t sm = fixed_bytes(GROUP) + token_bytes(len, GROUP, p.cap);
  auto run = [&](auto kern) -> moeblaze_status {
    MB_CUDA(smem_limit(kern, kQSmem));
    // the down projection's h comes from the launch before it, its routing and weights from before that
    MB_CUDA(launch_q(kern, (unsigned)sm_count(), kQThreads, sm, MODE == DOWN, st, p));
    count_launch();
    return MOEBLAZE_OK;
  };
  if (team == 1)
    return p.cap <= 8 ? run(int4_product_kernel<MODE, 1, GROUP, 1>) : run(int4_product_kernel<MODE, 2, GROUP, 1>);
  return p.cap <= 8 ? run(int4_product_kernel<MODE, 1, GROUP, kQTeam>) : run(int4_product_kernel<MODE, 2, GROUP, kQTeam>);
}

template <int MODE>
moeblaze_status launch_product(const QParams& p, int group, int tokens, cudaStream_t st) {
  switch (group) {
    case 32: return launch_product_g<MODE, 32>(p, tokens, st);
    case 64: return launch_product_g<MODE, 64>(p, tokens, st);
  }
  return launch_product_g<MODE, 128>(p, tokens, st);
}

}  // namespace

bool int4_shape_ok(const moeblaze_shape& s, int group) {
  return pass_cap(s.d, group) >= 1 && pass_cap(slice_len(s, most_slices(s)), group) >= 1;
}

size_t int4_ws_bytes(const moeblaze_shape& s, int group) {
  const int tokens = (int)std::min<int64_t>(s.L, kQMaxTokens);
  if (tokens == 0) return 0;
  // the slices depend on the tokens of a launch: the last one may have fewer
  size_t most = 0;
  for (const int t : {tokens, (int)(s.L % kQMaxTokens)}) {
    if (t == 0) continue;
    most = std::max(most, (size_t)down_slices(s, group, t) * t * s.K * s.d * sizeof(float));
  }
  return h_bytes(s, tokens) + align_up(most, 256);
}

moeblaze_status launch_int4_forward(const moeblaze_shape& s, const __nv_bfloat16* x, const int32_t* ids,
                                    const float* gates, const moeblaze_int4_experts& w, __nv_bfloat16* y, void* ws,
                                    cudaStream_t st) {
  for (int64_t t0 = 0; t0 < s.L; t0 += kQMaxTokens) {
    const int tokens = (int)std::min<int64_t>(s.L - t0, kQMaxTokens);
    __nv_bfloat16* H = static_cast<__nv_bfloat16*>(ws);
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + h_bytes(s, (int)std::min<int64_t>(s.L, kQMaxTokens)));
    const bool sw = s.act == MOEBLAZE_SWIGLU;
    QParams p = {};
    p.src = x + t0 * s.d;
    p.src_ld = s.d;
    p.w[0] = static_cast<const uint8_t*>(w.w1);
    p.s[0] = static_cast<const uint8_t*>(w.s1);
    p.w[1] = static_cast<const uint8_t*>(w.w2);
    p.s[1] = static_cast<const uint8_t*>(w.s2);
    p.ids = ids + t0 * s.K;
    p.pairs = tokens * s.K;
    p.E = s.E;
    p.K = s.K;
    p.R = s.d;
    p.N = s.h;
    p.slices = 1;
    p.H = H;
    moeblaze_status r = sw ? launch_product<GATED>(p, w.group, tokens, st) : launch_product<SINGLE>(p, w.group, tokens, st);
    if (r != MOEBLAZE_OK) return r;
    p.src = H;
    p.src_ld = s.h;
    p.w[0] = static_cast<const uint8_t*>(w.w3);
    p.s[0] = static_cast<const uint8_t*>(w.s3);
    p.R = s.h;
    p.N = s.d;
    p.slices = down_slices(s, w.group, tokens);
    p.H = nullptr;
    p.part = part;
    if ((r = launch_product<DOWN>(p, w.group, tokens, st)) != MOEBLAZE_OK) return r;
    const int64_t n = (int64_t)tokens * s.d / 4;
    auto combine = s.K <= 2 ? int4_combine_kernel<2> : int4_combine_kernel<kMaxK>;
    MB_CUDA(launch_q(combine, (unsigned)((n + 127) / 128), 128, 0, true, st, (const float*)part,
                     ids + t0 * s.K, gates + t0 * s.K, tokens, (int)s.d, (int)s.E, (int)s.K, p.slices, y + t0 * s.d));
    count_launch();
  }
  return MOEBLAZE_OK;
}

namespace {
unsigned flat_grid(int64_t n) {
  int64_t b = (n + 255) / 256;
  if (b > 32 * (int64_t)sm_count()) b = 32 * (int64_t)sm_count();
  return (unsigned)b;
}
}  // namespace

moeblaze_status launch_int4_quantize(int E, int R, int N, int group, int dtype, const void* W, int8_t* q, void* scales,
                                     cudaStream_t st) {
  const int64_t eg = (int64_t)E * (R / group);
  if (dtype == MOEBLAZE_BF16)
    int4_quantize_kernel<<<flat_grid(eg * N), 256, 0, st>>>(static_cast<const __nv_bfloat16*>(W), eg, group, N, q,
                                                            static_cast<__nv_bfloat16*>(scales));
  else
    int4_quantize_kernel<<<flat_grid(eg * N), 256, 0, st>>>(static_cast<const float*>(W), eg, group, N, q,
                                                            static_cast<__nv_bfloat16*>(scales));
  MB_CUDA(cudaGetLastError());
  count_launch();
  return MOEBLAZE_OK;
}

moeblaze_status launch_int4_pack(int E, int R, int N, int group, const int8_t* q, const void* scales, void* packed,
                                 void* packed_scales, cudaStream_t st) {
  const int64_t words = (int64_t)E * R * N / 8, ns = (int64_t)E * (R / group) * N;
  int4_pack_kernel<<<flat_grid(words), 256, 0, st>>>(q, words, R, N, static_cast<uint32_t*>(packed));
  MB_CUDA(cudaGetLastError());
  int4_pack_scales_kernel<<<flat_grid(ns), 256, 0, st>>>(static_cast<const __nv_bfloat16*>(scales), ns, R / group, N,
                                                         group, static_cast<__nv_bfloat16*>(packed_scales));
  MB_CUDA(cudaGetLastError());
  count_launch(2);
  return MOEBLAZE_OK;
}

moeblaze_status launch_int4_dequantize(int E, int R, int N, int group, const void* packed, const void* packed_scales,
                                       void* W, cudaStream_t st) {
  const int64_t n = (int64_t)E * R * N;
  int4_dequantize_kernel<<<flat_grid(n), 256, 0, st>>>(static_cast<const uint32_t*>(packed),
                                                       static_cast<const __nv_bfloat16*>(packed_scales), n, R, N, group,
                                                       static_cast<__nv_bfloat16*>(W));
  MB_CUDA(cudaGetLastError());
  count_launch();
  return MOEBLAZE_OK;
}

}  // namespace moeblaze
