// The experts' products on 8-bit floating-point weights, for prompts, on the
// sm_103a tensor cores (tcgen05 + TMEM, operands by TMA).
//
//   A = x W1, B = x W2      x rows e4m3 with a scale sx for each row and 128
//   H = SiLU(A) B           columns, W e4m3 with a scale for each 128 x 128
//   Y = H8 W3               H8: H in 8-bit rows (eight.cuh)
//
// With the reduction cut into blocks of 128, where the scales are constant,
//   A[q][n] = sum_kb (sx[q][kb] s1[n/128][kb]) sum_{k in kb} x8[q][k] w8[n][k]
// The inner sums are what the tensor cores give (products of e4m3 are exact,
// and 128 of them are added in TMEM); the outer one is fp32 in registers.
//
// Two CTAs on two SMs make a 256 x 256 tile (tcgen05.mma.cta_group::2): each
// stages its 128 rows and one half of the weights' 256, so a block of the
// reduction brings 32 KB to an SM for 8.4 MFLOP; one CTA with a 128 x 256 tile
// would take 48 KB, and what L2 delivers to the SMs is what bounds such tiles.
// Each block of the reduction goes to one of two TMEM accumulators of 256
// columns, which eight warps read back, scale and add to their registers (128
// a thread) while the other one is computed: 512 cycles of tensor pipe beside
// 256 of TMEM reads and 128 of packed FMAs.
//
// Measured: 8192 tokens, d 4096, h 14336, 2 of 8: up 1.60 and down 0.73 ms (2.41
// and 2.64 PFLOP/s; 1.9 is the bf16 peak of a plain product), 2.42 ms in all, 2.58
// to 2.64 in runs that last (the power cap); d 2048, h 1408, 6 of 64, 16000 tokens
// 1.02 to 1.06 ms.  The tensor pipe is busy for half
// of the time: a block takes 800 to 950 cycles, from the MMAs' end over the commit,
// the reads of TMEM and the arrivals on the other SM to the next MMAs into that
// accumulator.  (With half of each accumulator read, which is wrong, 2.8 PFLOP/s.)
// Tried for it: the scaling threads loading their own scales (5.9 ms in all);
// releasing arrivals at cluster scope (9.2); 16 scaling warps of 64 accumulators
// (2.9 to 3.1, spills); four accumulators of 128 columns (3.2 to 4.3: an MMA of
// half the columns is not twice as fast); the next tile's scales loaded before the
// epilogue (2.66); five stages, other groups of tiles: no difference.
//
//   warp 0        producer: TMA loads of both operands (each CTA its own; all of
//                 a stage's loads complete on rank 0's barrier)
//   warp 1        TMEM allocation; in rank 0 the MMA issuer
//   warps 4-11    scaling: a row a thread, 64 columns of A and 64 of B (SwiGLU)
//                 or 128 columns; then the tile's epilogue
// The first warpgroup gives registers to the others (setmaxnreg: 40 + 2 x 232 a
// thread, of 3 x 168 at launch).
//
// Row space: an expert's rows are a segment of a padded row space, 256-row
// aligned (fp8.cu); padding rows hold anything, and what they give is not read.
// Every wait is bounded; on expiry the CTA sets the error word, and the combine
// step answers with NaN.
#include "common.cuh"
#include "eight.cuh"
#include "fp8.cuh"
#include "tc_ptx.cuh"

namespace moeblaze {
namespace fp8 {

using namespace tc;

constexpr int BM = 128, BK = 128;              // rows of a CTA; a block of the reduction: 128 bytes a row
constexpr int TILE_BYTES = BM * BK;            // 16 KB of either operand
constexpr int STAGES = 6;
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int SCALE_WARPS = 8;
constexpr int THREADS = 128 + 32 * SCALE_WARPS;
constexpr int TMEM_COLS = 512;
constexpr int XCHG_BYTES = 2 * 2 * BM * 4;     // largest magnitudes of a row's two parts, of two tiles in turn
// A block's row scales come with its stage, but are read when its sums are: they
// have a ring of their own.  The scaling warps release the stages in turn, so that
// the loads of block i, which wait for the releases up to block i - STAGES, come
// after one of every warp at block i - STAGES - SCALE_WARPS + 1 or later: an ordered
// arrival (at the CTA's own barrier) behind its reads of all blocks before that.
// (One warp releasing every stage, which leaves the other warps' reads ordered by
// relaxed arrivals alone: 2.38 in place of 2.42 ms.)
constexpr int SLOTS = 16;
static_assert(SLOTS >= STAGES + SCALE_WARPS && SLOTS % SCALE_WARPS == 0, "row scales are read before they are replaced");
constexpr int SCALE_BYTES = SLOTS * BM * 4;
constexpr int SMEM = STAGES * STAGE_BYTES + SCALE_BYTES + XCHG_BYTES + 1024 + 256;

enum Mode : int { UP_SWIGLU = 0, UP_SILU, DOWN };

struct Params {
  CUtensorMap tmA;   // rows (rows, R) bytes
  CUtensorMap tmB0;  // packed weights
  CUtensorMap tmB1;  // W2 (SwiGLU)
  CUtensorMap tmS;   // rows' scales (R/128, rows) fp32
  const int32_t* hdr;
  const int32_t* tile_e;
  int32_t* err;
  const float* s0;   // weights' scales (E, N/128, R/128)
  const float* s1;
  uint8_t* h8;       // up: H8 (rows, N)
  float* sh;         // scales of H8 or y (N/128, rows)
  __half* y;         // down: (rows, N)
  int64_t rows;
  int N, kblocks, n_tiles;
  uint64_t wait_ns;
  int withhold;      // test of the failure path (down): a CTA's first stage is never loaded
};

// the copy lands in this CTA's shared memory and completes `bar`, which may be
// the other CTA's (a shared::cluster address)
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// Arrivals at a barrier of either CTA.  Relaxed: what they announce is a request
// for bytes, or TMEM reads that have returned (tcgen05.wait::ld); a release at
// cluster scope would wait for the thread's other memory operations as well.  They
// order no reads or writes of shared memory.
__device__ __forceinline__ void arrive_expect_pair(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void arrive_pair(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// An arrival at a barrier of this CTA, ordered behind the thread's reads; with a
// predicate, since a branch around it costs the scaling loop 4 to 6 % more.
__device__ __forceinline__ void arrive_if(uint32_t bar, bool on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar), "r"(on ? 1u : 0u)
      : "memory");
}
// e4m3 x e4m3 -> fp32, 256 x 256 over the pair, both operands K-major
constexpr uint32_t kIdesc = (1u << 4) | (256u >> 3 << 17) | (256u >> 4 << 24);
__device__ __forceinline__ void mma_pair(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(kIdesc), "r"(accum)
      : "memory");
}
// arrive on `bar` (a shared::cluster address) once the MMAs so far are done
__device__ __forceinline__ void commit_at(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
struct Tile {
  int e, row0, n0;  // row0: of the pair's 256 rows
};
__device__ __forceinline__ Tile decode(const Params& p, int tile, int num_mt) {
  // groups of 8 row tiles walk the weights together, so that what they share stays in L2
  constexpr int GM = 8;
  const int per_g = GM * p.n_tiles, g = tile / per_g, r = tile - g * per_g;
  const int gm = min(GM, num_mt - g * GM), mt = g * GM + r % gm;
  Tile t;
  t.e = p.tile_e[mt];
  t.row0 = mt * 256;
  t.n0 = r / gm;
  return t;
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) fp8_gemm_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES);      // [slot][row]
  uint32_t* xchg = reinterpret_cast<uint32_t*>(smem + STAGES * STAGE_BYTES + SCALE_BYTES);  // [tile parity][part][row]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES + SCALE_BYTES + XCHG_BYTES);
  // full[S], empty[S], tmem_full[2], tmem_empty[2], drain, exchange
  constexpr int B_FULL = 0, B_EMPTY = STAGES, B_TFULL = 2 * STAGES, B_TEMPTY = 2 * STAGES + 2, B_DRAIN = 2 * STAGES + 4,
                B_XCHG = 2 * STAGES + 5;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 6);
  volatile int* abort_s = reinterpret_cast<volatile int*>(bars + 2 * STAGES + 7);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t rank = cluster_rank();
  auto bar = [&](int i) { return smem_u32(bars + i); };
  auto lead = [&](int i) { return peer_addr(bar(i), 0); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar(B_FULL + s), 2);    // both CTAs' producers
      mbar_init(bar(B_EMPTY + s), 1);   // one of the scaling warps, in turn, that has seen the stage's MMAs end
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(B_TFULL + b), 1);
      mbar_init(bar(B_TEMPTY + b), 2 * SCALE_WARPS);
    }
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_XCHG), 32 * SCALE_WARPS);
    *abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before anything arrives from the other
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int num_mt = p.hdr[1];
  const int total = num_mt * p.n_tiles;
  const int first = blockIdx.x / 2, step = gridDim.x / 2;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0 && lane == 0) {
      // ================================================================ producer
      int s = 0, slot = 0;
      uint32_t ph = 0, used = 0;
      bool ok = true;
      for (int tile = first; ok && tile < total; tile += step) {
        const Tile t = decode(p, tile, num_mt);
        const CUtensorMap* mb = MODE == UP_SWIGLU && rank ? &p.tmB1 : &p.tmB0;
        const int arow = t.row0 + (int)rank * BM;
        // (past the last block of a matrix lies the next one's, or nothing: what it gives is not kept)
        const int64_t blk = (int64_t)t.e * (p.N / 128) + (MODE == UP_SWIGLU ? t.n0 : t.n0 * 2 + (int)rank);
        const int brow = (int)(blk * p.kblocks * 128);
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!(ok = wait_bounded(bar(B_EMPTY + s), ph ^ 1u, abort_s, p.err, p.wait_ns))) break;
          const uint32_t full = lead(B_FULL + s), dst = smem_base + s * STAGE_BYTES;
          if (!(MODE == DOWN && p.withhold && tile == first && kb == 0)) {
            arrive_expect_pair(full, STAGE_BYTES + BM * 4);
            tma_load_pair(dst, &p.tmA, kb * BK, arow, full);
            tma_load_pair(dst + TILE_BYTES, mb, 0, brow + kb * 128, full);
            tma_load_pair(smem_u32(scales + slot * BM), &p.tmS, arow, kb, full);
            used |= 1u << s;
          }
          slot = slot == SLOTS - 1 ? 0 : slot + 1;
          if (++s == STAGES) { s = 0; ph ^= 1u; }
        }
      }
      // what is in flight lands before the CTA leaves: each stage used is
      // released once more after its last MMAs, or the wait runs out
      for (int i = 0; i < STAGES; ++i) {
        if (used & (1u << s)) wait_bounded(bar(B_EMPTY + s), ph ^ 1u, nullptr, nullptr, ok ? p.wait_ns : kDrainNs);
        if (++s == STAGES) { s = 0; ph ^= 1u; }
      }
    } else if (warp == 1 && rank == 0) {
      // ================================================================ MMA issuer
      // The whole warp walks along, so that what it computes is uniform, and one
      // lane issues.  (One lane alone in the loop took 1240 cycles a block, of
      // them 430 for four MMAs and 270 for four commits; a stage's release is
      // left to the scaling warps, which see the same MMAs end.)
      int s = 0, buf = 0;
      const bool one = elect_one();
      uint32_t ph = 0, bph = 0;
      bool ok = true;
      const uint32_t tfull[2][2] = {{peer_addr(bar(B_TFULL), 0), peer_addr(bar(B_TFULL), 1)},
                                    {peer_addr(bar(B_TFULL + 1), 0), peer_addr(bar(B_TFULL + 1), 1)}};
      for (int tile = first; ok && tile < total; tile += step) {
        for (int kb = 0; kb < p.kblocks; ++kb) {
          ok = wait_bounded(bar(B_FULL + s), ph, abort_s, p.err, p.wait_ns) &&
               wait_bounded(bar(B_TEMPTY + buf), bph ^ 1u, abort_s, p.err, p.wait_ns);
          if (!(ok = __all_sync(0xffffffffu, ok ? 1 : 0) != 0)) break;
          tc_fence_after();
          const uint64_t a = smem_desc(smem_base + s * STAGE_BYTES, 16, 1024);
          const uint64_t b = a + (TILE_BYTES >> 4);  // (addresses in units of 16 bytes, below 2^18)
          if (one) {
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk) mma_pair(tmem_base + buf * 256, a + 2 * kk, b + 2 * kk, kk ? 1u : 0u);
            commit_at(tfull[buf][1]);
            commit_at(tfull[buf][0]);
          }
          __syncwarp();
          if (++s == STAGES) { s = 0; ph ^= 1u; }
          if (++buf == 2) { buf = 0; bph ^= 1u; }
        }
      }
      // all MMAs retire before TMEM is released
      if (one) commit_at(lead(B_DRAIN));
      __syncwarp();
      wait_bounded(bar(B_DRAIN), 0, nullptr, nullptr, ok ? p.wait_ns : kDrainNs);
    }
    __syncwarp();
  } else {
    // ================================================================ scaling and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int quarter = warp & 3, part = (warp - 4) >> 2, r = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    // column of chunk c (32 columns) in an accumulator
    auto col = [&](int c) { return MODE == UP_SWIGLU ? (c >> 1) * 128 + part * 64 + (c & 1) * 32 : part * 128 + c * 32; };
    int buf = 0, turn = 0, slot = 0, stage = 0;
    uint32_t bph = 0;
    bool ok = true;
    for (int tile = first; tile < total; tile += step, turn ^= 1) {
      const Tile t = decode(p, tile, num_mt);
      const int q = t.row0 + (int)rank * BM + r;
      const int nb = p.N / kBlock8;
      // the block of this thread's columns (SwiGLU: the tile's, in both matrices)
      const int blk = MODE == UP_SWIGLU ? t.n0 : t.n0 * 2 + part;
      const bool in = MODE == UP_SWIGLU || blk < nb;
      const int64_t so = ((int64_t)t.e * nb + (in ? blk : nb - 1)) * p.kblocks;
      const float* w0 = p.s0 + so;
      const float* w1 = MODE == UP_SWIGLU ? p.s1 + so : nullptr;
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
      // the weights' scales: 32 blocks' at a time, one a lane, handed round by shuffles
      float cw0 = 0.f, cw1 = 0.f, nw0, nw1 = 0.f;
      auto fetch_w = [&](int kb) {
        const int i = min(kb + lane, p.kblocks - 1);
        nw0 = w0[i];
        if (MODE == UP_SWIGLU) nw1 = w1[i];
      };
      fetch_w(0);
      for (int kb = 0; kb < p.kblocks; ++kb) {
        if ((kb & 31) == 0) {
          cw0 = nw0;
          cw1 = nw1;
          fetch_w(kb + 32);
        }
        const float m0 = __shfl_sync(0xffffffffu, cw0, kb & 31);
        const float m1 = MODE == UP_SWIGLU ? __shfl_sync(0xffffffffu, cw1, kb & 31) : m0;
        ok = __all_sync(0xffffffffu, wait_bounded(bar(B_TFULL + buf), bph, abort_s, p.err, p.wait_ns) ? 1 : 0) != 0;
        if (!ok) break;
        arrive_if(bar(B_EMPTY + stage), lane == 0 && (slot & (SCALE_WARPS - 1)) == warp - 4);
        stage = stage == STAGES - 1 ? 0 : stage + 1;
        // (landed: the MMAs waited for the stage that it came with)
        const float sr = scales[slot * BM + r];
        slot = slot == SLOTS - 1 ? 0 : slot + 1;
        tc_fence_after();
        const uint32_t tb = tmem_base + lanes + buf * 256;
        uint32_t ra[32], rb[32];
        auto add = [&](const uint32_t (&v)[32], int c) {
          const float m = sr * (c < 2 ? m0 : m1);
          const float2 mm = make_float2(m, m);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[c * 16 + i] = __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), mm, acc[c * 16 + i]);
        };
        MB_TMEM_LD32(tb + col(0), ra);
        MB_TMEM_LD32(tb + col(1), rb);
        tmem_wait_ld();
        add(ra, 0);
        add(rb, 1);
        MB_TMEM_LD32(tb + col(2), ra);
        MB_TMEM_LD32(tb + col(3), rb);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_pair(lead(B_TEMPTY + buf));
        add(ra, 2);
        add(rb, 3);
        if (++buf == 2) { buf = 0; bph ^= 1u; }
      }
      if (!ok) break;
      // (a block of the last half tile that does not exist is computed and left)
      if constexpr (MODE == DOWN) {
        if (in) {
          // fp16 at a power of two that brings the largest to 2^14 or more: a
          // rounding of 2^-11 in front of the 2^-8 of y's own, at half of fp32's
          // bytes, which the combine step reads again
          uint32_t m = 0u;
#pragma unroll
          for (int i = 0; i < 64; ++i) m = max(m, max(abs_bits(acc[i].x), abs_bits(acc[i].y)));
          const Scale8 sc = scale16(m);
          __half* dst = p.y + (int64_t)q * p.N + blk * kBlock8;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __half2 h = __floats2half2_rn(acc[8 * i + j].x * sc.inv, acc[8 * i + j].y * sc.inv);
              o[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            store_sector(dst + 16 * i, o);
          }
          p.sh[(int64_t)blk * p.rows + q] = sc.s;
        }
      } else {
        constexpr bool SW = MODE == UP_SWIGLU;
        constexpr int NH = SW ? 32 : 64;  // pairs of hidden columns of this thread
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          float2 a = acc[i];
          a.x = a.x * __fdividef(1.f, 1.f + __expf(-a.x));
          a.y = a.y * __fdividef(1.f, 1.f + __expf(-a.y));
          if constexpr (SW) a = __fmul2_rn(a, acc[32 + i]);
          acc[i] = a;
          m = max(m, max(abs_bits(a.x), abs_bits(a.y)));
        }
        if constexpr (SW) {  // the block's other 64 columns are the other part's
          uint32_t* x = xchg + turn * 2 * BM;
          x[part * BM + r] = m;
          mbar_arrive(bar(B_XCHG));
          // (an mbarrier, so that this wait is bounded too)
          if (lane == 0) ok = wait_bounded(bar(B_XCHG), (uint32_t)turn, abort_s, p.err, p.wait_ns);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          (void)mbar_try(bar(B_XCHG), (uint32_t)turn);
          m = max(x[r], x[BM + r]);
        }
        const Scale8 sc = scale8(m);
        if (in) {
          const int c0 = blk * kBlock8 + (SW ? part * 64 : 0);
          uint8_t* dst = p.h8 + (int64_t)q * p.N + c0;
#pragma unroll
          for (int i = 0; i < NH / 16; ++i) {
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2* a = &acc[16 * i + 2 * j];
              const float v[4] = {a[0].x, a[0].y, a[1].x, a[1].y};
              o[j] = e4m3x4(v, sc.inv);
            }
            store_sector(dst + 32 * i, o);
          }
          if (!SW || part == 0) p.sh[(int64_t)blk * p.rows + q] = sc.s;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing arrives at, or reads from, this CTA any more
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
}

// the row scales (blocks, rows), boxes of one block of 128 rows
bool scale_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t blocks) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {rows, blocks};
  cuuint64_t strides[1] = {rows * 4};
  cuuint32_t box[2] = {128, 1};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
moeblaze_status launch(const Params& p, int64_t bound, cudaStream_t st) {
  auto kern = fp8_gemm_kernel<MODE>;
  MB_CUDA(smem_limit(kern, SMEM));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const int64_t pairs = sm_count() / 2, g = bound < pairs ? bound : pairs;
  cfg.gridDim = dim3((unsigned)(2 * g));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MB_CUDA(cudaLaunchKernelEx(&cfg, kern, p));
  count_launch();
  return MOEBLAZE_OK;
}

}  // namespace fp8

using namespace fp8;

moeblaze_status launch_fp8_products(const moeblaze_shape& s, const moeblaze_fp8_experts& w, const Fp8Scratch& ws,
                                    cudaStream_t st) {
  const bool sw = s.act == MOEBLAZE_SWIGLU;
  Params p;
  memset(&p, 0, sizeof(p));
  p.hdr = ws.hdr;
  p.err = ws.hdr;
  p.tile_e = ws.tile_e;
  p.rows = ws.rows;
  fault_injection(&p.wait_ns, &p.withhold);
  if (p.wait_ns == 0) p.wait_ns = kTimeoutNs;
  const int64_t mt = ws.rows / 256;
  p.s0 = w.s1;
  p.s1 = w.s2;
  p.h8 = ws.h8;
  p.sh = ws.sh;
  p.N = s.h;
  p.kblocks = s.d / BK;
  p.n_tiles = sw ? s.h / 128 : (s.h + 255) / 256;
  if (!byte_map(&p.tmA, ws.x8, s.d, ws.rows, 128) || !scale_map(&p.tmS, ws.sx, ws.rows, s.d / BK) ||
      !weight_map(&p.tmB0, w.q1, s.E, s.h, s.d) ||
      (sw && !weight_map(&p.tmB1, w.q2, s.E, s.h, s.d)))
    return MOEBLAZE_ERR_CUDA;
  moeblaze_status r = sw ? launch<UP_SWIGLU>(p, mt * p.n_tiles, st) : launch<UP_SILU>(p, mt * p.n_tiles, st);
  if (r != MOEBLAZE_OK) return r;
  p.s0 = w.s3;
  p.y = ws.y;
  p.sh = ws.sy;
  p.N = s.d;
  p.kblocks = s.h / BK;
  p.n_tiles = (s.d + 255) / 256;
  if (!byte_map(&p.tmA, ws.h8, s.h, ws.rows, 128) || !scale_map(&p.tmS, ws.sh, ws.rows, s.h / BK) ||
      !weight_map(&p.tmB0, w.q3, s.E, s.d, s.h))
    return MOEBLAZE_ERR_CUDA;
  return launch<DOWN>(p, mt * p.n_tiles, st);
}

}  // namespace moeblaze
