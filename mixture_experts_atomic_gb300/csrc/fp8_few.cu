// The experts' products on 8-bit floating-point weights, for few tokens: a used
// expert's weights are read once for each 32 of its tokens, so once for most, and
// that is what the time goes to (fp8.cu: from when on not).
//
// The tensor cores take the weights as the M operand: a 128 x 128 block of them
// (or two, of W1 and W2, or of neighbouring output rows) against 16 or 32
// tokens; an expert with more has several tiles of them.  As for prompts
// (fp8_tc.cu) the sum over a block of the reduction is scaled and added to fp32
// registers: an output row a thread, its tokens side by side.  A tile's 128 hidden
// columns are one block of 8-bit rows, so that its scale is a maximum over the
// tile's threads.
//
// Work is cut into blocks of the reduction of all tiles of all used experts, in
// one row, of which every CTA takes an equal run (one token of 2 of 8 experts,
// d 4096, h 14336: 224 tiles for 152 SMs would leave half of them idle in the
// second turn).  A tile that two or more CTAs share is left in parts, and the
// CTA that comes last adds them up, in the order of the reduction whoever it is.
//
// Half an SM's shared memory and TMEM a CTA: the down projection's CTAs are
// resident beside the up projection's, and load their first weights while that
// ends.
//
// Measured, the whole call: d 4096, h 14336, 2 of 8 experts 1 token 89 us (352 MB:
// 4.0 TB/s), 16 tokens 186 to 214 us, by how many experts the draw uses (all eight:
// 1.41 GB, 6.6 TB/s); d 2048, h 1408, 6 of 64, 61 tokens 97 to 114 us.  At one token the weights stream at 7.1 TB/s from 8 us on,
// where rows, table and first loads have come; the CTAs end between 38 and 47 us,
// the down projection has its rows 8 us later, and the sum of the slots takes 5.
// Beside it: weights not packed in blocks 260 against 239 us (16 tokens); a tile's
// parts added one load after another 122 against 90 us (one token); all four steps
// in one launch with barriers over the grid 94 to 99 us (one token), 214 to 219
// (16 tokens), 96 to 99 (61 tokens).
#include "common.cuh"
#include "eight.cuh"
#include "fp8.cuh"
#include "tc_ptx.cuh"

namespace moeblaze {
namespace fp8 {

using namespace tc;

constexpr int BK = 128;
constexpr int W_BYTES = 128 * BK;           // a block of weights
constexpr int TOKENS = kFewTile;            // of a tile, at most
constexpr int X_BYTES = TOKENS * BK;
constexpr int STAGES = 3, NBUF = 4;
constexpr int STAGE_BYTES = 2 * W_BYTES + X_BYTES;
constexpr int SLOTS = STAGES + NBUF;        // of the tokens' scales: see fp8_tc.cu
constexpr int THREADS = 192, SCALE_THREADS = 128;
constexpr int TMEM_COLS = 256;              // NBUF x (32 + 32)
// Blocks of a CTA's run, at least: shorter ones end sooner, but their parts take
// longer to add up (one token, d 1024, h 4096, 1 of 16: 42, 31, 30, 31 us with 1,
// 2, 4 and 8; d 512, h 512, 2 of 8: 25, 25, 22, 29).
constexpr int kMinRun = 4;
static_assert(NBUF * 2 * TOKENS <= TMEM_COLS, "TMEM");
constexpr int RED_BYTES = 2 * 2 * 4 * TOKENS * 4;  // [turn][half][warp][token]
constexpr int SMEM = STAGES * STAGE_BYTES + SLOTS * TOKENS * 4 + RED_BYTES + 1024 + 256;
static_assert(SMEM <= (228 * 1024) / 2 - 1024, "two CTAs an SM");

enum Mode : int { UP_SWIGLU = 0, UP_SILU, DOWN };

struct FewParams {
  CUtensorMap tmX;   // tokens (rows, R) bytes, boxes of 16 rows
  CUtensorMap tmW0;  // packed weights
  CUtensorMap tmW1;  // W2 (SwiGLU)
  const int32_t* meta;   // hdr: [1] entries; entries of {expert, first row, tokens, 0}
  const int4* entries;
  int32_t* err;
  int32_t* cnt;      // parts that have come, of each tile
  float* parts;      // (CTAs, 2, 2, tokens, 128)
  const float* sx;   // tokens' scales (R/128, rows)
  const float* s0;   // weights' scales (E, N/128, R/128)
  const float* s1;
  uint8_t* h8;       // up: H8 (rows, N)
  float* sh;         // up: its scales (N/128, rows)
  float* y;          // down: (rows, N) fp32
  int64_t rows;
  int N, kblocks, tiles;  // tiles: of one expert
  int part_tokens;        // tokens of a part
  uint64_t wait_ns;
  int withhold;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void mma_f8(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

// Where a block of the whole row of work lies: tile after tile of entry after
// entry, the blocks of a tile's reduction side by side.
template <int MODE>
struct Place {
  int a, left;             // the entry, and those behind it
  int e, row0, n, chunks;  // its expert, rows and tokens; chunks of 16 tokens
  int m, kb;               // the tile, and the block of the reduction
  bool two;                // the tile's second half exists
  __device__ __forceinline__ void entry(const FewParams& p) {
    const int4 t = __ldcg(p.entries + a);
    e = t.x;
    row0 = t.y;
    n = t.z;
    chunks = (t.z + 15) >> 4;
  }
  __device__ __forceinline__ void start(const FewParams& p, int64_t b) {
    const int64_t u = b / p.kblocks;
    a = (int)(u / p.tiles);
    left = __ldcg(p.meta + 1) - 1 - a;
    m = (int)(u - (int64_t)a * p.tiles);
    kb = (int)(b - u * p.kblocks);
    two = MODE == UP_SWIGLU || m * 256 + 128 < p.N;
    if (left >= 0) entry(p);
  }
  __device__ __forceinline__ void skip(const FewParams& p, int blocks) {  // within the tile, or to the next one's start
    kb += blocks;
    if (kb < p.kblocks) return;
    kb = 0;
    if (++m == p.tiles) {
      m = 0;
      ++a;
      if (--left >= 0) entry(p);
    }
    two = MODE == UP_SWIGLU || m * 256 + 128 < p.N;
  }
};

template <int MODE>
__global__ void __launch_bounds__(THREADS, 2) fp8_few_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES);  // [slot][token]
  uint32_t* red = reinterpret_cast<uint32_t*>(scales + SLOTS * TOKENS);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(red) + RED_BYTES);
  constexpr int B_FULL = 0, B_EMPTY = STAGES, B_TFULL = 2 * STAGES, B_TEMPTY = B_TFULL + NBUF, B_DRAIN = B_TEMPTY + NBUF,
                B_SYNC = B_DRAIN + 1, B_END = B_SYNC + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_END);
  volatile int* abort_s = reinterpret_cast<volatile int*>(bars + B_END + 1);
  volatile int* last_s = reinterpret_cast<volatile int*>(bars + B_END + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem_base = smem_u32(smem);
  auto bar = [&](int i) { return smem_u32(bars + i); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 1);
    }
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(bar(B_TFULL + b), 1);
      mbar_init(bar(B_TEMPTY + b), SCALE_THREADS / 32);
    }
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_SYNC), SCALE_THREADS);
    *abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // The up projection waits for the rows and their table before it lets the
  // down projection start, so that the latter may read the table at once; it
  // waits for the hidden rows before it loads them.
  if (MODE != DOWN) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t total = (int64_t)__ldcg(p.meta + 1) * p.tiles * p.kblocks;
  const int64_t ctas = min((int64_t)gridDim.x, (total + kMinRun - 1) / kMinRun);  // those with work
  const bool idle = blockIdx.x >= ctas;
  const int64_t begin = idle ? 0 : total * blockIdx.x / ctas, end = idle ? 0 : total * (blockIdx.x + 1) / ctas;

  if (warp == 0) {
    // ================================================================ producer
    if (lane == 0) {
      uint32_t used = 0;
      bool ok = true;
      // weights of block b into its stage, and the bytes to come
      auto weights = [&](const Place<MODE>& w, int s) {
        const uint32_t full = bar(B_FULL + s), dst = smem_base + s * STAGE_BYTES;
        mbar_expect_tx(full, (w.two ? 2 : 1) * W_BYTES + w.chunks * (16 * BK + 64));
        used |= 1u << s;
        const int64_t blk = (int64_t)w.e * (p.N / 128) + w.m * (MODE == UP_SWIGLU ? 1 : 2);
        const int r = (int)((blk * p.kblocks + w.kb) * 128);
        tma_load_2d(dst, &p.tmW0, 0, r, full);
        if (w.two)
          tma_load_2d(dst + W_BYTES, MODE == UP_SWIGLU ? &p.tmW1 : &p.tmW0, 0, MODE == UP_SWIGLU ? r : r + p.kblocks * 128, full);
      };
      auto tokens = [&](const Place<MODE>& w, int s, int slot) {
        const uint32_t full = bar(B_FULL + s), dst = smem_base + s * STAGE_BYTES + 2 * W_BYTES;
        for (int c = 0; c < w.chunks; ++c) tma_load_2d(dst + c * 16 * BK, &p.tmX, w.kb * BK, w.row0 + 16 * c, full);
        bulk_load(smem_u32(scales + slot * TOKENS), p.sx + (int64_t)w.kb * p.rows + w.row0, w.chunks * 64, full);
      };
      const bool skip = MODE == DOWN && p.withhold;  // test of the failure path: the first stage is never loaded
      int64_t ahead = begin;                         // blocks whose weights are on their way before the tokens are there
      Place<MODE> w;
      w.start(p, begin);
      if (MODE == DOWN) {
        Place<MODE> first = w;
        for (int s = 0; s < STAGES && ahead < end; ++s, ++ahead) {
          if (!(skip && s == 0)) weights(first, s);
          first.skip(p, 1);
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
      }
      int s = 0, slot = 0;
      uint32_t ph = 0;
      for (int64_t b = begin; b < end; ++b) {
        if (!(ok = wait_bounded(bar(B_EMPTY + s), ph ^ 1u, abort_s, p.err, p.wait_ns))) break;
        if (!(skip && b == begin)) {
          if (b >= ahead) weights(w, s);
          tokens(w, s, slot);
        }
        w.skip(p, 1);
        slot = slot == SLOTS - 1 ? 0 : slot + 1;
        if (++s == STAGES) { s = 0; ph ^= 1u; }
      }
      // what is in flight lands before the CTA leaves: each stage used is
      // released once more by its last MMAs, or the wait runs out
      for (int i = 0; i < STAGES; ++i) {
        if (used & (1u << s)) wait_bounded(bar(B_EMPTY + s), ph ^ 1u, nullptr, nullptr, ok ? p.wait_ns : kDrainNs);
        if (++s == STAGES) { s = 0; ph ^= 1u; }
      }
    } else if (MODE == DOWN) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    if (lane == 0) {
      int s = 0, buf = 0;
      uint32_t ph = 0, bph = 0;
      bool ok = true;
      Place<MODE> w;
      w.start(p, begin);
      for (int64_t b = begin; b < end; ++b, w.skip(p, 1)) {
        if (!(ok = wait_bounded(bar(B_TEMPTY + buf), bph ^ 1u, abort_s, p.err, p.wait_ns))) break;
        if (!(ok = wait_bounded(bar(B_FULL + s), ph, abort_s, p.err, p.wait_ns))) break;
        tc_fence_after();
        const uint32_t wa = smem_base + s * STAGE_BYTES, x = wa + 2 * W_BYTES;
        // e4m3 x e4m3 -> fp32, 128 x (16 chunks), both operands K-major
        const uint32_t idesc = (1u << 4) | ((uint32_t)w.chunks * 2u << 17) | (128u >> 4 << 24);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half && !w.two) break;
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            mma_f8(tmem_base + (2 * buf + half) * TOKENS, smem_desc(wa + half * W_BYTES + kk * 32, 16, 1024),
                   smem_desc(x + kk * 32, 16, 1024), idesc, kk ? 1u : 0u);
        }
        mma_commit(bar(B_EMPTY + s));
        mma_commit(bar(B_TFULL + buf));
        if (++s == STAGES) { s = 0; ph ^= 1u; }
        if (++buf == NBUF) { buf = 0; bph ^= 1u; }
      }
      mma_commit(bar(B_DRAIN));
      wait_bounded(bar(B_DRAIN), 0, nullptr, nullptr, ok ? p.wait_ns : kDrainNs);
    }
    __syncwarp();
  } else {
    // ================================================================ scaling and epilogue
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    int buf = 0, slot = 0, turn = 0;
    uint32_t bph = 0, sph = 0;
    bool ok = true;
    // all four warps, bounded; false once the CTA gives up
    auto sync = [&]() -> bool {
      mbar_arrive(bar(B_SYNC));
      const bool got = wait_bounded(bar(B_SYNC), sph, abort_s, p.err, p.wait_ns);
      sph ^= 1u;
      return __all_sync(0xffffffffu, got ? 1 : 0) != 0;
    };
    Place<MODE> w, next;
    next.start(p, begin);
    for (int64_t b = begin; b < end;) {
      w = next;
      const int k0 = w.kb, k1 = (int)min((int64_t)p.kblocks, k0 + (end - b));
      const int nb = p.N / kBlock8;
      // the weights' scales: of both halves (or matrices), 32 blocks' at a time, one a lane
      const int64_t row = (int64_t)w.e * nb + (MODE == UP_SWIGLU ? w.m : 2 * w.m);
      const float* w0 = p.s0 + row * p.kblocks;
      const float* w1 = MODE == UP_SWIGLU ? p.s1 + row * p.kblocks : w.two ? w0 + p.kblocks : w0;
      float cw0, cw1, nw0 = w0[min(k0 + lane, p.kblocks - 1)], nw1 = w1[min(k0 + lane, p.kblocks - 1)];
      float acc[2][TOKENS];
#pragma unroll
      for (int i = 0; i < TOKENS; ++i) acc[0][i] = acc[1][i] = 0.f;
      for (int kb = k0; kb < k1; ++kb) {
        if (((kb - k0) & 31) == 0) {
          cw0 = nw0;
          cw1 = nw1;
          const int i = min(kb + 32 + lane, p.kblocks - 1);
          nw0 = w0[i];
          nw1 = w1[i];
        }
        const float m0 = __shfl_sync(0xffffffffu, cw0, (kb - k0) & 31), m1 = __shfl_sync(0xffffffffu, cw1, (kb - k0) & 31);
        ok = __all_sync(0xffffffffu, wait_bounded(bar(B_TFULL + buf), bph, abort_s, p.err, p.wait_ns) ? 1 : 0) != 0;
        if (!ok) break;
        tc_fence_after();
        const uint32_t tb = tmem_base + lanes + buf * 2 * TOKENS;
        const float4* sc = reinterpret_cast<const float4*>(scales + slot * TOKENS);
#pragma unroll
        for (int c = 0; c < TOKENS / 16; ++c) {
          if (c < w.chunks) {
            uint32_t ra[16], rb[16];
            MB_TMEM_LD16(tb + 16 * c, ra);
            MB_TMEM_LD16(tb + TOKENS + 16 * c, rb);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = sc[4 * c + i];
              const float t[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int q = 4 * i + j;
                acc[0][16 * c + q] = fmaf(__uint_as_float(ra[q]), t[j] * m0, acc[0][16 * c + q]);
                acc[1][16 * c + q] = fmaf(__uint_as_float(rb[q]), t[j] * m1, acc[1][16 * c + q]);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_TEMPTY + buf));
        slot = slot == SLOTS - 1 ? 0 : slot + 1;
        if (++buf == NBUF) { buf = 0; bph ^= 1u; }
      }
      if (!ok) break;
      b += k1 - k0;
      if (b < end) next.skip(p, k1 - k0);
      if (k0 != 0 || k1 != p.kblocks) {
        // a part: of the CTA that starts the tile in its second place
        const int64_t u = (b - 1) / p.kblocks;
        auto part = [&](int64_t cta, int second) {
          return p.parts + ((cta * 2 + second) * 2 * p.part_tokens) * 128 + r;
        };
        float* mine = part(blockIdx.x, k0 == 0 ? 1 : 0);
#pragma unroll
        for (int k = 0; k < TOKENS / 16; ++k)
          if (k < w.chunks) {
#pragma unroll
            for (int i = 16 * k; i < 16 * k + 16; ++i) {
              __stcg(mine + i * 128, acc[0][i]);
              __stcg(mine + (p.part_tokens + i) * 128, acc[1][i]);
            }
          }
        __threadfence();
        if (!(ok = sync())) break;
        // the CTAs that share the tile: block x belongs to CTA ((x + 1) ctas - 1) / total
        const int64_t c0 = ((u * p.kblocks + 1) * ctas - 1) / total;
        const int64_t c1 = ((u + 1) * p.kblocks * ctas - 1) / total;
        if (threadIdx.x == THREADS - SCALE_THREADS) *last_s = atomicAdd(p.cnt + u, 1) == (int)(c1 - c0) ? 1 : 0;
        if (!(ok = sync())) break;
        if (!*last_s) continue;
        __threadfence();
#pragma unroll
        for (int i = 0; i < TOKENS; ++i) acc[0][i] = acc[1][i] = 0.f;
        for (int64_t c = c0; c <= c1; ++c) {
          const float* q = part(c, c == c0 ? 1 : 0);
          // (32 loads in flight: one after the other they took 25 us of a token's 122)
#pragma unroll
          for (int k = 0; k < TOKENS / 16; ++k)
            if (k < w.chunks) {
              float v[2][16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                v[0][i] = __ldcg(q + (16 * k + i) * 128);
                v[1][i] = __ldcg(q + (p.part_tokens + 16 * k + i) * 128);
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                acc[0][16 * k + i] += v[0][i];
                acc[1][16 * k + i] += v[1][i];
              }
            }
        }
      }
      if constexpr (MODE == DOWN) {
        const int col = w.m * 256 + r;
#pragma unroll
        for (int i = 0; i < TOKENS; ++i) {
          if (i < w.n) {
            float* dst = p.y + (int64_t)(w.row0 + i) * p.N + col;
            dst[0] = acc[0][i];
            if (w.two) dst[128] = acc[1][i];
          }
        }
      } else {
        constexpr bool SW = MODE == UP_SWIGLU;
        constexpr int HALVES = SW ? 1 : 2;
        uint32_t* rd = red + turn * 2 * 4 * TOKENS;
        turn ^= 1;
#pragma unroll
        for (int half = 0; half < HALVES; ++half)
#pragma unroll
          for (int i = 0; i < TOKENS; ++i) {
            if (i < 16 * w.chunks) {
              float h = acc[half][i];
              h = h * __fdividef(1.f, 1.f + __expf(-h));
              if (SW) h *= acc[1][i];
              acc[half][i] = h;
              const uint32_t m = __reduce_max_sync(0xffffffffu, abs_bits(h));
              if (lane == 0) rd[(half * 4 + quarter) * TOKENS + i] = m;
            }
          }
        if (!(ok = sync())) break;
#pragma unroll
        for (int half = 0; half < HALVES; ++half) {
          if (half && !w.two) break;
          const int blk = SW ? w.m : 2 * w.m + half;
#pragma unroll
          for (int i = 0; i < TOKENS; ++i) {
            if (i < w.n) {
              const uint32_t* q = rd + half * 4 * TOKENS + i;
              const Scale8 s8 = scale8(max(max(q[0], q[TOKENS]), max(q[2 * TOKENS], q[3 * TOKENS])));
              p.h8[(int64_t)(w.row0 + i) * p.N + blk * kBlock8 + r] =
                  (uint8_t)__nv_cvt_float_to_fp8(acc[half][i] * s8.inv, __NV_SATFINITE, __NV_E4M3);
              if (r == 0) p.sh[(int64_t)blk * p.rows + w.row0 + i] = s8.s;
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
}

template <int MODE>
moeblaze_status launch_few(const FewParams& p, int ctas, cudaStream_t st) {
  auto kern = fp8_few_kernel<MODE>;
  MB_CUDA(smem_limit(kern, SMEM));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MB_CUDA(cudaLaunchKernelEx(&cfg, kern, p));
  count_launch();
  return MOEBLAZE_OK;
}

// ------------------------------------------------------------------ rows
// A CTA a token: which row each of its slots takes, and its row to those rows;
// the first CTA writes the table of the used experts besides.  Every CTA counts
// all slots for itself (there are at most 4096).  An expert's rows come in the
// order of its slots, its segment is padded to 16 rows.
constexpr int kPrepThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) few_rows_kernel(const T* __restrict__ x, const float* __restrict__ sx,
                                                                const int32_t* __restrict__ ids, int n, int d, int E, int K,
                                                                int64_t rows, int32_t* hdr, int4* entries, int32_t* cnt,
                                                                int counters, int32_t* pos, uint8_t* __restrict__ x8,
                                                                float* __restrict__ s8) {
  __shared__ int id_s[kFewSlots], hist[kMaxE], first_s[kMaxE], at_s[kMaxE], to_s[kMaxK];
  __shared__ int2 warp_s[kPrepThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5, t = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = tid; i < E; i += kPrepThreads) hist[i] = 0;
  for (int i = tid; i < n; i += kPrepThreads) id_s[i] = ids[i];
  for (int i = t * kPrepThreads + tid; i < counters; i += gridDim.x * kPrepThreads) cnt[i] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kPrepThreads)
    if ((unsigned)id_s[i] < (unsigned)E) atomicAdd(&hist[id_s[i]], 1);
  __syncthreads();
  // exclusive sums over the experts, two a thread: rows (padded), table entries
  static_assert(kMaxE <= 2 * kPrepThreads, "two experts a thread");
  const int e0 = 2 * tid;
  const int n0 = e0 < E ? hist[e0] : 0, n1 = e0 + 1 < E ? hist[e0 + 1] : 0;
  auto padded = [](int c) { return (c + 15) & ~15; };
  auto tiles = [](int c) { return (c + TOKENS - 1) / TOKENS; };
  int2 sum = make_int2(padded(n0) + padded(n1), tiles(n0) + tiles(n1));
  const int2 own = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, sum.x, o), b = __shfl_up_sync(0xffffffffu, sum.y, o);
    if (lane >= o) {
      sum.x += a;
      sum.y += b;
    }
  }
  if (lane == 31) warp_s[wp] = sum;
  __syncthreads();
  int2 base = make_int2(sum.x - own.x, sum.y - own.y);
  int all = 0;
  for (int i = 0; i < kPrepThreads / 32; ++i) {
    if (i < wp) {
      base.x += warp_s[i].x;
      base.y += warp_s[i].y;
    }
    all += warp_s[i].y;
  }
  if (e0 < E) {
    first_s[e0] = base.x;
    at_s[e0] = base.y;
  }
  if (e0 + 1 < E) {
    first_s[e0 + 1] = base.x + padded(n0);
    at_s[e0 + 1] = base.y + tiles(n0);
  }
  __syncthreads();
  if (t == 0) {
    for (int e = tid; e < E; e += kPrepThreads)
      for (int i = 0; i < tiles(hist[e]); ++i)
        entries[at_s[e] + i] = make_int4(e, first_s[e] + TOKENS * i, min(TOKENS, hist[e] - TOKENS * i), 0);
    if (tid == 0) {
      hdr[0] = 0;
      hdr[1] = all;
    }
  }
  if (wp < K) {  // a warp a slot: the slots before it on the same expert
    const int j = t * K + wp, id = id_s[j];
    int before = 0;
    for (int i = lane; i < j; i += 32) before += id_s[i] == id ? 1 : 0;
    before = __reduce_add_sync(0xffffffffu, before);
    const int row = (unsigned)id < (unsigned)E ? first_s[id] + before : -1;
    if (lane == 0) {
      to_s[wp] = row;
      pos[j] = row;
    }
  }
  __syncthreads();
  if constexpr (sizeof(T) == 1) {
    for (int c = tid; c < d / 16; c += kPrepThreads) {
      const uint4 v = reinterpret_cast<const uint4*>(x + (int64_t)t * d)[c];
      for (int k = 0; k < K; ++k)
        if (to_s[k] >= 0) reinterpret_cast<uint4*>(x8 + (int64_t)to_s[k] * d)[c] = v;
    }
    for (int b = tid; b < d / kBlock8; b += kPrepThreads) {
      const float v = sx[(int64_t)t * (d / kBlock8) + b];
      for (int k = 0; k < K; ++k)
        if (to_s[k] >= 0) s8[b * rows + to_s[k]] = v;
    }
  } else {
    for (int c0 = wp * 32; c0 < d / 8; c0 += kPrepThreads) {  // 8 columns a lane, 16 lanes a block
      const int c = c0 + lane;
      uint32_t v[4] = {0u, 0u, 0u, 0u}, m = 0u;
      float f[8];
      if (c < d / 8) {
        const uint4 u = reinterpret_cast<const uint4*>(x + (int64_t)t * d)[c];
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 q = unpack_bf16x2(v[i]);
        f[2 * i] = q.x;
        f[2 * i + 1] = q.y;
        m = max(m, max(abs_bits(q.x), abs_bits(q.y)));
      }
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
      const Scale8 sc = scale8(m);
      if (c < d / 8) {
        const uint2 o = make_uint2(e4m3x4(f, sc.inv), e4m3x4(f + 4, sc.inv));
        for (int k = 0; k < K; ++k)
          if (to_s[k] >= 0) {
            reinterpret_cast<uint2*>(x8 + (int64_t)to_s[k] * d)[c] = o;
            if ((lane & 15) == 0) s8[(int64_t)(c >> 4) * rows + to_s[k]] = sc.s;
          }
      }
    }
  }
}

}  // namespace fp8

using namespace fp8;

// rows with every used expert's segment padded to 16
int64_t few_max_rows(const moeblaze_shape& s) {
  const int64_t slots = s.L * s.K, used = s.E < slots ? s.E : slots;
  return (slots + 15 * used + 15) / 16 * 16;
}
int64_t few_max_entries(const moeblaze_shape& s) {
  const int64_t slots = s.L * s.K, used = s.E < slots ? s.E : slots;
  return used + slots / kFewTile;
}
int few_tiles_up(const moeblaze_shape& s) { return s.act == MOEBLAZE_SWIGLU ? s.h / 128 : (s.h + 255) / 256; }
int few_tiles_down(const moeblaze_shape& s) { return (s.d + 255) / 256; }
int few_part_tokens(const moeblaze_shape& s) {
  const int64_t slots = (s.L * s.K + 15) / 16 * 16;
  return (int)(slots < kFewTile ? slots : kFewTile);
}

moeblaze_status launch_fp8_few(const moeblaze_shape& s, const void* x, const float* x_scales, const int32_t* ids,
                               const moeblaze_fp8_experts& w, const Fp8FewScratch& ws, cudaStream_t st) {
  const bool sw = s.act == MOEBLAZE_SWIGLU;
  const int n = (int)(s.L * s.K), up = few_tiles_up(s), down = few_tiles_down(s);
  const int counters = (int)(few_max_entries(s) * (up + down));
  if (x_scales)
    few_rows_kernel<<<(unsigned)s.L, kPrepThreads, 0, st>>>((const uint8_t*)x, x_scales, ids, n, s.d, s.E, s.K, ws.rows,
                                                            ws.hdr, (int4*)ws.entries, ws.cnt, counters, ws.pos, ws.x8, ws.sx);
  else
    few_rows_kernel<<<(unsigned)s.L, kPrepThreads, 0, st>>>((const __nv_bfloat16*)x, x_scales, ids, n, s.d, s.E, s.K, ws.rows,
                                                            ws.hdr, (int4*)ws.entries, ws.cnt, counters, ws.pos, ws.x8, ws.sx);
  MB_CUDA(cudaGetLastError());
  count_launch();
  FewParams p;
  memset(&p, 0, sizeof(p));
  p.meta = ws.hdr;
  p.entries = (const int4*)ws.entries;
  p.err = ws.hdr;
  p.cnt = ws.cnt;
  p.parts = ws.parts;
  p.rows = ws.rows;
  p.part_tokens = few_part_tokens(s);
  fault_injection(&p.wait_ns, &p.withhold);
  if (p.wait_ns == 0) p.wait_ns = kTimeoutNs;
  p.sx = ws.sx;
  p.s0 = w.s1;
  p.s1 = w.s2;
  p.h8 = ws.h8;
  p.sh = ws.sh;
  p.N = s.h;
  p.kblocks = s.d / BK;
  p.tiles = up;
  if (!byte_map(&p.tmX, ws.x8, s.d, ws.rows, 16) || !weight_map(&p.tmW0, w.q1, s.E, s.h, s.d) ||
      (sw && !weight_map(&p.tmW1, w.q2, s.E, s.h, s.d)))
    return MOEBLAZE_ERR_CUDA;
  const int ctas = sm_count();
  moeblaze_status r = sw ? launch_few<UP_SWIGLU>(p, ctas, st) : launch_few<UP_SILU>(p, ctas, st);
  if (r != MOEBLAZE_OK) return r;
  p.cnt = ws.cnt + few_max_entries(s) * up;
  p.sx = ws.sh;
  p.s0 = w.s3;
  p.y = ws.y;
  p.N = s.d;
  p.kblocks = s.h / BK;
  p.tiles = down;
  if (!byte_map(&p.tmX, ws.h8, s.h, ws.rows, 16) || !weight_map(&p.tmW0, w.q3, s.E, s.d, s.h))
    return MOEBLAZE_ERR_CUDA;
  return launch_few<DOWN>(p, ctas, st);
}

}  // namespace moeblaze
