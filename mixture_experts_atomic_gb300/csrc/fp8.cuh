// What the 8-bit experts' steps share: the scratch of one call.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace moeblaze {

// Prompts.  Row space: expert e owns a multiple of 256 rows (a pair of CTAs' row
// tiles); its routed rows come first.
struct Fp8Scratch {
  int32_t* hdr;      // [0] error word, [1] row tiles of 256
  int32_t* cnt;      // (chunks, E): slots of each expert in each chunk of them
  int32_t* tile_e;   // expert of each row tile
  int32_t* pos;      // (L, K): a slot's row, -1 for an empty slot
  uint8_t* x8;       // (rows, d)
  float* sx;         // (d/128, rows)
  uint8_t* h8;       // (rows, h)
  float* sh;         // (h/128, rows)
  __half* y;         // (rows, d), with a scale for each 128 columns
  float* sy;         // (d/128, rows)
  int64_t rows;
};

// fp8_tc.cu: both products over the rows of ws, into ws.y
moeblaze_status launch_fp8_products(const moeblaze_shape& s, const moeblaze_fp8_experts& w, const Fp8Scratch& ws,
                                    cudaStream_t st);

// Few tokens.  Segments padded to 16 rows; an entry of the table is at most
// kFewTile tokens of one expert.
constexpr int kFewTile = 32;
constexpr int kFewSlots = 4096;  // L K at most
struct Fp8FewScratch {
  int32_t* hdr;      // [0] error word, [1] entries
  int32_t* entries;  // {expert, first row, tokens, 0}
  int32_t* cnt;      // parts that have come, of each tile of both products
  int32_t* pos;      // (L, K): a slot's row, -1 for an empty slot
  uint8_t* x8;       // (rows, d)
  float* sx;         // (d/128, rows)
  uint8_t* h8;       // (rows, h)
  float* sh;         // (h/128, rows)
  float* y;          // (rows, d)
  float* parts;      // (CTAs, 2, 2, few_part_tokens, 128)
  int64_t rows;
};
int64_t few_max_rows(const moeblaze_shape& s);
int64_t few_max_entries(const moeblaze_shape& s);
int few_tiles_up(const moeblaze_shape& s);
int few_tiles_down(const moeblaze_shape& s);
int few_part_tokens(const moeblaze_shape& s);

// fp8_few.cu: rows and both products, into ws.y
moeblaze_status launch_fp8_few(const moeblaze_shape& s, const void* x, const float* x_scales, const int32_t* ids,
                               const moeblaze_fp8_experts& w, const Fp8FewScratch& ws, cudaStream_t st);

// 2-D map of a row-major (rows x cols) byte matrix, boxes of 128 columns, 128-byte swizzle
inline bool byte_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// packed weights: a block of 128 x 128 is 128 rows of 128 bytes, row
// ((e N/128 + n/128) R/128 + r/128) 128 + n % 128
inline bool weight_map(CUtensorMap* m, const void* base, int E, int N, int R) {
  return byte_map(m, base, 128, (uint64_t)E * N * (R / 128), 128);
}

}  // namespace moeblaze
