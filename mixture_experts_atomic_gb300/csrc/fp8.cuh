// What the 8-bit experts' steps share: the scratch of one call.
#pragma once

#include "common.cuh"

namespace moeblaze {

// Row space: expert e owns rows [off[e], off[e+1]), a multiple of 256 of them
// (a pair of CTAs' row tiles); its routed rows come first.
struct Fp8Scratch {
  int32_t* hdr;      // [0] error word, [1] row tiles of 256
  int32_t* cnt;      // (chunks, E): slots of each expert in each chunk of them
  int32_t* tile_e;   // expert of each row tile
  int32_t* pos;      // (L, K): a slot's row, -1 for an empty slot
  uint8_t* x8;       // (rows, d)
  float* sx;         // (d/128, rows)
  uint8_t* h8;       // (rows, h)
  float* sh;         // (h/128, rows)
  float* y;          // (rows, d)
  int64_t rows;
};

// fp8_tc.cu: both products over the rows of ws, into ws.y
moeblaze_status launch_fp8_products(const moeblaze_shape& s, const moeblaze_fp8_experts& w, const Fp8Scratch& ws,
                                    cudaStream_t st);

}  // namespace moeblaze
