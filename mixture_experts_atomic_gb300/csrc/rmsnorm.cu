// Root-mean-square norm with the residual sum fused, with its rows in 8 bits
// where asked for, and its backward (see norm_impl.cuh).
#include "norm_impl.cuh"

namespace moeblaze {

size_t rmsnorm_ws_bytes(const moeblaze_shape& s) { return norm_scratch<true>(s); }

moeblaze_status launch_rmsnorm_forward(const moeblaze_shape& s, const void* x, const void* res, const float* w,
                                       float eps, void* sum, void* y, float* rstd, void* q, float* q_scales,
                                       cudaStream_t st) {
  return norm_forward<true>(
      s, FwdArgs{x, res, w, nullptr, eps, sum, y, nullptr, rstd, Rows8{(uint8_t*)q, q_scales}}, st);
}

moeblaze_status launch_rmsnorm_backward(const moeblaze_shape& s, const void* dy, const void* sum, const float* rstd,
                                        const float* w, const void* dsum, void* dx, float* dw, void* ws,
                                        cudaStream_t st) {
  return norm_backward<true>(s, BwdArgs{dy, sum, nullptr, rstd, w, dsum, dx, dw, nullptr, (float*)ws}, st);
}

}  // namespace moeblaze
