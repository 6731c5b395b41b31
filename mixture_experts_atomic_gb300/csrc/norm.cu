// Layer norm with the residual sum fused, and its backward (see norm_impl.cuh).
#include "norm_impl.cuh"

namespace moeblaze {

size_t norm_ws_bytes(const moeblaze_shape& s) { return norm_scratch<false>(s); }

moeblaze_status launch_layernorm_forward(const moeblaze_shape& s, const void* x, const void* res, const float* w,
                                         const float* b, float eps, void* sum, void* y, float* mean, float* rstd,
                                         cudaStream_t st) {
  return norm_forward<false>(s, FwdArgs{x, res, w, b, eps, sum, y, mean, rstd, Rows8{nullptr, nullptr}}, st);
}

moeblaze_status launch_layernorm_backward(const moeblaze_shape& s, const void* dy, const void* sum, const float* mean,
                                          const float* rstd, const float* w, const void* dsum, void* dx, float* dw,
                                          float* db, void* ws, cudaStream_t st) {
  return norm_backward<false>(s, BwdArgs{dy, sum, mean, rstd, w, dsum, dx, dw, db, (float*)ws}, st);
}

}  // namespace moeblaze
