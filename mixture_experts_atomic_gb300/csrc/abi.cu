// extern "C" entry points of the moeblaze library (declared in
// include/moeblaze.h): argument validation, scratch carving and the order of
// the stages; every stage runs in the kernels of dispatch.cu, identity.cu,
// simt.cu, gemm_tc.cu, router.cu, router_tc.cu, norm.cu, balance.cu and int4.cu.
#include <atomic>
#include <cstring>

#include "common.cuh"

namespace moeblaze {

int sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cached[dev] = n;
  }
  return cached[dev];
}

namespace {
std::atomic<int64_t> g_launches{0};
thread_local void** g_events = nullptr;
thread_local int32_t g_nevents = 0;
thread_local uint64_t g_wait_ns = 0;
thread_local int g_withhold = 0;
}  // namespace

void fault_injection(uint64_t* wait_ns, int* withhold) {
  *wait_ns = g_wait_ns;
  *withhold = g_withhold;
}

void count_launch(int n) { g_launches.fetch_add(n, std::memory_order_relaxed); }

void stage_event(int i, cudaStream_t st) {
  if (g_events && i < g_nevents && g_events[i]) cudaEventRecord(reinterpret_cast<cudaEvent_t>(g_events[i]), st);
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// shape checks shared by every entry point
moeblaze_status check_shape(const moeblaze_shape* s) {
  if (!s) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L < 0 || s->E < 1 || s->K < 1 || s->d < 1) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->K > s->E) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->dtype != MOEBLAZE_F32 && s->dtype != MOEBLAZE_BF16) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->act != MOEBLAZE_SWIGLU && s->act != MOEBLAZE_SILU && s->act != MOEBLAZE_IDENTITY)
    return MOEBLAZE_ERR_INVALID_ARG;
  if (s->act != MOEBLAZE_IDENTITY && s->h < 1) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->flags & ~MOEBLAZE_RECOMPUTE_H) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->E > kMaxE || s->K > kMaxK) return MOEBLAZE_ERR_UNSUPPORTED;
  if (s->L * (int64_t)s->K + (int64_t)s->E * kRowPad >= (int64_t(1) << 31)) return MOEBLAZE_ERR_UNSUPPORTED;
  if (s->act == MOEBLAZE_IDENTITY) {
    if (s->d % (s->dtype == MOEBLAZE_BF16 ? 8 : 4) != 0) return MOEBLAZE_ERR_UNSUPPORTED;
  } else if (s->dtype == MOEBLAZE_BF16) {
    if (s->d % 128 != 0 || s->h % 128 != 0) return MOEBLAZE_ERR_UNSUPPORTED;
  } else {
    if (s->d % 4 != 0 || s->h % 4 != 0) return MOEBLAZE_ERR_UNSUPPORTED;
  }
  return MOEBLAZE_OK;
}

moeblaze_status check_dispatch(const moeblaze_dispatch* d) {
  if (!d) return MOEBLAZE_ERR_INVALID_ARG;
  const void* ps[5] = {d->expert_token_indices, d->expert_token_offsets, d->token_expert_indices, d->token_index_map,
                       d->meta};
  for (const void* p : ps)
    if (!p || !aligned16(p)) return MOEBLAZE_ERR_INVALID_ARG;
  return MOEBLAZE_OK;
}

bool ok_ptr(const void* p) { return p && aligned16(p); }
bool ok_ptr4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// shape checks of the router entry points (h and act are not used)
moeblaze_status check_router_shape(const moeblaze_shape* s) {
  if (!s) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L < 0 || s->E < 1 || s->K < 1 || s->d < 1 || s->K > s->E) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->dtype != MOEBLAZE_F32 && s->dtype != MOEBLAZE_BF16) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->E > kMaxRouterE || s->K > kMaxK || s->d % 64 != 0) return MOEBLAZE_ERR_UNSUPPORTED;
  if (s->L * (int64_t)s->K >= (int64_t(1) << 31)) return MOEBLAZE_ERR_UNSUPPORTED;
  return MOEBLAZE_OK;
}

// shape checks of the layer norm (fields L, d, dtype)
moeblaze_status check_norm_shape(const moeblaze_shape* s) {
  if (!s || s->L < 0 || s->d < 1) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->dtype != MOEBLAZE_F32 && s->dtype != MOEBLAZE_BF16) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L >= (int64_t(1) << 31) || s->d > (1 << 24)) return MOEBLAZE_ERR_UNSUPPORTED;
  return MOEBLAZE_OK;
}

// shape checks of the router losses (fields L, E, K)
moeblaze_status check_balance_shape(const moeblaze_shape* s) {
  if (!s || s->L < 0 || s->E < 1 || s->K < 1 || s->K > s->E) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->E > kMaxE || s->K > kMaxK || s->L * (int64_t)s->K >= (int64_t(1) << 31)) return MOEBLAZE_ERR_UNSUPPORTED;
  return MOEBLAZE_OK;
}

// checks of one 4-bit matrix (E,R,N) and of the layer on such matrices
moeblaze_status check_int4_matrix(int E, int R, int N, int group) {
  if (E < 1 || R < 1 || N < 1) return MOEBLAZE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MOEBLAZE_ERR_INVALID_ARG;
  if (E > kMaxE || R % 128 != 0 || N % 128 != 0) return MOEBLAZE_ERR_UNSUPPORTED;
  return MOEBLAZE_OK;
}
moeblaze_status check_int4_shape(const moeblaze_shape* s, int group) {
  const moeblaze_status r = check_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if (group != 32 && group != 64 && group != 128) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->act == MOEBLAZE_IDENTITY || s->dtype != MOEBLAZE_BF16 || s->h > (1 << 22) || !int4_shape_ok(*s, group))
    return MOEBLAZE_ERR_UNSUPPORTED;
  return MOEBLAZE_OK;
}

size_t elem(const moeblaze_shape* s) { return s->dtype == MOEBLAZE_BF16 ? 2 : 4; }
int nbranch(const moeblaze_shape* s) { return s->act == MOEBLAZE_SWIGLU ? 2 : 1; }

// MOEBLAZE_RECOMPUTE_H applies to the bf16 expert layers: H and Hg are then
// recomputed from the saved A, B inside the down-projection and dW3 GEMMs
// and never stored.
bool recompute_h(const moeblaze_shape* s) {
  return s->dtype == MOEBLAZE_BF16 && s->act != MOEBLAZE_IDENTITY && (s->flags & MOEBLAZE_RECOMPUTE_H);
}

// saved:            A | B (SwiGLU) (rows x h each); bf16 with recompute: | one fp32 gate per row
// forward scratch:  H (rows x h; not when recomputed) | y32 (L x d fp32) + tile counters (bf16 only)
// backward scratch: bf16: Hg (rows x h; not when recomputed) | dX32 (L x d fp32) + tile counters
//                   (dA, dB overwrite the saved A, B);  fp32: dAB (rows x nb*h) | Hg (rows x h)
size_t fwd_ws(const moeblaze_shape* s) {
  if (s->act == MOEBLAZE_IDENTITY) return 0;
  const int64_t rows = max_padded_rows(s->L * s->K, s->E);
  size_t b = recompute_h(s) ? 0 : align_up((size_t)rows * s->h * elem(s), 256);
  if (s->dtype == MOEBLAZE_BF16) b += align_up((size_t)s->L * s->d * 4, 256) + kSchedBytes;
  return b;
}
size_t hg_bytes(const moeblaze_shape* s) {
  const int64_t rows = max_padded_rows(s->L * s->K, s->E);
  return recompute_h(s) ? 0 : align_up((size_t)rows * s->h * elem(s), 256);
}
size_t bwd_ws(const moeblaze_shape* s) {
  if (s->act == MOEBLAZE_IDENTITY) return 0;
  const int64_t rows = max_padded_rows(s->L * s->K, s->E);
  if (s->dtype == MOEBLAZE_BF16) return hg_bytes(s) + align_up((size_t)s->L * s->d * 4, 256) + kSchedBytes;
  return align_up((size_t)rows * nbranch(s) * s->h * elem(s), 256) + hg_bytes(s);
}

moeblaze_status zero_weight_grads(const moeblaze_shape* s, void* dW1, void* dW2, void* dW3, cudaStream_t st) {
  const size_t n = (size_t)s->E * s->d * s->h * elem(s);
  MB_CUDA(cudaMemsetAsync(dW1, 0, n, st));
  if (dW2) MB_CUDA(cudaMemsetAsync(dW2, 0, n, st));
  MB_CUDA(cudaMemsetAsync(dW3, 0, n, st));
  return MOEBLAZE_OK;
}

}  // namespace
}  // namespace moeblaze

using namespace moeblaze;

extern "C" {

int32_t moeblaze_version(void) { return 10000; }

void moeblaze_set_stage_events(void** events, int32_t n) {
  g_events = events;
  g_nevents = events ? n : 0;
}

int64_t moeblaze_kernel_launches(void) { return g_launches.load(std::memory_order_relaxed); }

void moeblaze_set_fault_injection(int64_t wait_limit_ns, int32_t withhold) {
  g_wait_ns = wait_limit_ns > 0 ? (uint64_t)wait_limit_ns : 0;
  g_withhold = withhold ? 1 : 0;
}

const char* moeblaze_status_string(moeblaze_status st) {
  switch (st) {
    case MOEBLAZE_OK: return "ok";
    case MOEBLAZE_ERR_INVALID_ARG: return "invalid argument";
    case MOEBLAZE_ERR_UNSUPPORTED: return "unsupported shape or type";
    case MOEBLAZE_ERR_BAD_ROUTING: return "bad routing: expert id out of range or repeated within a token";
    case MOEBLAZE_ERR_WORKSPACE: return "workspace too small";
    case MOEBLAZE_ERR_TIMEOUT: return "a device-side wait timed out";
    case MOEBLAZE_ERR_CUDA: return "CUDA error";
  }
  return "unknown status";
}

size_t moeblaze_dispatch_meta_bytes(const moeblaze_shape* s) {
  if (check_shape(s) != MOEBLAZE_OK) return 0;
  return meta_bytes(s->L * s->K, s->E);
}

size_t moeblaze_dispatch_workspace_bytes(const moeblaze_shape* s) {
  if (check_shape(s) != MOEBLAZE_OK) return 0;
  return dispatch_ws_bytes(*s);
}

size_t moeblaze_saved_bytes(const moeblaze_shape* s) {
  if (check_shape(s) != MOEBLAZE_OK || s->act == MOEBLAZE_IDENTITY) return 0;
  const int64_t rows = max_padded_rows(s->L * s->K, s->E);
  return (size_t)rows * nbranch(s) * s->h * elem(s) + (recompute_h(s) ? (size_t)rows * 4 : 0);
}

size_t moeblaze_forward_workspace_bytes(const moeblaze_shape* s) {
  if (check_shape(s) != MOEBLAZE_OK) return 0;
  return fwd_ws(s);
}

size_t moeblaze_backward_workspace_bytes(const moeblaze_shape* s) {
  if (check_shape(s) != MOEBLAZE_OK) return 0;
  return bwd_ws(s);
}

moeblaze_status moeblaze_dispatch_build(const moeblaze_shape* s, const int32_t* topk_ids,
                                        const moeblaze_dispatch* out, void* ws, size_t ws_bytes, int validate,
                                        moeblaze_stream stream) {
  moeblaze_status r = check_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if ((r = check_dispatch(out)) != MOEBLAZE_OK) return r;
  if (s->L > 0 && !ok_ptr(topk_ids)) return MOEBLAZE_ERR_INVALID_ARG;
  if (ws_bytes < dispatch_ws_bytes(*s)) return MOEBLAZE_ERR_WORKSPACE;
  if (!ok_ptr(ws)) return MOEBLAZE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  r = launch_dispatch(*s, topk_ids, *out, ws, st);
  if (r != MOEBLAZE_OK || !validate) return r;
  int32_t code = 0;
  MB_CUDA(cudaMemcpyAsync(&code, out->meta, sizeof(int32_t), cudaMemcpyDeviceToHost, st));
  MB_CUDA(cudaStreamSynchronize(st));
  return (code & kErrBadRouting) ? MOEBLAZE_ERR_BAD_ROUTING : MOEBLAZE_OK;
}

moeblaze_status moeblaze_dispatch_build_static(const moeblaze_shape* s, const int32_t* topk_ids,
                                               const moeblaze_dispatch* out, int validate, moeblaze_stream stream) {
  moeblaze_status r = check_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if ((r = check_dispatch(out)) != MOEBLAZE_OK) return r;
  if (s->L > 0 && !ok_ptr(topk_ids)) return MOEBLAZE_ERR_INVALID_ARG;
  if (dispatch_ws_bytes(*s) > MOEBLAZE_STATIC_SCRATCH_BYTES) return MOEBLAZE_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  r = launch_dispatch_static(*s, topk_ids, *out, st);
  if (r != MOEBLAZE_OK || !validate) return r;
  int32_t code = 0;
  MB_CUDA(cudaMemcpyAsync(&code, out->meta, sizeof(int32_t), cudaMemcpyDeviceToHost, st));
  MB_CUDA(cudaStreamSynchronize(st));
  return (code & kErrBadRouting) ? MOEBLAZE_ERR_BAD_ROUTING : MOEBLAZE_OK;
}

moeblaze_status moeblaze_forward(const moeblaze_shape* s, const void* x, const float* gates,
                                 const moeblaze_dispatch* disp, const void* W1, const void* W2, const void* W3,
                                 void* y, void* saved, void* ws, size_t ws_bytes, moeblaze_stream stream) {
  moeblaze_status r = check_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if ((r = check_dispatch(disp)) != MOEBLAZE_OK) return r;
  // token-sized buffers may be empty (NULL) when L == 0
  const bool tok_ok = s->L == 0 || (ok_ptr(x) && ok_ptr(gates) && ok_ptr(y));
  if (!tok_ok) return MOEBLAZE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (s->act == MOEBLAZE_IDENTITY) return launch_identity_combine(*s, x, *disp, gates, y, st);
  const bool sw = s->act == MOEBLAZE_SWIGLU;
  if (!ok_ptr(W1) || !ok_ptr(W3) || (sw && !ok_ptr(W2)) || !ok_ptr(saved)) return MOEBLAZE_ERR_INVALID_ARG;
  if (ws_bytes < fwd_ws(s)) return MOEBLAZE_ERR_WORKSPACE;
  if (!ok_ptr(ws)) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L == 0) return MOEBLAZE_OK;
  const int64_t rows = max_padded_rows(s->L * s->K, s->E);
  char* w = reinterpret_cast<char*>(ws);
  if (s->dtype == MOEBLAZE_F32) {
    return simt_forward(*s, (const float*)x, gates, *disp, (const float*)W1, sw ? (const float*)W2 : nullptr,
                        (const float*)W3, (float*)y, (float*)saved, (float*)w, st);
  }
  const size_t hb = recompute_h(s) ? 0 : align_up((size_t)rows * s->h * 2, 256);
  __nv_bfloat16* H = hb ? reinterpret_cast<__nv_bfloat16*>(w) : nullptr;
  return tc_forward(*s, (const __nv_bfloat16*)x, gates, *disp, (const __nv_bfloat16*)W1,
                    sw ? (const __nv_bfloat16*)W2 : nullptr, (const __nv_bfloat16*)W3, (__nv_bfloat16*)y,
                    (__nv_bfloat16*)saved, H, reinterpret_cast<float*>(w + hb), st);
}

moeblaze_status moeblaze_backward(const moeblaze_shape* s, const void* dY, const void* x, const float* gates,
                                  const moeblaze_dispatch* disp, const void* W1, const void* W2, const void* W3,
                                  void* saved, void* dX, void* dW1, void* dW2, void* dW3, float* dgates,
                                  void* ws, size_t ws_bytes, moeblaze_stream stream) {
  moeblaze_status r = check_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if ((r = check_dispatch(disp)) != MOEBLAZE_OK) return r;
  const bool tok_ok = s->L == 0 || (ok_ptr(dY) && ok_ptr(gates) && ok_ptr(dX) && ok_ptr(x));
  if (!tok_ok) return MOEBLAZE_ERR_INVALID_ARG;
  if (dgates && !aligned16(dgates)) return MOEBLAZE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (s->act == MOEBLAZE_IDENTITY) {
    r = launch_identity_combine(*s, dY, *disp, gates, dX, st);
    if (r != MOEBLAZE_OK || !dgates) return r;
    return launch_identity_dgates(*s, x, dY, dgates, st);
  }
  const bool sw = s->act == MOEBLAZE_SWIGLU;
  if (!ok_ptr(W1) || !ok_ptr(W3) || (sw && !ok_ptr(W2)) || !ok_ptr(saved)) return MOEBLAZE_ERR_INVALID_ARG;
  if (!ok_ptr(dW1) || !ok_ptr(dW3) || (sw && !ok_ptr(dW2))) return MOEBLAZE_ERR_INVALID_ARG;
  if (ws_bytes < bwd_ws(s)) return MOEBLAZE_ERR_WORKSPACE;
  if (!ok_ptr(ws)) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L == 0) return zero_weight_grads(s, dW1, sw ? dW2 : nullptr, dW3, st);
  if (dgates) MB_CUDA(cudaMemsetAsync(dgates, 0, sizeof(float) * s->L * s->K, st));
  const int64_t rows = max_padded_rows(s->L * s->K, s->E);
  char* w = reinterpret_cast<char*>(ws);
  const size_t es = elem(s);
  if (s->dtype == MOEBLAZE_F32) {
    char* dAB = w;
    char* Hg = w + align_up((size_t)rows * nbranch(s) * s->h * es, 256);
    return simt_backward(*s, (const float*)dY, (const float*)x, gates, *disp, (const float*)W1,
                         sw ? (const float*)W2 : nullptr, (const float*)W3, (const float*)saved, (float*)dX,
                         (float*)dW1, sw ? (float*)dW2 : nullptr, (float*)dW3, dgates, (float*)dAB, (float*)Hg, st);
  }
  // bf16: Hg (not when recomputed) | dX32; dA, dB go over the saved A, B
  char* dX32 = w + hg_bytes(s);
  return tc_backward(*s, (const __nv_bfloat16*)dY, (const __nv_bfloat16*)x, gates, *disp, (const __nv_bfloat16*)W1,
                     sw ? (const __nv_bfloat16*)W2 : nullptr, (const __nv_bfloat16*)W3, (__nv_bfloat16*)saved,
                     (__nv_bfloat16*)dX, (__nv_bfloat16*)dW1, sw ? (__nv_bfloat16*)dW2 : nullptr, (__nv_bfloat16*)dW3,
                     dgates, recompute_h(s) ? nullptr : (__nv_bfloat16*)w, (float*)dX32, st);
}

moeblaze_status moeblaze_device_error(const moeblaze_shape* s, const moeblaze_dispatch* disp, int32_t* code,
                                      moeblaze_stream stream) {
  moeblaze_status r = check_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if (!disp || !ok_ptr(disp->meta) || !code) return MOEBLAZE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int32_t c = 0;
  MB_CUDA(cudaMemcpyAsync(&c, disp->meta, sizeof(int32_t), cudaMemcpyDeviceToHost, st));
  MB_CUDA(cudaStreamSynchronize(st));
  *code = c;
  if (c & kErrBadRouting) return MOEBLAZE_ERR_BAD_ROUTING;
  if (c & kErrTimeout) return MOEBLAZE_ERR_TIMEOUT;
  if (c & kErrShapeMismatch) return MOEBLAZE_ERR_INVALID_ARG;
  return MOEBLAZE_OK;
}

moeblaze_status moeblaze_dispatch_meta_check(const moeblaze_shape* s, const void* meta_header) {
  moeblaze_status r = check_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if (!meta_header) return MOEBLAZE_ERR_INVALID_ARG;
  return meta_matches(reinterpret_cast<const int32_t*>(meta_header), s->L, s->E, s->K) ? MOEBLAZE_OK
                                                                                     : MOEBLAZE_ERR_INVALID_ARG;
}

size_t moeblaze_router_backward_workspace_bytes(const moeblaze_shape* s) {
  if (check_router_shape(s) != MOEBLAZE_OK) return 0;
  return router_ws_bytes(*s);
}

moeblaze_status moeblaze_router_forward(const moeblaze_shape* s, const void* x, const float* Wr, const float* bias,
                                        int32_t* topk_ids, float* gates, moeblaze_stream stream) {
  moeblaze_status r = check_router_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if (!ok_ptr4(Wr) || (bias && !ok_ptr4(bias))) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L > 0 && (!ok_ptr(x) || !ok_ptr4(topk_ids) || !ok_ptr4(gates))) return MOEBLAZE_ERR_INVALID_ARG;
  return launch_router_forward(*s, x, Wr, bias, topk_ids, gates, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

size_t moeblaze_router_dispatch_workspace_bytes(const moeblaze_shape* s) {
  if (check_shape(s) != MOEBLAZE_OK || check_router_shape(s) != MOEBLAZE_OK) return 0;
  return router_dispatch_fused(*s) ? router_dispatch_ws_bytes(*s) : dispatch_ws_bytes(*s);
}

static moeblaze_status router_dispatch(const moeblaze_shape* s, const void* x, const float* Wr, const float* bias,
                                       int32_t* topk_ids, float* gates, float* logits, const moeblaze_dispatch* out,
                                       void* ws, size_t ws_bytes, moeblaze_stream stream) {
  moeblaze_status r = check_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if ((r = check_router_shape(s)) != MOEBLAZE_OK) return r;
  if ((r = check_dispatch(out)) != MOEBLAZE_OK) return r;
  if (!ok_ptr4(Wr) || (bias && !ok_ptr4(bias))) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L > 0 && (!ok_ptr(x) || !ok_ptr4(topk_ids) || !ok_ptr4(gates))) return MOEBLAZE_ERR_INVALID_ARG;
  if (ws_bytes < moeblaze_router_dispatch_workspace_bytes(s)) return MOEBLAZE_ERR_WORKSPACE;
  if (!ok_ptr(ws)) return MOEBLAZE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (router_dispatch_fused(*s)) return launch_router_dispatch(*s, x, Wr, bias, topk_ids, gates, logits, *out, ws, st);
  // shapes the fused kernel does not take (fp32 x, more than 64 experts, no
  // tokens): the router, then the dispatch build on its ids
  if (s->L > 0 && (r = launch_router_forward(*s, x, Wr, bias, topk_ids, gates, logits, st)) != MOEBLAZE_OK) return r;
  return launch_dispatch(*s, topk_ids, *out, ws, st);
}

moeblaze_status moeblaze_router_dispatch_build(const moeblaze_shape* s, const void* x, const float* Wr,
                                               const float* bias, int32_t* topk_ids, float* gates,
                                               const moeblaze_dispatch* out, void* ws, size_t ws_bytes,
                                               moeblaze_stream stream) {
  return router_dispatch(s, x, Wr, bias, topk_ids, gates, nullptr, out, ws, ws_bytes, stream);
}

moeblaze_status moeblaze_router_dispatch_build_logits(const moeblaze_shape* s, const void* x, const float* Wr,
                                                      const float* bias, int32_t* topk_ids, float* gates,
                                                      float* logits, const moeblaze_dispatch* out, void* ws,
                                                      size_t ws_bytes, moeblaze_stream stream) {
  if (s && s->L > 0 && !ok_ptr(logits)) return MOEBLAZE_ERR_INVALID_ARG;
  return router_dispatch(s, x, Wr, bias, topk_ids, gates, logits, out, ws, ws_bytes, stream);
}

moeblaze_status moeblaze_router_forward_logits(const moeblaze_shape* s, const void* x, const float* Wr,
                                               const float* bias, int32_t* topk_ids, float* gates, float* logits,
                                               moeblaze_stream stream) {
  moeblaze_status r = check_router_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if (!ok_ptr4(Wr) || (bias && !ok_ptr4(bias))) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L > 0 && (!ok_ptr(x) || !ok_ptr4(topk_ids) || !ok_ptr4(gates) || !ok_ptr(logits)))
    return MOEBLAZE_ERR_INVALID_ARG;
  return launch_router_forward(*s, x, Wr, bias, topk_ids, gates, logits, reinterpret_cast<cudaStream_t>(stream));
}

moeblaze_status moeblaze_router_backward(const moeblaze_shape* s, const void* x, const float* Wr,
                                         const int32_t* topk_ids, const float* gates, const float* dgates,
                                         float* dWr, float* dbias, void* dx, void* ws, size_t ws_bytes,
                                         moeblaze_stream stream) {
  moeblaze_status r = check_router_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if (!ok_ptr4(Wr) || !ok_ptr4(dWr) || (dbias && !ok_ptr4(dbias))) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L > 0 && (!ok_ptr(x) || !ok_ptr4(topk_ids) || !ok_ptr4(gates) || !ok_ptr4(dgates) || (dx && !ok_ptr(dx))))
    return MOEBLAZE_ERR_INVALID_ARG;
  if (ws_bytes < router_ws_bytes(*s)) return MOEBLAZE_ERR_WORKSPACE;
  if (s->L > 0 && !ok_ptr(ws)) return MOEBLAZE_ERR_INVALID_ARG;
  return launch_router_backward(*s, x, Wr, topk_ids, gates, dgates, dWr, dbias, dx, ws,
                                reinterpret_cast<cudaStream_t>(stream));
}

size_t moeblaze_router_backward_logits_workspace_bytes(const moeblaze_shape* s) {
  if (check_router_shape(s) != MOEBLAZE_OK) return 0;
  return router_dense_ws_bytes(*s);
}

moeblaze_status moeblaze_router_backward_logits(const moeblaze_shape* s, const void* x, const float* Wr,
                                                const float* dlogits, float* dWr, float* dbias, void* dx,
                                                int32_t accumulate, void* ws, size_t ws_bytes,
                                                moeblaze_stream stream) {
  moeblaze_status r = check_router_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if (!ok_ptr4(Wr) || !ok_ptr4(dWr) || (dbias && !ok_ptr4(dbias))) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L > 0 && (!ok_ptr(x) || !ok_ptr(dlogits) || (dx && !ok_ptr(dx)))) return MOEBLAZE_ERR_INVALID_ARG;
  if (ws_bytes < router_dense_ws_bytes(*s)) return MOEBLAZE_ERR_WORKSPACE;
  if (s->L > 0 && !ok_ptr(ws)) return MOEBLAZE_ERR_INVALID_ARG;
  return launch_router_dense(*s, x, Wr, dlogits, dWr, dbias, dx, accumulate != 0, ws,
                             reinterpret_cast<cudaStream_t>(stream));
}

moeblaze_status moeblaze_layernorm_forward(const moeblaze_shape* s, const void* x, const void* residual,
                                           const float* weight, const float* bias, float eps, void* sum, void* y,
                                           float* mean, float* rstd, moeblaze_stream stream) {
  moeblaze_status r = check_norm_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if (!(eps >= 0.f) || !ok_ptr(weight) || (bias && !ok_ptr(bias))) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L > 0 && (!ok_ptr(x) || !ok_ptr(y) || !ok_ptr4(mean) || !ok_ptr4(rstd) || (residual && !ok_ptr(residual)) ||
                   (sum && !ok_ptr(sum))))
    return MOEBLAZE_ERR_INVALID_ARG;
  return launch_layernorm_forward(*s, x, residual, weight, bias, eps, sum, y, mean, rstd,
                                  reinterpret_cast<cudaStream_t>(stream));
}

size_t moeblaze_layernorm_backward_workspace_bytes(const moeblaze_shape* s) {
  if (check_norm_shape(s) != MOEBLAZE_OK) return 0;
  return norm_ws_bytes(*s);
}

moeblaze_status moeblaze_layernorm_backward(const moeblaze_shape* s, const void* dy, const void* sum, const float* mean,
                                            const float* rstd, const float* weight, const void* dsum, void* dx,
                                            float* dweight, float* dbias, void* ws, size_t ws_bytes,
                                            moeblaze_stream stream) {
  moeblaze_status r = check_norm_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if (!ok_ptr(weight) || !ok_ptr4(dweight) || (dbias && !ok_ptr4(dbias))) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L > 0 && (!ok_ptr(dy) || !ok_ptr(sum) || !ok_ptr(dx) || !ok_ptr4(mean) || !ok_ptr4(rstd) ||
                   (dsum && !ok_ptr(dsum))))
    return MOEBLAZE_ERR_INVALID_ARG;
  if (ws_bytes < norm_ws_bytes(*s)) return MOEBLAZE_ERR_WORKSPACE;
  if (s->L > 0 && !ok_ptr(ws)) return MOEBLAZE_ERR_INVALID_ARG;
  return launch_layernorm_backward(*s, dy, sum, mean, rstd, weight, dsum, dx, dweight, dbias, ws,
                                   reinterpret_cast<cudaStream_t>(stream));
}

size_t moeblaze_balance_workspace_bytes(const moeblaze_shape* s) {
  if (check_balance_shape(s) != MOEBLAZE_OK) return 0;
  return balance_ws_bytes(*s);
}

moeblaze_status moeblaze_balance_forward(const moeblaze_shape* s, const float* logits, const int32_t* topk_ids,
                                         const uint8_t* valid, float* losses, int32_t* counts, float* lse, void* ws,
                                         size_t ws_bytes, moeblaze_stream stream) {
  moeblaze_status r = check_balance_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if (!ok_ptr4(losses) || !ok_ptr4(counts)) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L > 0 && (!ok_ptr(logits) || !ok_ptr4(topk_ids) || !ok_ptr4(lse))) return MOEBLAZE_ERR_INVALID_ARG;
  if (ws_bytes < balance_ws_bytes(*s)) return MOEBLAZE_ERR_WORKSPACE;
  if (!ok_ptr(ws)) return MOEBLAZE_ERR_INVALID_ARG;
  return launch_balance_forward(*s, logits, topk_ids, valid, losses, counts, lse, ws,
                                reinterpret_cast<cudaStream_t>(stream));
}

moeblaze_status moeblaze_balance_backward_masked(const moeblaze_shape* s, const float* logits, const float* lse,
                                                 const int32_t* counts, const float* dlosses, const uint8_t* valid,
                                                 const int32_t* topk_ids, const float* gates, const float* dgates,
                                                 int32_t gates_of_all, float* dlogits, moeblaze_stream stream) {
  moeblaze_status r = check_balance_shape(s);
  if (r != MOEBLAZE_OK) return r;
  if (!ok_ptr4(counts) || !ok_ptr4(dlosses)) return MOEBLAZE_ERR_INVALID_ARG;
  // the gates' part: all three arguments or none
  if ((gates != nullptr) != (dgates != nullptr) || (gates != nullptr) != (topk_ids != nullptr))
    return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L > 0 && (!ok_ptr(logits) || !ok_ptr4(lse) || !ok_ptr(dlogits))) return MOEBLAZE_ERR_INVALID_ARG;
  if (gates && (!ok_ptr4(gates) || !ok_ptr4(dgates) || !ok_ptr4(topk_ids))) return MOEBLAZE_ERR_INVALID_ARG;
  return launch_balance_backward(*s, logits, lse, counts, dlosses, topk_ids, gates, dgates, valid, gates_of_all != 0,
                                 dlogits, reinterpret_cast<cudaStream_t>(stream));
}

moeblaze_status moeblaze_balance_backward(const moeblaze_shape* s, const float* logits, const float* lse,
                                          const int32_t* counts, const float* dlosses, const int32_t* topk_ids,
                                          const float* gates, const float* dgates, float* dlogits,
                                          moeblaze_stream stream) {
  return moeblaze_balance_backward_masked(s, logits, lse, counts, dlosses, nullptr, topk_ids, gates, dgates, 0, dlogits,
                                          stream);
}

size_t moeblaze_int4_weight_bytes(int32_t E, int32_t R, int32_t N) {
  return check_int4_matrix(E, R, N, 128) == MOEBLAZE_OK ? (size_t)E * R * N / 2 : 0;
}

size_t moeblaze_int4_scale_bytes(int32_t E, int32_t R, int32_t N, int32_t group) {
  return check_int4_matrix(E, R, N, group) == MOEBLAZE_OK ? (size_t)E * (R / group) * N * 2 : 0;
}

moeblaze_status moeblaze_int4_quantize(int32_t E, int32_t R, int32_t N, int32_t group, int32_t dtype, const void* W,
                                       int8_t* q, void* scales, moeblaze_stream stream) {
  const moeblaze_status r = check_int4_matrix(E, R, N, group);
  if (r != MOEBLAZE_OK) return r;
  if ((dtype != MOEBLAZE_F32 && dtype != MOEBLAZE_BF16) || !ok_ptr(W) || !ok_ptr(q) || !ok_ptr(scales))
    return MOEBLAZE_ERR_INVALID_ARG;
  return launch_int4_quantize(E, R, N, group, dtype, W, q, scales, reinterpret_cast<cudaStream_t>(stream));
}

moeblaze_status moeblaze_int4_pack(int32_t E, int32_t R, int32_t N, int32_t group, const int8_t* q, const void* scales,
                                   void* packed, void* packed_scales, moeblaze_stream stream) {
  const moeblaze_status r = check_int4_matrix(E, R, N, group);
  if (r != MOEBLAZE_OK) return r;
  if (!ok_ptr(q) || !ok_ptr(scales) || !ok_ptr(packed) || !ok_ptr(packed_scales)) return MOEBLAZE_ERR_INVALID_ARG;
  return launch_int4_pack(E, R, N, group, q, scales, packed, packed_scales, reinterpret_cast<cudaStream_t>(stream));
}

moeblaze_status moeblaze_int4_dequantize(int32_t E, int32_t R, int32_t N, int32_t group, const void* packed,
                                         const void* packed_scales, void* W, moeblaze_stream stream) {
  const moeblaze_status r = check_int4_matrix(E, R, N, group);
  if (r != MOEBLAZE_OK) return r;
  if (!ok_ptr(packed) || !ok_ptr(packed_scales) || !ok_ptr(W)) return MOEBLAZE_ERR_INVALID_ARG;
  return launch_int4_dequantize(E, R, N, group, packed, packed_scales, W, reinterpret_cast<cudaStream_t>(stream));
}

size_t moeblaze_int4_workspace_bytes(const moeblaze_shape* s, int32_t group) {
  return check_int4_shape(s, group) == MOEBLAZE_OK ? int4_ws_bytes(*s, group) : 0;
}

moeblaze_status moeblaze_int4_forward(const moeblaze_shape* s, const void* x, const int32_t* topk_ids,
                                      const float* gates, const moeblaze_int4_experts* w, void* y, void* ws,
                                      size_t ws_bytes, moeblaze_stream stream) {
  if (!w) return MOEBLAZE_ERR_INVALID_ARG;
  const moeblaze_status r = check_int4_shape(s, w->group);
  if (r != MOEBLAZE_OK) return r;
  if (!ok_ptr(w->w1) || !ok_ptr(w->s1) || !ok_ptr(w->w3) || !ok_ptr(w->s3)) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->act == MOEBLAZE_SWIGLU && (!ok_ptr(w->w2) || !ok_ptr(w->s2))) return MOEBLAZE_ERR_INVALID_ARG;
  if (s->L > 0 && (!ok_ptr(x) || !ok_ptr(y) || !ok_ptr4(topk_ids) || !ok_ptr4(gates))) return MOEBLAZE_ERR_INVALID_ARG;
  if (ws_bytes < int4_ws_bytes(*s, w->group)) return MOEBLAZE_ERR_WORKSPACE;
  if (s->L > 0 && !ok_ptr(ws)) return MOEBLAZE_ERR_INVALID_ARG;
  return launch_int4_forward(*s, (const __nv_bfloat16*)x, topk_ids, gates, *w, (__nv_bfloat16*)y, ws,
                             reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
