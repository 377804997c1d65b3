// C ABI of the 8-bit floating-point experts (include/moe.h): argument checks
// and the launch sequence of each call. No entry point allocates device memory.
#include "fp8.cuh"
#include "moe_layer_ops.h"

using namespace moe;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define MOE_CHECK(x)             \
  do {                           \
    moe_status_t _s = (x);       \
    if (_s != MOE_OK) return _s; \
  } while (0)

#define MOE_PTR(p)                                                                             \
  do {                                                                                         \
    if (!(p)) { set_error("%s is NULL", #p); return MOE_ERR_INVALID_ARG; }                     \
    if (!aligned16(p)) { set_error("%s is not 16-byte aligned", #p); return MOE_ERR_INVALID_ARG; } \
  } while (0)

// rows that the expert products move in whole 32-byte sectors
#define MOE_PTR32(p)                                                                           \
  do {                                                                                         \
    MOE_PTR(p);                                                                                \
    if (reinterpret_cast<uintptr_t>(p) & 31u) { set_error("%s is not 32-byte aligned", #p); return MOE_ERR_INVALID_ARG; } \
  } while (0)

#define MOE_PTR_OPT(p)                                                                         \
  do {                                                                                         \
    if ((p) && !aligned16(p)) { set_error("%s is not 16-byte aligned", #p); return MOE_ERR_INVALID_ARG; } \
  } while (0)

#define S(st) static_cast<cudaStream_t>(st)
#define BF(p) reinterpret_cast<const bf16*>(p)
#define BFW(p) reinterpret_cast<bf16*>(p)

moe_status_t check_ws(const moe_layer_desc_t& d, void* ws, size_t ws_bytes) {
  MOE_PTR(ws);
  if (ws_bytes < ws_layout(d).total) {
    set_error("workspace of %zu bytes is smaller than moe_workspace_size() = %zu", ws_bytes,
              ws_layout(d).total);
    return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

int* status_of(void* ws) { return static_cast<int*>(ws); }
int* dep_of(const moe_layer_desc_t& d, void* ws) {
  return reinterpret_cast<int*>(static_cast<char*>(ws) + ws_layout(d).dep);
}

moe_status_t cuda_ok(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MOE_OK;
  set_error("%s: %s", what, cudaGetErrorString(e));
  return MOE_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t moe_fp8_scale_bytes(int64_t rows, int32_t blocks) {
  if (rows < 0 || blocks < 0) return 0;
  return ((size_t)blocks + 3) / 4 * 4 * (size_t)rows;
}

moe_status_t moe_fp8_quantize_weights(const moe_layer_desc_t* d, const moe_bf16* w1,
                                      const moe_bf16* w2, moe_e4m3* w1q, moe_e8m0* w1s,
                                      moe_e4m3* w2q, moe_e8m0* w2s, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(w1); MOE_PTR(w2); MOE_PTR(w1q); MOE_PTR(w1s); MOE_PTR(w2q); MOE_PTR(w2s);
  return launch_fp8_quantize_weights(*d, BF(w1), BF(w2), w1q, w1s, w2q, w2s, S(stream));
}

moe_status_t moe_permute_fp8(const moe_layer_desc_t* d, const moe_bf16* x, const int32_t* slot,
                             moe_e4m3* xq, moe_e8m0* xs, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(x); MOE_PTR(slot); MOE_PTR(xq); MOE_PTR(xs);
  return launch_permute_fp8(*d, BF(x), slot, xq, xs, S(stream));
}

moe_status_t moe_expert_ffn_fwd_fp8(const moe_layer_desc_t* d, const moe_e4m3* xq,
                                    const moe_e8m0* xs, const int32_t* off, const moe_e4m3* w1q,
                                    const moe_e8m0* w1s, const moe_e4m3* w2q, const moe_e8m0* w2s,
                                    moe_bf16* a, moe_bf16* h, moe_e4m3* hq, moe_e8m0* hs,
                                    moe_bf16* o, void* ws, size_t ws_bytes, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(xq); MOE_PTR(xs); MOE_PTR(off); MOE_PTR(w1q); MOE_PTR(w1s); MOE_PTR(w2q); MOE_PTR(w2s);
  if (a) MOE_PTR32(a);
  if (h) MOE_PTR32(h);
  MOE_PTR32(hq); MOE_PTR(hs); MOE_PTR32(o);
  MOE_CHECK(check_ws(*d, ws, ws_bytes));
  return launch_ffn_fwd_fp8(*d, xq, xs, off, Fp8Weights{w1q, w1s, w2q, w2s}, BFW(a), BFW(h), hq,
                            hs, BFW(o), status_of(ws), dep_of(*d, ws), S(stream));
}

moe_status_t moe_combine_bwd_fp8(const moe_layer_desc_t* d, const moe_bf16* dy, const moe_bf16* o,
                                 const int32_t* slot, const float* gates, moe_bf16* d_o,
                                 moe_e4m3* dq, moe_e8m0* ds, float* dgates, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(dy); MOE_PTR(o); MOE_PTR(slot); MOE_PTR(gates); MOE_PTR_OPT(d_o); MOE_PTR(dq);
  MOE_PTR(ds); MOE_PTR(dgates);
  return launch_combine_bwd_fp8(*d, BF(dy), BF(o), slot, gates, BFW(d_o), dq, ds, dgates,
                                S(stream));
}

moe_status_t moe_expert_ffn_bwd_dgrad_fp8(const moe_layer_desc_t* d, const moe_e4m3* dq,
                                          const moe_e8m0* ds, const moe_bf16* a,
                                          const int32_t* off, const moe_e4m3* w1q,
                                          const moe_e8m0* w1s, const moe_e4m3* w2q,
                                          const moe_e8m0* w2s, moe_bf16* da, moe_e4m3* daq,
                                          moe_e8m0* das, moe_bf16* dx_perm, void* ws,
                                          size_t ws_bytes, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(dq); MOE_PTR(ds); MOE_PTR32(a); MOE_PTR(off); MOE_PTR(w1q); MOE_PTR(w1s); MOE_PTR(w2q);
  MOE_PTR(w2s); MOE_PTR32(daq); MOE_PTR(das); MOE_PTR32(dx_perm);
  if (da) MOE_PTR32(da);
  MOE_CHECK(check_ws(*d, ws, ws_bytes));
  return launch_ffn_dgrad_fp8(*d, dq, ds, BF(a), off, Fp8Weights{w1q, w1s, w2q, w2s}, BFW(da), daq,
                              das, BFW(dx_perm), status_of(ws), dep_of(*d, ws), S(stream));
}

}  // extern "C"

namespace {

moe_status_t check_weights(const moe_fp8_bufs_t* q) {
  if (!q) { set_error("8-bit buffer struct is NULL"); return MOE_ERR_INVALID_ARG; }
  MOE_PTR(q->w1q); MOE_PTR(q->w1s); MOE_PTR(q->w2q); MOE_PTR(q->w2s);
  return MOE_OK;
}

Fp8Weights weights(const moe_fp8_bufs_t* q) { return {q->w1q, q->w1s, q->w2q, q->w2s}; }

}  // namespace

extern "C" {

moe_status_t moe_layer_forward_fp8(const moe_layer_desc_t* d, const moe_mb_bufs_t* b,
                                   const moe_fp8_bufs_t* q, int32_t save, void* stream) {
  MOE_CHECK(validate(d));
  MOE_CHECK(check_weights(q));
  MOE_PTR(q->xq); MOE_PTR(q->xs); MOE_PTR32(q->hq); MOE_PTR(q->hs);
  if (!b) { set_error("buffer struct is NULL"); return MOE_ERR_INVALID_ARG; }
  MOE_PTR(b->x); MOE_PTR(b->w_r); MOE_PTR_OPT(b->bias); MOE_PTR_OPT(b->logits); MOE_PTR(b->idx);
  MOE_PTR(b->gates); MOE_PTR(b->cnt); MOE_PTR(b->off); MOE_PTR(b->slot); MOE_PTR(b->row_src);
  MOE_PTR(b->cnt_re); MOE_PTR(b->rank_off); MOE_PTR32(b->o); MOE_PTR(b->y);
  if (save) { MOE_PTR(b->x_perm); MOE_PTR32(b->a); MOE_PTR32(b->h); }
  MOE_CHECK(check_ws(*d, b->ws, b->ws_bytes));
  const WsLayout w = ws_layout(*d);
  char* ws = static_cast<char*>(b->ws);
  cudaStream_t st = S(stream);
  if (save) {
    MOE_CHECK(op_dispatch(*d, b, st));
  } else {
    float* z = b->logits ? b->logits : reinterpret_cast<float*>(ws + w.logits);
    MOE_CHECK(launch_route(*d, BF(b->x), BF(b->w_r), b->bias, z, b->idx, b->gates,
                           status_of(b->ws), st));
    MOE_CHECK(launch_layout(*d, b->idx, b->cnt, b->off, b->slot, b->row_src, b->cnt_re,
                            b->rank_off, reinterpret_cast<int*>(ws + w.hist), status_of(b->ws),
                            st));
  }
  MOE_CHECK(launch_permute_fp8(*d, BF(b->x), b->slot, q->xq, q->xs, st));
  MOE_CHECK(launch_ffn_fwd_fp8(*d, q->xq, q->xs, b->off, weights(q), save ? BFW(b->a) : nullptr,
                               save ? BFW(b->h) : nullptr, q->hq, q->hs, BFW(b->o),
                               status_of(b->ws), dep_of(*d, b->ws), st));
  return op_combine_mb(*d, b, st);
}

moe_status_t moe_layer_backward_fp8(const moe_layer_desc_t* d, const moe_mb_bufs_t* b,
                                    const moe_fp8_bufs_t* q, int32_t run_wgrad, void* stream) {
  MOE_CHECK(validate(d));
  MOE_CHECK(check_weights(q));
  MOE_PTR(q->dq); MOE_PTR(q->ds); MOE_PTR32(q->daq); MOE_PTR(q->das);
  if (!b) { set_error("buffer struct is NULL"); return MOE_ERR_INVALID_ARG; }
  MOE_PTR(b->x); MOE_PTR(b->dy); MOE_PTR(b->w_r); MOE_PTR(b->idx); MOE_PTR(b->gates);
  MOE_PTR(b->off); MOE_PTR(b->slot); MOE_PTR(b->row_src); MOE_PTR32(b->a); MOE_PTR(b->o);
  MOE_PTR(b->dgates); MOE_PTR32(b->dx_perm); MOE_PTR(b->dx); MOE_PTR(b->dw_r);
  if (run_wgrad) {  // the weight gradients are products of the bf16 rows
    MOE_PTR(b->x_perm); MOE_PTR(b->h); MOE_PTR(b->d_o); MOE_PTR32(b->da);
    if (d->flags & MOE_FLAG_WGRAD_ACCUM_FP32) { MOE_PTR(b->main_dw1); MOE_PTR(b->main_dw2); }
    else { MOE_PTR(b->dw1); MOE_PTR(b->dw2); }
  } else {
    MOE_PTR_OPT(b->d_o);
    if (b->da) MOE_PTR32(b->da);
  }
  MOE_CHECK(check_ws(*d, b->ws, b->ws_bytes));
  cudaStream_t st = S(stream);
  // it clears dW_r's chunk counters, which follow the experts' counters
  MOE_CHECK(launch_combine_bwd_fp8(*d, BF(b->dy), BF(b->o), b->slot, b->gates, BFW(b->d_o), q->dq,
                                   q->ds, b->dgates, st, dep_of(*d, b->ws) + d->E, dep_ints(*d) - d->E));
  MOE_CHECK(launch_ffn_dgrad_fp8(*d, q->dq, q->ds, BF(b->a), b->off, weights(q), BFW(b->da),
                                 q->daq, q->das, BFW(b->dx_perm), status_of(b->ws),
                                 dep_of(*d, b->ws), st));
  if (!run_wgrad) return op_dispatch_bwd_mb(*d, b, st);
  if (profiling_active()) {
    MOE_CHECK(op_dispatch_bwd_mb(*d, b, st));
    return op_wgrad_mb(*d, b, 0, st);
  }
  // as in moe_layer_backward: the weight gradients on the side stream beside
  // the dispatch backward, joined before the call returns
  CopyLane* cl = copy_lane();
  if (!cl) return MOE_ERR_CUDA;
  std::lock_guard<std::mutex> lk(cl->side_mu);
  MOE_CHECK(cuda_ok(cudaEventRecord(cl->fork, st), "side stream"));
  MOE_CHECK(cuda_ok(cudaStreamWaitEvent(cl->side, cl->fork, 0), "side stream"));
  moe_status_t s = op_wgrad_mb(*d, b, 0, cl->side);
  const moe_status_t joined = cuda_ok(cudaEventRecord(cl->join, cl->side), "side stream");
  if (s == MOE_OK) s = joined;
  if (s == MOE_OK) s = op_dispatch_bwd_mb(*d, b, st);
  const moe_status_t waits = cuda_ok(cudaStreamWaitEvent(st, cl->join, 0), "side stream");
  return s != MOE_OK ? s : waits;
}

}  // extern "C"
