// C ABI of the microscaled 4-bit experts (include/moe.h): argument checks and the launch
// sequence of each call. No entry point allocates device memory.
#include "api_checks.cuh"
#include "fp4.cuh"
#include "moe_layer_ops.h"

using namespace moe;

#define S(st) static_cast<cudaStream_t>(st)
#define BF(p) reinterpret_cast<const bf16*>(p)
#define BFW(p) reinterpret_cast<bf16*>(p)

namespace {

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

}  // namespace

extern "C" {

size_t moe_fp4_scale_bytes(int64_t rows, int32_t blocks) {
  if (rows < 0 || blocks < 0) return 0;
  return ((size_t)blocks + 7) / 8 * 8 * (((size_t)rows + 1) & ~(size_t)1);
}

moe_status_t moe_fp4_quantize_weights(const moe_layer_desc_t* d, const moe_bf16* w1,
                                      const moe_bf16* w2, moe_e2m1x2* w1q, moe_e8m0* w1s,
                                      moe_e2m1x2* w2q, moe_e8m0* w2s, moe_bf16* w1v,
                                      moe_bf16* w2v, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(w1); MOE_PTR(w2); MOE_PTR(w1q); MOE_PTR(w1s); MOE_PTR(w2q); MOE_PTR(w2s);
  MOE_PTR_OPT(w1v); MOE_PTR_OPT(w2v);
  if (!w1v != !w2v) { set_error("w1v and w2v are given together or not at all"); return MOE_ERR_INVALID_ARG; }
  return launch_fp4_quantize_weights(*d, BF(w1), BF(w2), w1q, w1s, w2q, w2s, BFW(w1v), BFW(w2v),
                                     S(stream));
}

moe_status_t moe_permute_fp4(const moe_layer_desc_t* d, const moe_bf16* x, const int32_t* slot,
                             moe_e2m1x2* xq, moe_e8m0* xs, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(x); MOE_PTR(slot); MOE_PTR(xq); MOE_PTR(xs);
  return launch_permute_fp4(*d, BF(x), slot, xq, xs, S(stream));
}

moe_status_t moe_expert_ffn_fwd_fp4(const moe_layer_desc_t* d, const moe_e2m1x2* xq,
                                    const moe_e8m0* xs, const int32_t* off, const moe_e2m1x2* w1q,
                                    const moe_e8m0* w1s, const moe_e2m1x2* w2q,
                                    const moe_e8m0* w2s, moe_bf16* a, moe_bf16* h, moe_e2m1x2* hq,
                                    moe_e8m0* hs, moe_bf16* o, void* ws, size_t ws_bytes,
                                    void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(xq); MOE_PTR(xs); MOE_PTR(off); MOE_PTR(w1q); MOE_PTR(w1s); MOE_PTR(w2q); MOE_PTR(w2s);
  MOE_PTR32_OPT(a); MOE_PTR32_OPT(h); MOE_PTR32(hq); MOE_PTR(hs); MOE_PTR32(o);
  MOE_CHECK(check_ws(*d, ws, ws_bytes));
  return launch_ffn_fwd_fp4(*d, xq, xs, off, Fp4Weights{w1q, w1s, w2q, w2s}, BFW(a), BFW(h), hq,
                            hs, BFW(o), status_of(ws), dep_of(*d, ws), S(stream));
}

moe_status_t moe_layer_forward_fp4(const moe_layer_desc_t* d, const moe_mb_bufs_t* b,
                                   const moe_fp4_bufs_t* q, int32_t save, void* stream) {
  MOE_CHECK(validate(d));
  if (!q) { set_error("4-bit buffer struct is NULL"); return MOE_ERR_INVALID_ARG; }
  if (!b) { set_error("buffer struct is NULL"); return MOE_ERR_INVALID_ARG; }
  MOE_PTR(q->w1q); MOE_PTR(q->w1s); MOE_PTR(q->w2q); MOE_PTR(q->w2s);
  MOE_PTR(q->xq); MOE_PTR(q->xs); MOE_PTR32(q->hq); MOE_PTR(q->hs);
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
  MOE_CHECK(launch_permute_fp4(*d, BF(b->x), b->slot, q->xq, q->xs, st, dep_of(*d, b->ws),
                               status_of(b->ws)));
  MOE_CHECK(launch_ffn_fwd_fp4(*d, q->xq, q->xs, b->off, Fp4Weights{q->w1q, q->w1s, q->w2q, q->w2s},
                               save ? BFW(b->a) : nullptr, save ? BFW(b->h) : nullptr, q->hq, q->hs,
                               BFW(b->o), status_of(b->ws), dep_of(*d, b->ws), st,
                               /*counters_zeroed=*/true));
  return op_combine_mb(*d, b, st);
}

}  // extern "C"
