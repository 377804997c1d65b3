// C ABI entry points (include/moe.h): argument checks, workspace carving and
// the launch sequence of each call. No entry point allocates device memory.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "api_checks.cuh"
#include "moe_internal.cuh"
#include "moe_layer_ops.h"

namespace moe {

namespace {
thread_local char g_err[512] = "";

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
}  // namespace

void set_error(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
}

moe_status_t check_launch(const char* what) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("%s: %s", what, cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

CopyLane* copy_lane() {
  constexpr int kMaxDevices = 64;
  static CopyLane lanes[kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    set_error("no usable current device for the copy stream");
    return nullptr;
  }
  std::lock_guard<std::mutex> lk(mu);
  CopyLane& l = lanes[dev];
  if (!l.stream) {
    cudaError_t e = cudaStreamCreateWithFlags(&l.stream, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&l.side, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&l.d2h, cudaStreamNonBlocking);
    for (int s = 0; s < 2; ++s)
      for (cudaEvent_t* ev : {&l.in_ready[s], &l.step_done[s],
                              &l.out_done[s]})
        if (e == cudaSuccess) e = cudaEventCreateWithFlags(ev, cudaEventDisableTiming);
    for (cudaEvent_t* ev : {&l.start, &l.dy_in, &l.fwd_done, &l.y_out, &l.dx_ready, &l.fork,
                            &l.join})
      if (e == cudaSuccess) e = cudaEventCreateWithFlags(ev, cudaEventDisableTiming);
    if (e != cudaSuccess) {
      set_error("copy stream setup: %s", cudaGetErrorString(e));
      l.stream = nullptr;
      return nullptr;
    }
  }
  return &l;
}

int device_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
  return n > 0 ? n : 1;
}

// ints of the ws counter area (see WsLayout::dep)
int dep_ints(const moe_layer_desc_t& d) { return d.E + d.E * ceil_div(d.H / 8, 256); }

WsLayout ws_layout(const moe_layer_desc_t& d) {
  WsLayout w;
  const long long N = (long long)d.T * d.k;
  const int nb = d.T > 0 ? ceil_div(d.T, kLayoutTokensPerBlock) : 1;
  const long long chunks = (N + kRouteBwdRowsPerChunk - 1) / kRouteBwdRowsPerChunk + d.E;
  size_t o = 0;
  w.status = o;
  o += kStatusBytes;
  w.logits = o;
  o = align256(o + (size_t)d.T * d.E * sizeof(float));
  w.hist = o;  // dispatch layout: per-block expert counts, then a row of totals
  o = align256(o + (size_t)(nb + 1) * d.E * sizeof(int));
  w.dz = o;
  o = align256(o + (size_t)N * sizeof(float));
  w.dwr_part = o;
  o = align256(o + (size_t)chunks * d.H * sizeof(float));
  w.dep = o;
  o = align256(o + (size_t)dep_ints(d) * sizeof(int));
  w.fhist = o;  // fused dispatch: per-tile expert counts (tiles of >= 4 tokens) + totals
  o = align256(o + ((size_t)(d.T + 3) / 4 + 1) * d.E * sizeof(int));
  w.bar = o;
  o = align256(o + sizeof(int));
  w.total = o;
  return w;
}

moe_status_t validate(const moe_layer_desc_t* d) {
  if (!d) { set_error("descriptor is NULL"); return MOE_ERR_INVALID_ARG; }
  if (d->T < 0 || d->H <= 0 || d->E <= 0 || d->k <= 0 || d->F <= 0 || d->R <= 0) {
    set_error("shape must have T >= 0 and H, E, k, F, R > 0 (T=%d H=%d E=%d k=%d F=%d R=%d)",
              d->T, d->H, d->E, d->k, d->F, d->R);
    return MOE_ERR_INVALID_ARG;
  }
  if (d->k > d->E) { set_error("k=%d exceeds E=%d: the k experts of a token must be distinct", d->k, d->E); return MOE_ERR_INVALID_ARG; }
  if (d->E % d->R) { set_error("E=%d is not a multiple of R=%d", d->E, d->R); return MOE_ERR_INVALID_ARG; }
  if (d->mode != MOE_ROUTE_SOFTMAX_TOPK && d->mode != MOE_ROUTE_FORCED_BALANCED) {
    set_error("unknown routing mode %d", d->mode); return MOE_ERR_INVALID_ARG;
  }
  if ((d->flags & ~MOE_FLAG_WGRAD_ACCUM_FP32) != 0) {
    set_error("unknown flags 0x%x", (unsigned)d->flags);
    return MOE_ERR_INVALID_ARG;
  }
  if (d->H % 64 || d->F % 64) {
    set_error("H=%d and F=%d must be multiples of 64", d->H, d->F); return MOE_ERR_UNSUPPORTED;
  }
  if (d->E > 256 || d->k > 32) { set_error("E <= 256 and k <= 32 are supported (E=%d k=%d)", d->E, d->k); return MOE_ERR_UNSUPPORTED; }
  if (d->H > 16384 || d->F > 16384) { set_error("H, F <= 16384 are supported"); return MOE_ERR_UNSUPPORTED; }
  if ((long long)d->T * d->k >= (1ll << 31) || (long long)d->T * d->H >= (1ll << 40)) {
    set_error("T*k must stay below 2^31"); return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

static moe_status_t check_ws(const moe_layer_desc_t& d, void* ws, size_t ws_bytes) {
  MOE_PTR(ws);
  if (ws_bytes < ws_layout(d).total) {
    set_error("workspace of %zu bytes is smaller than moe_workspace_size() = %zu", ws_bytes,
              ws_layout(d).total);
    return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

static int* status_of(void* ws) { return reinterpret_cast<int*>(static_cast<char*>(ws)); }
template <typename T>
static T* ws_at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

// ------------------------------------------------------------------ internal ops
moe_status_t op_route(const moe_layer_desc_t& d, const bf16* x, const bf16* w_r, const float* bias,
                      float* logits, int32_t* idx, float* gates, void* ws, cudaStream_t st) {
  float* z = logits ? logits : ws_at<float>(ws, ws_layout(d).logits);
  return launch_route(d, x, w_r, bias, z, idx, gates, status_of(ws), st);
}

moe_status_t op_layout(const moe_layer_desc_t& d, const int32_t* idx, int32_t* cnt, int32_t* off,
                       int32_t* slot, int32_t* row_src, int32_t* cnt_re, int32_t* rank_off,
                       void* ws, cudaStream_t st) {
  return launch_layout(d, idx, cnt, off, slot, row_src, cnt_re, rank_off,
                       ws_at<int>(ws, ws_layout(d).hist), status_of(ws), st);
}

// counters_zeroed: the chain's per-expert counters in ws were cleared by the
// launch just before it on the stream (the layer path's fused dispatch, or
// combine backward for the dgrad chain), so the chain needs no memset.
moe_status_t op_ffn_fwd(const moe_layer_desc_t& d, const bf16* x_perm, const int32_t* off,
                        const bf16* w1, const bf16* w2, bf16* a, bf16* h, bf16* o, void* ws,
                        int max_ctas, cudaStream_t st, bool counters_zeroed = false) {
  GemmArgs g = {};
  g.mode = GEMM_FC1_FWD;
  g.A = x_perm;
  g.B = w1;
  g.off = off;
  g.out0 = a;
  g.out1 = h;
  g.status = status_of(ws);
  g.max_ctas = max_ctas;
  g.dep = ws_at<int>(ws, ws_layout(d).dep);
  GemmArgs g2 = g;
  g2.mode = GEMM_FC2_FWD;
  g2.A = h;
  g2.B = w2;
  g2.out0 = o;
  g2.out1 = nullptr;
  // FC2 tiles of an expert start as soon as its FC1 tiles are stored
  return launch_grouped_gemm_chain(d, g, g2, st, counters_zeroed);
}

moe_status_t op_dgrad(const moe_layer_desc_t& d, const bf16* d_o, const bf16* a,
                      const int32_t* off, const bf16* w1, const bf16* w2, bf16* da,
                      bf16* dx_perm, void* ws, int max_ctas, cudaStream_t st,
                      bool counters_zeroed = false) {
  GemmArgs g = {};
  g.mode = GEMM_FC2_DGRAD;
  g.A = d_o;
  g.B = w2;
  g.off = off;
  g.out0 = da;
  g.aux = a;
  g.status = status_of(ws);
  g.max_ctas = max_ctas;
  g.dep = ws_at<int>(ws, ws_layout(d).dep);
  GemmArgs g2 = g;
  g2.mode = GEMM_FC1_DGRAD;
  g2.A = da;
  g2.B = w1;
  g2.out0 = dx_perm;
  g2.aux = nullptr;
  // FC1 dgrad tiles of an expert start as soon as its da is stored
  return launch_grouped_gemm_chain(d, g, g2, st, counters_zeroed);
}

// One weight gradient (GEMM_WGRAD_W1: dW1 from da and x_perm; GEMM_WGRAD_W2:
// dW2 from d_o and h): stored as bf16 into dw, or, when main is given, added
// in fp32 into that main gradient (dw unused).
moe_status_t op_wgrad_one(const moe_layer_desc_t& d, int mode, const bf16* A, const bf16* B,
                          const int32_t* off, bf16* dw, float* main, void* ws, int max_ctas,
                          cudaStream_t st) {
  GemmArgs g = {};
  g.mode = mode;
  g.A = A;
  g.B = B;
  g.off = off;
  if (mode == GEMM_WGRAD_W1) g.out0 = main ? nullptr : dw;
  else g.out1 = main ? nullptr : dw;
  g.acc = main;
  g.status = status_of(ws);
  g.max_ctas = max_ctas;
  return launch_grouped_gemm(d, g, st);
}

// Weight gradients: stored as bf16 into dw1/dw2, or, when main_dw1/main_dw2
// are given, added in fp32 into those main gradients (dw1/dw2 unused).
moe_status_t op_wgrad(const moe_layer_desc_t& d, const bf16* x_perm, const bf16* h,
                      const bf16* d_o, const bf16* da, const int32_t* off, bf16* dw1, bf16* dw2,
                      float* main_dw1, float* main_dw2, void* ws, int max_ctas, cudaStream_t st) {
  if (!main_dw1 && !main_dw2 && (long long)d.T * d.k > 0) {
    // both weight gradients in one persistent launch (bf16 outputs)
    GemmArgs g1 = {};
    g1.mode = GEMM_WGRAD_W1;
    g1.A = da;
    g1.B = x_perm;
    g1.off = off;
    g1.out0 = dw1;
    g1.status = status_of(ws);
    g1.max_ctas = max_ctas;
    GemmArgs g2 = g1;
    g2.mode = GEMM_WGRAD_W2;
    g2.A = d_o;
    g2.B = h;
    g2.out0 = nullptr;
    g2.out1 = dw2;
    return launch_grouped_gemm_chain(d, g1, g2, st);
  }
  MOE_CHECK(op_wgrad_one(d, GEMM_WGRAD_W1, da, x_perm, off, dw1, main_dw1, ws, max_ctas, st));
  return op_wgrad_one(d, GEMM_WGRAD_W2, d_o, h, off, dw2, main_dw2, ws, max_ctas, st);
}

// cnt_zeroed: dW_r's chunk counters in ws were cleared by an earlier launch
// on the stream (the layer path's combine backward), so no memset is issued.
moe_status_t op_route_bwd(const moe_layer_desc_t& d, const float* dgates, const float* gates,
                          const int32_t* idx, const bf16* x, const bf16* w_r,
                          const int32_t* row_src, const int32_t* off, const float* dx32,
                          const bf16* dx_perm, const int32_t* slot, bf16* dx, float* dw_r,
                          void* ws, cudaStream_t st, bool cnt_zeroed = false) {
  const WsLayout w = ws_layout(d);
  return launch_route_bwd(d, dgates, gates, idx, x, w_r, row_src, off, dx32, dx_perm, slot, dx,
                          dw_r, ws_at<float>(ws, w.dz), ws_at<float>(ws, w.dwr_part),
                          ws_at<int>(ws, w.dep) + d.E, cnt_zeroed, status_of(ws), st);
}

// Route + dispatch layout + permute: one cooperative launch when the block
// routes every expert of its tokens (E <= 128), else the three launches.
moe_status_t op_dispatch_all(const moe_layer_desc_t& d, const bf16* x, const bf16* w_r,
                             const float* bias, float* logits, int32_t* idx, float* gates,
                             int32_t* cnt, int32_t* off, int32_t* slot, int32_t* row_src,
                             int32_t* cnt_re, int32_t* rank_off, bf16* x_perm, void* ws,
                             cudaStream_t st, int max_ctas = 0) {
  if (d.T > 0 && d.E <= 128) {
    const WsLayout w = ws_layout(d);
    float* z = logits ? logits : ws_at<float>(ws, w.logits);
    // it also clears the forward chain's counters (op_ffn_fwd_mb relies on it)
    return launch_dispatch_fused(d, x, w_r, bias, z, idx, gates, cnt, off, slot, row_src, cnt_re,
                                 rank_off, x_perm, ws_at<int>(ws, w.fhist), ws_at<int>(ws, w.bar),
                                 status_of(ws), st, ws_at<int>(ws, w.dep), d.E, max_ctas);
  }
  MOE_CHECK(op_route(d, x, w_r, bias, logits, idx, gates, ws, st));
  MOE_CHECK(op_layout(d, idx, cnt, off, slot, row_src, cnt_re, rank_off, ws, st));
  return launch_permute(d, x, row_src, x_perm, st);
}

moe_status_t op_dispatch(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, cudaStream_t st,
                         int max_ctas) {
  return op_dispatch_all(d, reinterpret_cast<const bf16*>(b->x),
                         reinterpret_cast<const bf16*>(b->w_r), b->bias, b->logits, b->idx,
                         b->gates, b->cnt, b->off, b->slot, b->row_src, b->cnt_re, b->rank_off,
                         reinterpret_cast<bf16*>(b->x_perm), b->ws, st, max_ctas);
}

moe_status_t op_ffn_fwd_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, int max_ctas,
                           cudaStream_t st) {
  // the fused dispatch (T > 0, E <= 128) that precedes this phase has cleared
  // the chain's counters; the three-launch dispatch has not
  return op_ffn_fwd(d, reinterpret_cast<const bf16*>(b->x_perm), b->off,
                    reinterpret_cast<const bf16*>(b->w1), reinterpret_cast<const bf16*>(b->w2),
                    reinterpret_cast<bf16*>(b->a), reinterpret_cast<bf16*>(b->h),
                    reinterpret_cast<bf16*>(b->o), b->ws, max_ctas, st, d.T > 0 && d.E <= 128);
}

moe_status_t op_combine_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, cudaStream_t st) {
  return launch_combine(d, reinterpret_cast<const bf16*>(b->o), b->slot, b->gates,
                        reinterpret_cast<bf16*>(b->y), st);
}

moe_status_t op_combine_bwd_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b,
                               cudaStream_t st) {
  // it also clears the dgrad chain's counters and dW_r's chunk counters
  // (op_dgrad_mb and op_dispatch_bwd_mb rely on it)
  return launch_combine_bwd(d, reinterpret_cast<const bf16*>(b->dy),
                            reinterpret_cast<const bf16*>(b->o), b->slot, b->gates,
                            reinterpret_cast<bf16*>(b->d_o), b->dgates, st,
                            ws_at<int>(b->ws, ws_layout(d).dep), dep_ints(d));
}

moe_status_t op_dgrad_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, int max_ctas,
                         cudaStream_t st) {
  return op_dgrad(d, reinterpret_cast<const bf16*>(b->d_o), reinterpret_cast<const bf16*>(b->a),
                  b->off, reinterpret_cast<const bf16*>(b->w1),
                  reinterpret_cast<const bf16*>(b->w2), reinterpret_cast<bf16*>(b->da),
                  reinterpret_cast<bf16*>(b->dx_perm), b->ws, max_ctas, st,
                  /*counters_zeroed=*/true);
}

moe_status_t op_dispatch_bwd_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b,
                                cudaStream_t st) {
  // the dispatch backward (row sums of dx_perm) is fused into the router's
  // dx pass; dx32 is not written on this path
  return op_route_bwd(d, b->dgates, b->gates, b->idx, reinterpret_cast<const bf16*>(b->x),
                      reinterpret_cast<const bf16*>(b->w_r), b->row_src, b->off, nullptr,
                      reinterpret_cast<const bf16*>(b->dx_perm), b->slot,
                      reinterpret_cast<bf16*>(b->dx), b->dw_r, b->ws, st,
                      /*cnt_zeroed=*/true);
}

moe_status_t op_wgrad_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, int max_ctas,
                         cudaStream_t st) {
  const bool acc = (d.flags & MOE_FLAG_WGRAD_ACCUM_FP32) != 0;
  return op_wgrad(d, reinterpret_cast<const bf16*>(b->x_perm), reinterpret_cast<const bf16*>(b->h),
                  reinterpret_cast<const bf16*>(b->d_o), reinterpret_cast<const bf16*>(b->da),
                  b->off, reinterpret_cast<bf16*>(b->dw1), reinterpret_cast<bf16*>(b->dw2),
                  acc ? b->main_dw1 : nullptr, acc ? b->main_dw2 : nullptr, b->ws, max_ctas, st);
}

moe_status_t check_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, bool bwd) {
  if (!b) { set_error("buffer struct is NULL"); return MOE_ERR_INVALID_ARG; }
  MOE_PTR(b->x); MOE_PTR(b->w_r); MOE_PTR(b->w1); MOE_PTR(b->w2); MOE_PTR_OPT(b->bias);
  MOE_PTR_OPT(b->logits); MOE_PTR(b->idx); MOE_PTR(b->gates); MOE_PTR(b->cnt); MOE_PTR(b->off);
  MOE_PTR(b->slot); MOE_PTR(b->row_src); MOE_PTR(b->cnt_re); MOE_PTR(b->rank_off);
  MOE_PTR(b->x_perm); MOE_PTR(b->a); MOE_PTR(b->h); MOE_PTR(b->o); MOE_PTR(b->y);
  if (bwd) {
    MOE_PTR(b->dy); MOE_PTR(b->d_o); MOE_PTR(b->dgates); MOE_PTR(b->da); MOE_PTR(b->dx_perm);
    MOE_PTR(b->dx32); MOE_PTR(b->dx); MOE_PTR(b->dw_r);
    if (d.flags & MOE_FLAG_WGRAD_ACCUM_FP32) {
      MOE_PTR(b->main_dw1); MOE_PTR(b->main_dw2);
    } else {
      MOE_PTR(b->dw1); MOE_PTR(b->dw2);
    }
  }
  return check_ws(d, b->ws, b->ws_bytes);
}

}  // namespace moe

using namespace moe;

#define S(st) static_cast<cudaStream_t>(st)
#define BF(p) reinterpret_cast<const bf16*>(p)
#define BFW(p) reinterpret_cast<bf16*>(p)

extern "C" {

int32_t moe_abi_version(void) { return 2; }  // 2: moe_mb_bufs_t gained main_dw1, main_dw2

const char* moe_last_error(void) { return g_err; }

moe_status_t moe_layer_desc_validate(const moe_layer_desc_t* d) {
  moe_status_t s = validate(d);
  if (s == MOE_OK) g_err[0] = 0;
  return s;
}

size_t moe_workspace_size(const moe_layer_desc_t* d) {
  if (validate(d) != MOE_OK) return 0;
  return ws_layout(*d).total;
}

moe_status_t moe_device_status(const moe_layer_desc_t* d, void* ws, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(ws);
  int h[ST_NUM] = {0};
  cudaError_t e = cudaStreamSynchronize(S(stream));
  if (e == cudaSuccess) e = cudaMemcpy(h, ws, sizeof(h), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(ws, 0, sizeof(h));
  if (e != cudaSuccess) {
    set_error("moe_device_status: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  if (h[ST_TIMEOUT]) {
    set_error("a pipeline wait ran out of time (site %d)", h[ST_TIMEOUT]);
    return MOE_ERR_TIMEOUT;
  }
  if (h[ST_BAD_INDEX]) {
    set_error("%d out-of-range expert or row indices were skipped", h[ST_BAD_INDEX]);
    return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

moe_status_t moe_route(const moe_layer_desc_t* d, const moe_bf16* x, const moe_bf16* w_r,
                       const float* bias, float* logits, int32_t* idx, float* gates, void* ws,
                       size_t ws_bytes, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(x); MOE_PTR(w_r); MOE_PTR_OPT(bias); MOE_PTR_OPT(logits); MOE_PTR(idx); MOE_PTR(gates);
  MOE_CHECK(check_ws(*d, ws, ws_bytes));
  return op_route(*d, BF(x), BF(w_r), bias, logits, idx, gates, ws, S(stream));
}

moe_status_t moe_dispatch_fused(const moe_layer_desc_t* d, const moe_bf16* x, const moe_bf16* w_r,
                                const float* bias, float* logits, int32_t* idx, float* gates,
                                int32_t* cnt, int32_t* off, int32_t* slot, int32_t* row_src,
                                int32_t* cnt_re, int32_t* rank_off, moe_bf16* x_perm, void* ws,
                                size_t ws_bytes, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(x); MOE_PTR(w_r); MOE_PTR_OPT(bias); MOE_PTR_OPT(logits); MOE_PTR(idx); MOE_PTR(gates);
  MOE_PTR(cnt); MOE_PTR(off); MOE_PTR(slot); MOE_PTR(row_src); MOE_PTR(cnt_re);
  MOE_PTR(rank_off); MOE_PTR(x_perm);
  MOE_CHECK(check_ws(*d, ws, ws_bytes));
  return op_dispatch_all(*d, BF(x), BF(w_r), bias, logits, idx, gates, cnt, off, slot, row_src,
                         cnt_re, rank_off, BFW(x_perm), ws, S(stream));
}

moe_status_t moe_dispatch_layout(const moe_layer_desc_t* d, const int32_t* idx, int32_t* cnt,
                                 int32_t* off, int32_t* slot, int32_t* row_src, int32_t* cnt_re,
                                 int32_t* rank_off, void* ws, size_t ws_bytes, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(idx); MOE_PTR(cnt); MOE_PTR(off); MOE_PTR(slot); MOE_PTR(row_src); MOE_PTR(cnt_re);
  MOE_PTR(rank_off);
  MOE_CHECK(check_ws(*d, ws, ws_bytes));
  return op_layout(*d, idx, cnt, off, slot, row_src, cnt_re, rank_off, ws, S(stream));
}

moe_status_t moe_permute(const moe_layer_desc_t* d, const moe_bf16* x, const int32_t* row_src,
                         moe_bf16* x_perm, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(x); MOE_PTR(row_src); MOE_PTR(x_perm);
  return launch_permute(*d, BF(x), row_src, BFW(x_perm), S(stream));
}

moe_status_t moe_expert_ffn_fwd(const moe_layer_desc_t* d, const moe_bf16* x_perm,
                                const int32_t* off, const moe_bf16* w1, const moe_bf16* w2,
                                moe_bf16* a, moe_bf16* h, moe_bf16* o, void* ws, size_t ws_bytes,
                                void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(x_perm); MOE_PTR(off); MOE_PTR(w1); MOE_PTR(w2); MOE_PTR(a); MOE_PTR(h); MOE_PTR(o);
  MOE_CHECK(check_ws(*d, ws, ws_bytes));
  return op_ffn_fwd(*d, BF(x_perm), off, BF(w1), BF(w2), BFW(a), BFW(h), BFW(o), ws, 0, S(stream));
}

moe_status_t moe_combine(const moe_layer_desc_t* d, const moe_bf16* o, const int32_t* slot,
                         const float* gates, moe_bf16* y, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(o); MOE_PTR(slot); MOE_PTR(gates); MOE_PTR(y);
  return launch_combine(*d, BF(o), slot, gates, BFW(y), S(stream));
}

moe_status_t moe_combine_bwd(const moe_layer_desc_t* d, const moe_bf16* dy, const moe_bf16* o,
                             const int32_t* slot, const float* gates, moe_bf16* d_o,
                             float* dgates, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(dy); MOE_PTR(o); MOE_PTR(slot); MOE_PTR(gates); MOE_PTR(d_o); MOE_PTR(dgates);
  return launch_combine_bwd(*d, BF(dy), BF(o), slot, gates, BFW(d_o), dgates, S(stream));
}

moe_status_t moe_expert_ffn_bwd_dgrad(const moe_layer_desc_t* d, const moe_bf16* d_o,
                                      const moe_bf16* a, const int32_t* off, const moe_bf16* w1,
                                      const moe_bf16* w2, moe_bf16* da, moe_bf16* dx_perm,
                                      void* ws, size_t ws_bytes, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(d_o); MOE_PTR(a); MOE_PTR(off); MOE_PTR(w1); MOE_PTR(w2); MOE_PTR(da); MOE_PTR(dx_perm);
  MOE_CHECK(check_ws(*d, ws, ws_bytes));
  return op_dgrad(*d, BF(d_o), BF(a), off, BF(w1), BF(w2), BFW(da), BFW(dx_perm), ws, 0,
                  S(stream));
}

moe_status_t moe_expert_ffn_bwd_wgrad(const moe_layer_desc_t* d, const moe_bf16* x_perm,
                                      const moe_bf16* h, const moe_bf16* d_o, const moe_bf16* da,
                                      const int32_t* off, moe_bf16* dw1, moe_bf16* dw2, void* ws,
                                      size_t ws_bytes, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(x_perm); MOE_PTR(h); MOE_PTR(d_o); MOE_PTR(da); MOE_PTR(off); MOE_PTR(dw1); MOE_PTR(dw2);
  MOE_CHECK(check_ws(*d, ws, ws_bytes));
  return op_wgrad(*d, BF(x_perm), BF(h), BF(d_o), BF(da), off, BFW(dw1), BFW(dw2), nullptr,
                  nullptr, ws, 0, S(stream));
}

moe_status_t moe_expert_ffn_bwd_wgrad_accum(const moe_layer_desc_t* d, const moe_bf16* x_perm,
                                            const moe_bf16* h, const moe_bf16* d_o,
                                            const moe_bf16* da, const int32_t* off,
                                            float* main_dw1, float* main_dw2, void* ws,
                                            size_t ws_bytes, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(x_perm); MOE_PTR(h); MOE_PTR(d_o); MOE_PTR(da); MOE_PTR(off); MOE_PTR(main_dw1);
  MOE_PTR(main_dw2);
  MOE_CHECK(check_ws(*d, ws, ws_bytes));
  return op_wgrad(*d, BF(x_perm), BF(h), BF(d_o), BF(da), off, nullptr, nullptr, main_dw1,
                  main_dw2, ws, 0, S(stream));
}

moe_status_t moe_permute_bwd(const moe_layer_desc_t* d, const moe_bf16* dx_perm,
                             const int32_t* slot, float* dx32, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(dx_perm); MOE_PTR(slot); MOE_PTR(dx32);
  return launch_permute_bwd(*d, BF(dx_perm), slot, dx32, S(stream));
}

moe_status_t moe_route_bwd(const moe_layer_desc_t* d, const float* dgates, const float* gates,
                           const int32_t* idx, const moe_bf16* x, const moe_bf16* w_r,
                           const int32_t* row_src, const int32_t* off, const float* dx32,
                           moe_bf16* dx, float* dw_r, void* ws, size_t ws_bytes, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(dgates); MOE_PTR(gates); MOE_PTR(idx); MOE_PTR(x); MOE_PTR(w_r); MOE_PTR(row_src);
  MOE_PTR(off); MOE_PTR(dx32); MOE_PTR(dx); MOE_PTR(dw_r);
  MOE_CHECK(check_ws(*d, ws, ws_bytes));
  return op_route_bwd(*d, dgates, gates, idx, BF(x), BF(w_r), row_src, off, dx32, nullptr,
                      nullptr, BFW(dx), dw_r, ws, S(stream));
}

moe_status_t moe_layer_forward(const moe_layer_desc_t* d, const moe_mb_bufs_t* b, void* stream) {
  MOE_CHECK(validate(d));
  MOE_CHECK(check_mb(*d, b, false));
  MOE_CHECK(op_dispatch(*d, b, S(stream)));
  MOE_CHECK(op_ffn_fwd_mb(*d, b, 0, S(stream)));
  return op_combine_mb(*d, b, S(stream));
}

}  // extern "C"

// The layer backward on `st`. When dx_ready is given, it is recorded on `st`
// as soon as dx is complete (after the dispatch backward, before the weight
// gradients are joined), so that a caller can start copying dx out while the
// weight gradients still run.
static moe_status_t layer_backward(const moe_layer_desc_t* d, const moe_mb_bufs_t* b,
                                   int32_t run_wgrad, cudaStream_t st, cudaEvent_t dx_ready) {
  auto mark_dx = [&]() -> moe_status_t {
    if (!dx_ready) return MOE_OK;
    const cudaError_t e = cudaEventRecord(dx_ready, st);
    if (e != cudaSuccess) {
      set_error("cudaEventRecord: %s", cudaGetErrorString(e));
      return MOE_ERR_CUDA;
    }
    return MOE_OK;
  };
  MOE_CHECK(op_combine_bwd_mb(*d, b, st));
  MOE_CHECK(op_dgrad_mb(*d, b, 0, st));
  if (!run_wgrad) {
    MOE_CHECK(op_dispatch_bwd_mb(*d, b, st));
    return mark_dx();
  }
  if (profiling_active()) {
    // per-launch timing: every launch in order on `stream`, each timed alone
    MOE_CHECK(op_dispatch_bwd_mb(*d, b, st));
    MOE_CHECK(mark_dx());
    return op_wgrad_mb(*d, b, 0, st);
  }
  // fork: the weight gradients (write-heavy) on the side stream beside the
  // dispatch backward (read-heavy) on `stream`; join before return. Measured
  // on the 4096-token layer: 1.070 ms per step against 1.084 ms in order.
  CopyLane* cl = copy_lane();
  if (!cl) return MOE_ERR_CUDA;
  std::lock_guard<std::mutex> lk(cl->side_mu);
  cudaError_t e = cudaEventRecord(cl->fork, st);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(cl->side, cl->fork, 0);
  if (e != cudaSuccess) {
    set_error("side stream: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  MOE_CHECK(op_wgrad_mb(*d, b, 0, cl->side));
  e = cudaEventRecord(cl->join, cl->side);
  if (e != cudaSuccess) {
    set_error("side stream: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  moe_status_t s = op_dispatch_bwd_mb(*d, b, st);
  if (s == MOE_OK) s = mark_dx();
  e = cudaStreamWaitEvent(st, cl->join, 0);
  if (e != cudaSuccess) {
    set_error("side stream: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return s;
}

extern "C" {

moe_status_t moe_layer_backward(const moe_layer_desc_t* d, const moe_mb_bufs_t* b,
                                int32_t run_wgrad, void* stream) {
  MOE_CHECK(validate(d));
  MOE_CHECK(check_mb(*d, b, true));
  return layer_backward(d, b, run_wgrad, S(stream), nullptr);
}

moe_status_t moe_layer_step_host(const moe_layer_desc_t* d, const moe_mb_bufs_t* b,
                                 const moe_bf16* host_x, const moe_bf16* host_dy,
                                 moe_bf16* host_y, moe_bf16* host_dx, void* stream) {
  MOE_CHECK(validate(d));
  MOE_CHECK(check_mb(*d, b, true));
  if (!host_x || !host_dy || !host_y || !host_dx) {
    set_error("host buffers must not be NULL");
    return MOE_ERR_INVALID_ARG;
  }
  const size_t bytes = (size_t)d->T * d->H * sizeof(moe_bf16);
  cudaStream_t st = S(stream);
  CopyLane* cl = copy_lane();
  if (!cl) return MOE_ERR_CUDA;
  // x goes in first on the compute stream. dy goes in on the copy stream while
  // the forward runs. y comes out on the copy stream while the backward runs.
  // dx comes out last.
  cudaError_t e = cudaEventRecord(cl->start, st);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(cl->stream, cl->start, 0);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(const_cast<moe_bf16*>(b->x), host_x, bytes, cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(const_cast<moe_bf16*>(b->dy), host_dy, bytes, cudaMemcpyHostToDevice,
                        cl->stream);
  if (e == cudaSuccess) e = cudaEventRecord(cl->dy_in, cl->stream);
  if (e != cudaSuccess) {
    set_error("host to device copy: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  MOE_CHECK(moe_layer_forward(d, b, stream));
  e = cudaEventRecord(cl->fwd_done, st);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(cl->stream, cl->fwd_done, 0);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(host_y, b->y, bytes, cudaMemcpyDeviceToHost, cl->stream);
  if (e == cudaSuccess) e = cudaEventRecord(cl->y_out, cl->stream);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(st, cl->dy_in, 0);
  if (e != cudaSuccess) {
    set_error("copy stream: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  // dx comes out on the copy stream as soon as the dispatch backward has
  // written it, while the weight gradients still run
  MOE_CHECK(layer_backward(d, b, 1, st, cl->dx_ready));
  e = cudaStreamWaitEvent(cl->stream, cl->dx_ready, 0);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(host_dx, b->dx, bytes, cudaMemcpyDeviceToHost, cl->stream);
  if (e == cudaSuccess) e = cudaEventRecord(cl->y_out, cl->stream);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(st, cl->y_out, 0);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) {
    set_error("device to host copy: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

moe_status_t moe_layer_steps_host(const moe_layer_desc_t* d, const moe_mb_bufs_t* b,
                                  int32_t n, const moe_bf16* const* host_x,
                                  const moe_bf16* const* host_dy, moe_bf16* const* host_y,
                                  moe_bf16* const* host_dx, void* stream) {
  MOE_CHECK(validate(d));
  if (!b) {
    set_error("buffer structs are NULL");
    return MOE_ERR_INVALID_ARG;
  }
  MOE_CHECK(check_mb(*d, &b[0], true));
  MOE_CHECK(check_mb(*d, &b[1], true));
  if (n < 0 || (n > 0 && (!host_x || !host_dy || !host_y || !host_dx))) {
    set_error("n must be >= 0 and the host pointer arrays given");
    return MOE_ERR_INVALID_ARG;
  }
  for (int i = 0; i < n; ++i) {
    if (!host_x[i] || !host_dy[i] || !host_y[i] || !host_dx[i]) {
      set_error("host buffer of step %d is NULL", i);
      return MOE_ERR_INVALID_ARG;
    }
  }
  if (b[0].x == b[1].x || b[0].dy == b[1].dy || b[0].y == b[1].y || b[0].dx == b[1].dx) {
    set_error("the two buffer sets need their own x, dy, y and dx");
    return MOE_ERR_INVALID_ARG;
  }
  if (n == 0) return MOE_OK;
  const size_t bytes = (size_t)d->T * d->H * sizeof(moe_bf16);
  cudaStream_t st = S(stream);
  CopyLane* cl = copy_lane();
  if (!cl) return MOE_ERR_CUDA;
  cudaError_t e = cudaSuccess;
  auto ok = [&](cudaError_t r) {
    if (e == cudaSuccess) e = r;
    return e == cudaSuccess;
  };
  // step i uses slot i % 2: its x, dy go in on the copy stream while step i-1
  // computes (after step i-2, the slot's last user, has finished reading
  // them), and its y, dx come out on the second copy stream while step i+1
  // computes; step i waits for its inputs and for step i-2's outputs to have
  // left the slot's y and dx. The outputs go out once the whole step is done:
  // an event recorded between two of the step's kernels (as soon as y, or dx,
  // is written) would stop the next kernel's launch from overlapping the
  // previous one's drain, and the copies overlap the next step anyway.
  auto upload = [&](int i) {
    const int s = i & 1;
    if (i >= 2) ok(cudaStreamWaitEvent(cl->stream, cl->step_done[s], 0));
    ok(cudaMemcpyAsync(const_cast<moe_bf16*>(b[s].x), host_x[i], bytes, cudaMemcpyHostToDevice,
                       cl->stream));
    ok(cudaMemcpyAsync(const_cast<moe_bf16*>(b[s].dy), host_dy[i], bytes,
                       cudaMemcpyHostToDevice, cl->stream));
    ok(cudaEventRecord(cl->in_ready[s], cl->stream));
  };
  ok(cudaEventRecord(cl->start, st));
  ok(cudaStreamWaitEvent(cl->stream, cl->start, 0));
  ok(cudaStreamWaitEvent(cl->d2h, cl->start, 0));
  upload(0);
  for (int i = 0; i < n && e == cudaSuccess; ++i) {
    const int s = i & 1;
    if (i + 1 < n) upload(i + 1);
    ok(cudaStreamWaitEvent(st, cl->in_ready[s], 0));
    if (i >= 2) ok(cudaStreamWaitEvent(st, cl->out_done[s], 0));
    if (e != cudaSuccess) break;
    MOE_CHECK(moe_layer_forward(d, &b[s], stream));
    MOE_CHECK(layer_backward(d, &b[s], 1, st, nullptr));
    ok(cudaEventRecord(cl->step_done[s], st));
    ok(cudaStreamWaitEvent(cl->d2h, cl->step_done[s], 0));
    ok(cudaMemcpyAsync(host_y[i], b[s].y, bytes, cudaMemcpyDeviceToHost, cl->d2h));
    ok(cudaMemcpyAsync(host_dx[i], b[s].dx, bytes, cudaMemcpyDeviceToHost, cl->d2h));
    ok(cudaEventRecord(cl->out_done[s], cl->d2h));
  }
  for (int s = 0; s < 2 && s < n; ++s) ok(cudaStreamWaitEvent(st, cl->out_done[s], 0));
  ok(cudaStreamSynchronize(st));
  if (e != cudaSuccess) {
    set_error("moe_layer_steps_host: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
