// Per-phase operations on one micro-batch's buffers, shared by the C ABI's
// whole-layer calls and the two-stream scheduler.
#pragma once

#include <mutex>

#include "moe_internal.cuh"

namespace moe {

moe_status_t validate(const moe_layer_desc_t* d);
// Per-device helper streams and events (the host-buffer step's copy stream,
// the backward's side stream), created on first use with that device current
// and kept until exit.
struct CopyLane {
  cudaStream_t stream = nullptr;
  cudaEvent_t start = nullptr, dy_in = nullptr, fwd_done = nullptr, y_out = nullptr;
  cudaEvent_t dx_ready = nullptr;
  // moe_layer_steps_host: a second copy stream (device to host) and, per
  // input slot, the events of its pipeline
  cudaStream_t d2h = nullptr;
  cudaEvent_t in_ready[2] = {}, step_done[2] = {}, out_done[2] = {};
  // moe_layer_backward's side stream: the weight gradients run on it beside
  // the dispatch backward (they depend on the dgrad only, not on each other)
  cudaStream_t side = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
  std::mutex side_mu;  // one fork/join enqueued at a time
};
// The current device's lane; NULL (with an error message) on failure.
CopyLane* copy_lane();
moe_status_t check_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, bool bwd);
// ints of the workspace's counter area (WsLayout::dep)
int dep_ints(const moe_layer_desc_t& d);

// route + dispatch layout + permute; max_ctas > 0 caps the fused launch's grid
moe_status_t op_dispatch(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, cudaStream_t st,
                         int max_ctas = 0);
moe_status_t op_ffn_fwd_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, int max_ctas,
                           cudaStream_t st);
moe_status_t op_combine_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, cudaStream_t st);
moe_status_t op_combine_bwd_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b,
                               cudaStream_t st);
moe_status_t op_dgrad_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, int max_ctas,
                         cudaStream_t st);
// permute backward + router backward
moe_status_t op_dispatch_bwd_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b,
                                cudaStream_t st);
moe_status_t op_wgrad_mb(const moe_layer_desc_t& d, const moe_mb_bufs_t* b, int max_ctas,
                         cudaStream_t st);

}  // namespace moe
