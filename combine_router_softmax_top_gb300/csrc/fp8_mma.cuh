// Device and host helpers shared by the 8-bit expert kernels (grouped_gemm_fp8.cu,
// rows_fp8.cu): block-scaled tcgen05, scale cells in TMEM, SwiGLU arithmetic, TMA maps.
#pragma once

#include <mutex>

#include "fp8.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace fp8 {

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s without progress -> give up

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}

// s(x) = 1 / (1 + e^-x) = 1 / (1 + 2^(-x log2 e)). Rounding log2 e and the product to
// fp32 makes e^-x off by up to 7.4e-8 |x| of its value, on top of the two instructions'
// few 2^-23: a relative error of some 5e-7 for |x| < 2 and up to 7e-6 near x = -87, where s leaves the normal numbers and is taken as 0 (rounding s to
// bf16 is 2^-8). The flushing
// forms of the two approximate instructions need no scaling around them, which
// is a third of the instructions of a SwiGLU element.
__device__ __forceinline__ float sigmoid_f(float x) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

// ---------------------------------------------------------------- tcgen05, block-scaled
// kind::mxf8f6f4 instruction descriptor: e4m3 operands (format 0), UE8M0 scales
// (bit 23), fp32 D; bits 4-5 and 29-30 select the byte of the scale cells.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N, int b_mn) {
  return ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A B^T with the scales of their rows' 32-value groups, one CTA.
__device__ __forceinline__ void umma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X "
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// This warp's 32 lanes x 4 TMEM columns
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, const uint32_t (&w)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 lanes x 8 columns: thread i receives lane i's
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait_x8(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// As ptx::mbar_wait, acquiring what another CTA of the cluster released.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity,
                                                  volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(ptx::smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 63) == 0) {
      if (t0 == 0) t0 = ptx::globaltimer_ns();
      if (*abort || ptx::globaltimer_ns() - t0 > kWaitLimitNs) return false;
    }
  }
}

// After an abort: waits (bounded) until the loads that a producer has issued have
// landed, so that none writes into shared memory that is no longer this
// kernel's. stage, phase: the producer's place in the ring.
__device__ __forceinline__ void drain_loads(uint64_t* full, int stages, int stage,
                                            uint32_t phase) {
  int none = 0;
  for (int s = 0; s < stages; ++s)
    ptx::mbar_wait(&full[s], s < stage ? phase : phase ^ 1, &none, kWaitLimitNs / stages);
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// Load map of e4m3 bytes, up to three dimensions (innermost first), boxes of
// 128 bytes x box1 x box2, 128-byte swizzle; what lies outside reads as zero.
inline bool make_map(CUtensorMap* m, const void* base, int dims, long long d0, long long d1, long long d2,
              int box1, int box2) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return false;
  }
  cuuint64_t dim[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
  cuuint64_t strides[2] = {(cuuint64_t)d0, (cuuint64_t)(d0 * d1)};
  cuuint32_t box[3] = {128, (cuuint32_t)box1, (cuuint32_t)box2};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = encode_map(enc, m, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, const_cast<void*>(base), dim, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for a %lld x %lld x %lld map", (int)r, d2, d1,
              d0);
    return false;
  }
  return true;
}

// Map of bf16 (or, in boxes of 64 columns, e4m3) rows [rows, cols] in boxes of 64
// bytes x box_rows, 64-byte swizzle.
inline bool make_rows_map(CUtensorMap* m, const void* base, long long rows, long long cols,
                          int box_rows, bool fp8 = false) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return false;
  }
  cuuint64_t dim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)cols * (fp8 ? 1 : 2)};
  cuuint32_t box[2] = {fp8 ? 64u : 32u, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  CUresult r = encode_map(enc, m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dim, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for a %lld x %lld map", (int)r, rows, cols);
    return false;
  }
  return true;
}

// Clears n <= 256 counters and the tile counter on the stream.
cudaError_t launch_zero_counters(int* dep, int n, int* tile, cudaStream_t st);
// The tile counter of a workspace: a word after the status words, in their area.
inline int* tile_counter(int* status) { return status + 2 * ST_NUM; }

}  // namespace fp8
}  // namespace moe
