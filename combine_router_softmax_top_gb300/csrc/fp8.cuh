// 8-bit floating-point experts: declarations shared by their translation units
// and the block-scale arithmetic of every kernel that quantises.
//
// A block of values (128 consecutive columns of an activation row, or a
// 128 x 128 block of a weight matrix) shares one power-of-two scale 2^(b-127),
// held as the byte b (UE8M0). A value is held as q = e4m3(value / scale).
// b is the smallest one that brings the block's largest magnitude to 448 (the
// largest e4m3 value) or below, so no value is ever clamped, and as dividing by
// a power of two is exact, e4m3 is the only rounding. Power-of-two scales are
// what the tensor cores apply themselves (tcgen05 kind::mxf8f6f4), and they
// cost no precision: e4m3 is a floating-point format, its relative step does
// not depend on where in its range the block's maximum lies.
#pragma once

#include <cuda_fp8.h>

#include "moe_internal.cuh"

namespace moe {

constexpr int kFp8Block = 128;  // values (or rows and columns) that share a scale

enum Fp8KernelId {  // kernel ids past those of the bf16 layer
  K_FP8_QUANT_W = K_NUM, K_FP8_PERMUTE, K_FP8_COMBINE_BWD, K_FP8_FFN_FWD, K_FP8_FFN_DGRAD,
  K_FP8_ZERO, K_FP8_ROWS_FFN, K_ALL
};

// ---------------------------------------------------------------- block scales
// Scale byte of a block whose largest magnitude has the given fp32 bits:
// 127 + ceil(log2(amax / 448)), at least 0. With amax = m 2^E (1 <= m < 2) and
// 448 = 1.75 * 2^8 that is E - 8 when m <= 1.75 and E - 7 above, so adding
// 0x1FFFFF to the mantissa (1.75 has mantissa bits 0x600000) carries exactly
// then. 255 (NaN) for a block with a NaN or an infinity.
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const uint32_t e = (amax_bits + 0x1FFFFFu) >> 23;
  return e > 8u ? e - 8u : 0u;
}
__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// 1 / scale as two packed bf16, exact for b <= 247 (no finite block needs more):
// 2^(127 - b) has an exponent field of 254 - b >= 7. NaN for b = 255, which turns
// every value of the block into e4m3's NaN.
__device__ __forceinline__ uint32_t fp8_inv_scale2(uint32_t b) {
  return b == 255u ? 0x7FFF7FFFu : (254u - b) * 0x00800080u;
}
// Four bf16 (two words) scaled by inv2 -> four e4m3. The bf16 products are exact:
// a power of two moves exponents alone, and what falls below bf16's normal range
// is far below e4m3's smallest step.
__device__ __forceinline__ uint32_t fp8x4_of_bf16(uint32_t w0, uint32_t w1, uint32_t inv2) {
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w0) : "r"(inv2));
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w1) : "r"(inv2));
  return fp8x4(bf16_lo(w0), bf16_hi(w0), bf16_lo(w1), bf16_hi(w1));
}
// Larger magnitude in each half of two packed pairs of bf16 (its sign bit is
// arbitrary); NaN if either is.
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t m, uint32_t w) {
  asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w));
  return m;
}
// fp32 bits of the larger half of a packed maximum: without signs, bf16 patterns
// order like unsigned integers, NaN on top
__device__ __forceinline__ uint32_t absmax_bits(uint32_t m) {
  const uint32_t lo = (m << 16) & 0x7FFF0000u, hi = m & 0x7FFF0000u;
  return lo > hi ? lo : hi;
}

inline int fp8_blocks(int n) { return ceil_div(n, kFp8Block); }

// ---------------------------------------------------------------- launchers
moe_status_t launch_fp8_quantize_weights(const moe_layer_desc_t& d, const bf16* w1, const bf16* w2,
                                         uint8_t* w1q, uint8_t* w1s, uint8_t* w2q, uint8_t* w2s,
                                         cudaStream_t st);
moe_status_t launch_permute_fp8(const moe_layer_desc_t& d, const bf16* x, const int32_t* slot,
                                uint8_t* xq, uint8_t* xs, cudaStream_t st);
// zero/nzero: as for launch_combine_bwd
moe_status_t launch_combine_bwd_fp8(const moe_layer_desc_t& d, const bf16* dy, const bf16* o,
                                    const int32_t* slot, const float* gates, bf16* d_o,
                                    uint8_t* dq, uint8_t* ds, float* dgates, cudaStream_t st,
                                    int* zero = nullptr, int nzero = 0);

struct Fp8Weights {
  const uint8_t *w1q, *w1s, *w2q, *w2s;
};
// Expert FFN forward: a and h (bf16) are written when given.
moe_status_t launch_ffn_fwd_fp8(const moe_layer_desc_t& d, const uint8_t* xq, const uint8_t* xs,
                                const int32_t* off, const Fp8Weights& w, bf16* a, bf16* h,
                                uint8_t* hq, uint8_t* hs, bf16* o, int* status, int* dep,
                                cudaStream_t st);
// The forward for few rows an expert (rows_fp8.cu), which launch_ffn_fwd_fp8 takes
// up to kFp8FewRows rows an expert on average. Measured, this kernel against the
// GEMM chain, us, nothing kept (a and h kept: 1 to 8 us more on both sides):
//   rows an expert on average            4         16        32        48        64
//   128 experts, H 2048, F 768     92 / 127  95 / 133 100 / 141 124 / 151 123 / 158
//     skewed                       88 / 121  97 / 133 104 / 138 122 / 144 147 / 150
//     all on 8 of the experts       20 / 29   36 / 25   61 / 32   86 / 36  111 / 42
//   64 experts, H 2048, F 1408     86 / 106  89 / 110  91 / 120 108 / 128 100 / 137
//   16 experts, H 1024, F 1024      15 / 26   18 / 23   18 / 24   27 / 25   27 / 26
//   8 experts, H 4096, F 1408       33 / 41   34 / 41   37 / 43   51 / 45   40 / 49
//   32 experts, H 512, F 512        12 / 22   14 / 22   16 / 22   24 / 23   25 / 23
// Where the weights come from HBM it is ahead past 48 rows, balanced or skewed; out of
// L2 the two meet between 32 and 48. What it loses is routing that leaves most experts
// without rows: the rule sees the average alone, as the offsets are on the device.
constexpr long long kFp8FewRows = 48;
moe_status_t launch_ffn_rows_fp8(const moe_layer_desc_t& d, const uint8_t* xq, const uint8_t* xs,
                                 const int32_t* off, const Fp8Weights& w, bf16* a, bf16* h,
                                 uint8_t* hq, uint8_t* hs, bf16* o, int* status, int* dep,
                                 cudaStream_t st);
// Expert FFN activation gradient: da (bf16) is written when given.
moe_status_t launch_ffn_dgrad_fp8(const moe_layer_desc_t& d, const uint8_t* dq, const uint8_t* ds,
                                  const bf16* a, const int32_t* off, const Fp8Weights& w, bf16* da,
                                  uint8_t* daq, uint8_t* das, bf16* dx_perm, int* status, int* dep,
                                  cudaStream_t st);

}  // namespace moe
