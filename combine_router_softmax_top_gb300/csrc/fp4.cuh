// Microscaled 4-bit experts: declarations shared by their translation units and the
// block-scale arithmetic of every kernel that quantises.
//
// 32 consecutive values along K (columns of a row, of an activation or of a weight
// matrix) share one power-of-two scale 2^(b-127), held as the byte b (UE8M0). A value is
// held as q = e2m1(value / scale): 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, two
// of them a byte, the lower column in the low bits. b is the smallest one that brings
// the block's largest magnitude to 6 or below: nothing is clamped and dividing is exact,
// so e2m1's rounding (to nearest, ties to even) is the only one. The tensor cores take
// the bytes and the scales as they lie (tcgen05 kind::mxf4).
//
// Scale bytes of rows [R, C] lie as [ceil(C / 256)][R][8]: the eight blocks of 256 columns
// (128 bytes of values, one operand stage) side by side, rows of a stage consecutive, so
// that a stage's scales are one contiguous copy. Activations have R rounded up to even:
// a copy starts on an even row, which is a 16-byte boundary.
#pragma once

#include "fp8.cuh"

namespace moe {

constexpr int kFp4Block = 32, kFp4Group = 256;

inline int fp4_groups(int n) { return ceil_div(n, kFp4Group); }

// Scale byte of a block whose largest magnitude has the given fp32 bits: 127 +
// ceil(log2(amax / 6)), at least 0. 6 = 1.5 * 2^2, so that is the exponent field less 2
// when the mantissa is 1.5 or below, and less 1 above: adding 0x3FFFFF carries exactly
// then. 255 (NaN) for a block with a NaN or an infinity.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const uint32_t e = (amax_bits + 0x3FFFFFu) >> 23;
  return e > 2u ? e - 2u : 0u;
}
// 1 / scale: exact (b is 253 at most, but for a block that is not finite: NaN)
__device__ __forceinline__ float fp4_inv_scale(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7FFFFFFFu : (254u - b) << 23);
}
// Eight values, already divided by their scale -> eight e2m1 codes, v[0] in the low bits.
__device__ __forceinline__ uint32_t fp4x8(const float* v) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}
// Larger magnitude; NaN if either is
__device__ __forceinline__ float absmax_nan(float m, float v) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v)));
  return m;
}

// ---------------------------------------------------------------- launchers
struct Fp4Weights {
  const uint8_t *w1q, *w1s, *w2q, *w2s;
};
// w1v, w2v (may be NULL): the values that the codes stand for
moe_status_t launch_fp4_quantize_weights(const moe_layer_desc_t& d, const bf16* w1, const bf16* w2,
                                         uint8_t* w1q, uint8_t* w1s, uint8_t* w2q, uint8_t* w2s,
                                         bf16* w1v, bf16* w2v, cudaStream_t st);
// dep, status: counters of the expert products that follow on the stream, which the launch
// clears for them (the layer path: one launch less).
moe_status_t launch_permute_fp4(const moe_layer_desc_t& d, const bf16* x, const int32_t* slot,
                                uint8_t* xq, uint8_t* xs, cudaStream_t st, int* dep = nullptr,
                                int* status = nullptr);
// Expert FFN forward: a and h (bf16) are written when given. counters_zeroed: the launch
// before it on the stream has cleared its counters.
moe_status_t launch_ffn_fwd_fp4(const moe_layer_desc_t& d, const uint8_t* xq, const uint8_t* xs,
                                const int32_t* off, const Fp4Weights& w, bf16* a, bf16* h,
                                uint8_t* hq, uint8_t* hs, bf16* o, int* status, int* dep,
                                cudaStream_t st, bool counters_zeroed = false);
// The forward for few rows an expert (rows_fp4.cu), which launch_ffn_fwd_fp4 takes up to
// kFp4FewRows rows an expert on average. Measured, this kernel against the GEMMs, us,
// nothing kept:
//   rows an expert on average            4         16        32        64        96
//   128 experts, H 2048, F 768      54 / 92   57 / 93   59 / 96  83 / 106  119 / 95
//     skewed                        51 / 86   60 / 93   69 / 97 106 / 105 139 / 111
//   64 experts, H 2048, F 1408      50 / 71   52 / 73   53 / 77   71 / 88  102 / 74
//   16 experts, H 1024, F 1024      12 / 20   14 / 20   14 / 21   20 / 22   20 / 21
//   8 experts, H 4096, F 1408       22 / 28   23 / 28   24 / 30   27 / 33   33 / 29
//   32 experts, H 512, F 512        11 / 19   11 / 19   12 / 19   17 / 19   18 / 20
//   16 experts, H 320, F 448, skewed 10 / 14  11 / 14   11 / 15   13 / 15   15 / 15
// The rule sees the average alone, as the offsets are on the device. With all rows in a few experts
// (`hot`, evenly) the few-rows kernel walks each 32 rows at a time; against the GEMMs on the same
// rows (given as a layer of few enough experts), us:
//   rows an expert on average            4         16        32        64
//   128 experts, H 2048, F 768, 4 hot   18 / 17   27 / 19   42 / 25   75 / 34
//                               16 hot            27 / 27   44 / 26   80 / 35
//   64 experts, H 2048, F 1408, 4 hot             25 / 20   38 / 25   66 / 32
//   16 experts, H 1024, F 1024, 4 hot                       13 / 16   19 / 16
constexpr long long kFp4FewRows = 64;
moe_status_t launch_ffn_rows_fp4(const moe_layer_desc_t& d, const uint8_t* xq, const uint8_t* xs,
                                 const int32_t* off, const Fp4Weights& w, bf16* a, bf16* h,
                                 uint8_t* hq, uint8_t* hs, bf16* o, int* status, int* dep,
                                 cudaStream_t st, bool counters_zeroed);

}  // namespace moe
