// The quantising passes of the 4-bit experts: the weights, and the permute (tokens sorted
// by expert into the send layout). Both are bound by HBM.
#include <algorithm>

#include "fp4_mma.cuh"

namespace moe {

namespace {

__device__ __forceinline__ uint32_t max8(uint32_t m, const uint4& v) {
  m = absmax_bf16x2(m, v.x);
  m = absmax_bf16x2(m, v.y);
  m = absmax_bf16x2(m, v.z);
  return absmax_bf16x2(m, v.w);
}
// eight bf16 times 1 / scale (two packed bf16) -> eight codes. The bf16 products are exact: a
// power of two moves exponents alone, and what falls below bf16's normal range is far
// below e2m1's smallest step.
__device__ __forceinline__ uint32_t codes(const uint4& v, uint32_t inv2) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w[j]) : "r"(inv2));
    f[2 * j] = bf16_lo(w[j]);
    f[2 * j + 1] = bf16_hi(w[j]);
  }
  return fp4x8(f);
}

// ------------------------------------------------------------------ weights
// A warp takes 256 columns of kRows consecutive rows, a lane 8 columns of each: four
// lanes share a block. After the maxima every lane of a block has all rows' bytes, and
// lane i of the block's four stores those of the rows i and i + 4, so that four rows' scales
// leave as one 32-byte sector. 128 experts of 2048 x 768, values kept: 2737 MB in 391 us, 7.0
// TB/s (more than a copy).
struct Fp4Mat {
  const bf16* w;
  uint8_t *q, *s;
  bf16* v;
  int R, C, groups;
  long long tasks;  // over all matrices
};
constexpr int kRows = 8;

// The values of the eight codes c of v's elements as bf16, exact: two significant bits, and
// the smallest one is 2^-128, on bf16's grid of 2^-133 there. Byte tables give the two
// halves of each magnitude's bf16 pattern, four codes at a time; the signs are the elements'.
// (Twelve instructions for four values; with the arithmetic spelled out the kernel was bound
// by issuing it: 527 us for the 128-expert layer's weights.)
__device__ __forceinline__ uint4 values(const uint4& v, uint32_t c, uint32_t scale2) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t sel = (c >> (16 * j)) & 0x7777u;
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);  // 0 .5 1 1.5 | 2 3 4 6
    const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel);
    w[2 * j] = __byte_perm(lo, hi, 0x5140u);
    w[2 * j + 1] = __byte_perm(lo, hi, 0x7362u);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w[j]) : "r"(scale2));
    w[j] |= x[j] & 0x80008000u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(256) quantize_weights_fp4_kernel(const Fp4Mat m1, const Fp4Mat m2) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const bool first = task < m1.tasks;
  const Fp4Mat& m = first ? m1 : m2;
  if (!first) task -= m1.tasks;
  if (task >= m.tasks) return;  // (a whole warp)
  const int g = (int)(task % m.groups);
  const long long rest = task / m.groups;
  const int r0 = (int)(rest % (m.R / kRows)) * kRows;
  const long long mat = rest / (m.R / kRows);
  const int col = g * kFp4Group + lane * 8;
  const bool ok = col < m.C;  // C is a multiple of 64: a block is in or out whole
  const size_t at = ((size_t)mat * m.R + r0) * m.C + col;
  uint4 v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    v[i] = ok ? __ldcs(reinterpret_cast<const uint4*>(m.w + at + (size_t)i * m.C)) : make_uint4(0, 0, 0, 0);
  uint32_t mine[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    uint32_t mx = absmax_bits(max8(0, v[i]));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const uint32_t b = fp4_scale_byte(mx);
    if ((lane & 3) == (i & 3)) mine[i >> 2] = b;
    if (!ok) continue;
    const uint32_t c = codes(v[i], fp8_inv_scale2(b));
    const size_t e = at + (size_t)i * m.C;
    *reinterpret_cast<uint32_t*>(m.q + e / 2) = c;
    if (m.v) {
      // b = 255: NaN; byte 0 is 2^-127, a subnormal
      const uint32_t scale2 = b == 255u ? 0x7FFF7FFFu : b ? b * 0x00800080u : 0x00400040u;
      __stcs(reinterpret_cast<uint4*>(m.v + e), values(v[i], c, scale2));
    }
  }
  uint8_t* s = m.s + (((size_t)mat * m.groups + g) * m.R + r0 + (lane & 3)) * 8 + (lane >> 2);
  s[0] = (uint8_t)mine[0];
  s[32] = (uint8_t)mine[1];
}

// ------------------------------------------------------------------ permute
// Row slot[t,j] of (xq, xs) = quantised x[t], for every j. A warp takes one token's 1024
// columns, a lane the 32 of a block: x is read and rounded once and written to the token's k
// rows, 16 bytes a lane. Lane j holds the token's j-th slot. 4096 tokens of 2048, 8 rows each:
// 52 MB in 8.5 us, 6.1 TB/s (16 columns a lane 9.4, plain stores 10.2).
__global__ void __launch_bounds__(256) permute_fp4_kernel(const bf16* __restrict__ x,
                                                          const int32_t* __restrict__ slot,
                                                          uint8_t* __restrict__ xq,
                                                          uint8_t* __restrict__ xs, int T, int H,
                                                          int k, long long N, int nseg, int* dep,
                                                          int ndep, int* tile) {
  pdl_wait();
  if (dep && blockIdx.x == 0) {
    if ((int)threadIdx.x < ndep) dep[threadIdx.x] = 0;
    if (threadIdx.x == 0) *tile = 0;
  }
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
  const long long tasks = (long long)T * nseg, np = fp4::scale_rows(N);
  for (long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < tasks;
       w += warps) {
    const int t = (int)(w / nseg), seg = (int)(w % nseg);
    const int col = seg * 1024 + lane * 32;
    const bool ok = col < H;
    const uint4* src = reinterpret_cast<const uint4*>(x + (size_t)t * H + col);
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ok ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
    int sl = lane < k ? slot[(size_t)t * k + lane] : -1;
    if (sl >= N) sl = -1;
    const uint32_t b = fp4_scale_byte(absmax_bits(max8(max8(max8(max8(0, v[0]), v[1]), v[2]), v[3])));
    const uint32_t inv = fp8_inv_scale2(b);
    const uint4 q = make_uint4(codes(v[0], inv), codes(v[1], inv), codes(v[2], inv), codes(v[3], inv));
    // the eight bytes of 256 columns
    uint32_t word = b << (8 * (lane & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 4);
    const uint2 scales = make_uint2(word, other);  // in the first lane of a group's eight
    const int g = seg * 4 + (lane >> 3);
    const bool holds = (lane & 7) == 0 && g * kFp4Group < H;
    for (int j = 0; j < k; ++j) {
      const int s = __shfl_sync(0xffffffffu, sl, j);
      if (s < 0) continue;
      if (ok) __stcs(reinterpret_cast<uint4*>(xq + ((size_t)s * H + col) / 2), q);
      if (holds) *reinterpret_cast<uint2*>(xs + ((size_t)g * np + s) * 8) = scales;
    }
  }
}

moe_status_t launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) {
    set_error("%s launch: %s", what, cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return check_launch(what);
}

}  // namespace

moe_status_t launch_fp4_quantize_weights(const moe_layer_desc_t& d, const bf16* w1, const bf16* w2,
                                         uint8_t* w1q, uint8_t* w1s, uint8_t* w2q, uint8_t* w2s,
                                         bf16* w1v, bf16* w2v, cudaStream_t st) {
  const int gh = fp4_groups(d.H), gf = fp4_groups(d.F);
  const Fp4Mat m1 = {w1, w1q, w1s, w1v, d.F, d.H, gh, 2ll * d.E * (d.F / kRows) * gh};
  const Fp4Mat m2 = {w2, w2q, w2s, w2v, d.H, d.F, gf, (long long)d.E * (d.H / kRows) * gf};
  cudaError_t e;
  {
    LaunchScope _ls(K_FP4_QUANT_W, st);
    e = launch_k(quantize_weights_fp4_kernel, dim3((unsigned)((m1.tasks + m2.tasks + 7) / 8)), 256, 0,
                 st, m1, m2);
  }
  return launched(e, "quantize_weights_fp4_kernel");
}

moe_status_t launch_permute_fp4(const moe_layer_desc_t& d, const bf16* x, const int32_t* slot,
                                uint8_t* xq, uint8_t* xs, cudaStream_t st, int* dep, int* status) {
  const long long N = (long long)d.T * d.k;
  if (N == 0) return MOE_OK;
  const int nseg = ceil_div(d.H, 1024);
  const long long blocks = ((long long)d.T * nseg + 7) / 8;
  const int grid = (int)std::min<long long>(blocks, (long long)device_sm_count() * 16);
  cudaError_t e;
  {
    LaunchScope _ls(K_FP4_PERMUTE, st);
    e = launch_k(permute_fp4_kernel, grid, 256, 0, st, x, slot, xq, xs, d.T, d.H, d.k, N, nseg, dep,
                 dep ? d.E : 0, dep ? fp8::tile_counter(status) : nullptr);
  }
  return launched(e, "permute_fp4_kernel");
}

}  // namespace moe
