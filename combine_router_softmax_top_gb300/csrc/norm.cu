// The norm in front of the layer: the residual's addition and root-mean-square
// norm, its rows in bf16 and, when asked for, as e4m3 with block scales; and its
// gradient. Everything is bound by HBM, or by latency for a few rows.
//
//   r = bf16(x + res),  rstd = (mean(r^2) + eps)^-1/2,  y = bf16(r rstd w)
//   xh = r rstd,  g = dy w
//   dx = bf16(rstd (g - xh mean(g xh)) + dr),  dw = sum over rows of dy xh
//
// A row lives in the registers of its threads between the pass that sums the
// squares and the one that scales, so it is read once. Sums are fp32: a thread's
// columns in order, then the threads in a fixed tree, so results do not change
// from call to call.
//
// Rows of 2048: 4096 with their sum 67 MB in 11.8 us (a library copy of as many bytes takes 14.2:
// at this size launch and ramps count), 32768 with 8-bit rows 604 MB in 88 us, 6.9 TB/s, a
// copy's rate; one row 3.0 us, the call itself. Gradient of 4096 rows: 67 MB in 13.9 us, and 2.7
// us for dw's sum over blocks, which reads their 456 partial rows in a fixed order. (Each
// thread's columns of the next rows on their way into shared memory by cp.async, 5 rows in three
// blocks of 128 threads, to 8 in two: 20 to 25 us against 17.2; too few warps for a row's chain of
// latencies.)
#include <algorithm>
#include <float.h>
#include <math.h>

#include "api_checks.cuh"
#include "fp8.cuh"
#include "moe_layer_ops.h"

namespace moe {

namespace {

// Threads of a row: a power of two, each with up to `vecs` groups of 8 columns, and at
// least the 16 that hold a block of 128.
int row_threads(int H, int vecs) {
  int tpr = H > 64 ? 16 : 8;
  while (tpr * vecs * 8 < H) tpr <<= 1;
  return tpr;
}

// Sum over the threads of a row; s_part: a word for each warp of the block. Rows of
// more than a warp meet at a barrier, of the whole block (all its rows do) or, with OWN, of the
// row alone: a block's rows then drift apart, and one's loads run beside another's arithmetic
// (norm_grad_layer 17.2 -> 16.6 us), but a block takes all sixteen of its barriers, which leaves an
// SM four blocks. Two calls in a row need different s_part.
template <bool OWN>
__device__ __forceinline__ float row_sum(float v, int tpr, float* s_part) {
  const int width = tpr < 32 ? tpr : 32;
#pragma unroll
  for (int o = 16; o; o >>= 1)
    if (o < width) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tpr <= 32) return v;
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  if (OWN) asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / tpr), "r"(tpr) : "memory");
  else __syncthreads();
  const int first = threadIdx.x / tpr * (tpr / 32);
  v = s_part[first];
  for (int w = 1; w < tpr / 32; ++w) v += s_part[first + w];
  return v;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint4 add8(const uint4& x, const uint4& y) {
  auto add = [](uint32_t a, uint32_t b) { return pack2(bf16_lo(a) + bf16_lo(b), bf16_hi(a) + bf16_hi(b)); };
  return make_uint4(add(x.x, y.x), add(x.y, y.y), add(x.z, y.z), add(x.w, y.w));
}

struct NormParams {
  const bf16 *x, *res, *w;
  float eps;
  bf16 *r, *y;
  uint8_t* yq;
  uint32_t* ys;
  float* rstd;
  int T, H, tpr;
  float low, high;  // a row whose sum of squares is outside of these is looked at again (redo_row)
};

// ---- rows whose squares leave fp32's range: from 2^64 on, or below 2^-50 beside an eps that small
// All threads of such a row (and of its warp) go through the following, once the kernel has done
// the rest. A barrier of the row's threads: the block, one of its two halves, a warp.
__device__ __forceinline__ void row_sync(int tpr) {
  if (tpr <= 32) __syncwarp();
  else if (tpr >= 128) __syncthreads();
  else if (threadIdx.x < 64) asm volatile("bar.sync 1, 64;" ::: "memory");
  else asm volatile("bar.sync 2, 64;" ::: "memory");
}
template <class T, class Op>
__device__ __forceinline__ T row_reduce(T v, int tpr, float* s_part, Op op) {
  const int width = tpr < 32 ? tpr : 32;
  for (int o = 16; o; o >>= 1)
    if (o < width) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (tpr <= 32) return v;
  T* part = reinterpret_cast<T*>(s_part);
  row_sync(tpr);  // the last result has been read
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  row_sync(tpr);
  const int first = threadIdx.x / tpr * (tpr / 32);
  v = part[first];
  for (int w = 1; w < tpr / 32; ++w) v = op(v, part[first + w]);
  return v;
}
// The row is summed again under a power of two, 2^-k with 2^k its largest magnitude or eps' root, and
// its outputs are written again, as the kernel writes them. It reads its input again, in a
// function of its own: what it needs of a thread's registers would otherwise be taken from
// ordinary rows (64 a thread for 48, norm_prompts 88 -> 94 us; with the kernel's own loop
// shared between the two 89.4). In the same warp, rows that are in range and those with an
// infinity keep their rstd, and their outputs' bits.
__device__ __noinline__ void redo_row(const NormParams& p, int t, int sub, float ms, float* s_part,
                                      uint32_t* words) {
  // (the sum where it was kept: it may have taken x's or res' place)
  const bf16 *x = p.r ? p.r : p.x, *res = p.r ? nullptr : p.res;
  const size_t at = (size_t)t * p.H;
  const int cpr = p.H / 8;
  auto row = [&](int c) {
    if (t >= p.T || c >= cpr) return make_uint4(0, 0, 0, 0);
    const uint4 v = reinterpret_cast<const uint4*>(x + at)[c];
    return res ? add8(v, reinterpret_cast<const uint4*>(res + at)[c]) : v;
  };
  auto larger = [](uint32_t a, uint32_t b) { return max(a, b); };
  row_sync(p.tpr);  // s_part and words have been read
  uint32_t m = 0;
#pragma unroll 1
  for (int c = sub; c < cpr; c += p.tpr) {
    const uint4 v = row(c);
    m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(m, v.x), v.y), v.z), v.w);
  }
  m = row_reduce(absmax_bits(m), p.tpr, s_part, larger);
  const uint32_t e = max(m, __float_as_uint(sqrtf(p.eps))) >> 23;
  const float down = __uint_as_float((254u - min(max(e, 1u), 253u)) << 23);
  float ss = 0.f;
#pragma unroll 1
  for (int c = sub; c < cpr; c += p.tpr) {
    const uint4 v = row(c);
    const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = bf16_lo(a[j]) * down, hi = bf16_hi(a[j]) * down;
      ss = fmaf(hi, hi, fmaf(lo, lo, ss));
    }
  }
  ss = row_reduce(ss, p.tpr, s_part, [](float a, float b) { return a + b; });
  float rs = 1.f / sqrtf(ms);
  if ((ms < 0x1p-100f || ms > FLT_MAX) && m < 0x7F800000u)
    rs = 1.f / sqrtf(ss / (float)p.H + p.eps * down * down) * down;
  if (p.rstd && sub == 0 && t < p.T) p.rstd[t] = rs;
#pragma unroll 1
  for (int c = sub; c - sub < cpr; c += p.tpr) {
    const bool ok = t < p.T && c < cpr;
    uint4 v = row(c);
    const uint4 w = ok ? __ldg(reinterpret_cast<const uint4*>(p.w) + c) : make_uint4(0, 0, 0, 0);
    uint32_t* a = reinterpret_cast<uint32_t*>(&v);
    const uint32_t* wp = reinterpret_cast<const uint32_t*>(&w);
    uint32_t mx = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = pack2(bf16_lo(a[j]) * rs * bf16_lo(wp[j]), bf16_hi(a[j]) * rs * bf16_hi(wp[j]));
      mx = absmax_bf16x2(mx, a[j]);
    }
    if (ok && p.y) reinterpret_cast<uint4*>(p.y + at)[c] = v;
    if (!p.yq) continue;
    mx = c < cpr ? absmax_bits(mx) : 0;
    for (int o = 1; o < 16; o <<= 1)
      if (o < p.tpr) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const uint32_t b = fp8_scale_byte(mx), inv = fp8_inv_scale2(b);
    if (ok)
      reinterpret_cast<uint2*>(p.yq + at)[c] =
          make_uint2(fp8x4_of_bf16(a[0], a[1], inv), fp8x4_of_bf16(a[2], a[3], inv));
    if ((c & 15) == 0 && c < cpr) reinterpret_cast<uint8_t*>(words)[c >> 4] = (uint8_t)b;
  }
  if (p.yq) {
    row_sync(p.tpr);
    for (int i = sub; i < (p.H + 511) / 512; i += p.tpr)
      if (t < p.T) p.ys[(size_t)i * p.T + t] = words[i];
  }
}

// THREADS: of a block at most. REGS a thread: 1024 of 48, or two blocks of 512 of 64, on an SM
template <int V, int THREADS, int REGS>
__global__ void __maxnreg__(REGS) rms_norm_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ uint32_t s_words[];  // scale words of the block's rows
  __shared__ float s_part[THREADS / 32];
  const int rows = blockDim.x / p.tpr, lr = threadIdx.x / p.tpr, sub = threadIdx.x % p.tpr;
  const int cpr = p.H / 8, nw = (p.H + 511) / 512;
  if (p.yq)  // bytes past a row's blocks stay 0
    for (int i = threadIdx.x; i < rows * nw; i += blockDim.x) s_words[i] = 0;
  pdl_wait();
  if (p.yq) __syncthreads();
  const int t = blockIdx.x * rows + lr;
  const size_t at = (size_t)t * p.H;
  uint4 v[V], q[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = sub + i * p.tpr;
    const bool ok = t < p.T && c < cpr;
    v[i] = ok ? reinterpret_cast<const uint4*>(p.x + at)[c] : make_uint4(0, 0, 0, 0);
    if (p.res)
      q[i] = ok ? reinterpret_cast<const uint4*>(p.res + at)[c] : make_uint4(0, 0, 0, 0);
  }
  uint4 wv[V];  // (on its way beside the row)
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = sub + i * p.tpr;
    wv[i] = c < cpr ? __ldg(reinterpret_cast<const uint4*>(p.w) + c) : make_uint4(0, 0, 0, 0);
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    uint32_t* a = reinterpret_cast<uint32_t*>(&v[i]);
    if (p.res) {
      const uint32_t* b = reinterpret_cast<const uint32_t*>(&q[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[j] = pack2(bf16_lo(a[j]) + bf16_lo(b[j]), bf16_hi(a[j]) + bf16_hi(b[j]));
      const int c = sub + i * p.tpr;
      if (p.r && t < p.T && c < cpr) __stcs(reinterpret_cast<uint4*>(p.r + at) + c, v[i]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ss = fmaf(bf16_lo(a[j]), bf16_lo(a[j]), ss);
      ss = fmaf(bf16_hi(a[j]), bf16_hi(a[j]), ss);
    }
  }
  ss = row_sum<false>(ss, p.tpr, s_part);
  const float ms = ss / (float)p.H + p.eps, rs = 1.f / sqrtf(ms);
  if (p.rstd && sub == 0 && t < p.T) p.rstd[t] = rs;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = sub + i * p.tpr;
    const bool ok = t < p.T && c < cpr;
    const uint32_t* wp = reinterpret_cast<const uint32_t*>(&wv[i]);
    uint32_t* a = reinterpret_cast<uint32_t*>(&v[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      a[j] = pack2(bf16_lo(a[j]) * rs * bf16_lo(wp[j]), bf16_hi(a[j]) * rs * bf16_hi(wp[j]));
    if (ok && p.y) __stcs(reinterpret_cast<uint4*>(p.y + at) + c, v[i]);
    if (!p.yq) continue;
    // a block is 16 threads' columns (8 threads' in a row of 64)
    uint32_t m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(0, a[0]), a[1]), a[2]), a[3]);
    m = c < cpr ? absmax_bits(m) : 0;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1)
      if (o < p.tpr) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t b = fp8_scale_byte(m), inv = fp8_inv_scale2(b);
    if (ok)
      reinterpret_cast<uint2*>(p.yq + at)[c] =
          make_uint2(fp8x4_of_bf16(a[0], a[1], inv), fp8x4_of_bf16(a[2], a[3], inv));
    if ((c & 15) == 0 && c < cpr)
      reinterpret_cast<uint8_t*>(s_words)[lr * 4 * nw + (c >> 4)] = (uint8_t)b;
  }
  if (p.yq) {  // whole words: their bytes come from several threads
    if (p.tpr <= 32) __syncwarp();
    else __syncthreads();
    for (int i = sub; i < nw; i += p.tpr)
      if (t < p.T) p.ys[(size_t)i * p.T + t] = s_words[lr * nw + i];
  }
  bool again = ss < p.low || ss > p.high;  // (not for a NaN)
  if (p.tpr <= 32) again = __any_sync(0xffffffffu, again);
  if (again) redo_row(p, t, sub, ms, s_part, s_words + lr * nw);
}

struct NormBwdParams {
  const bf16 *dy, *dr, *r, *w;
  const float* rstd;
  bf16* dx;
  float* part;  // [blocks][H]
  int T, H, tpr;
};

// BLOCKS resident on an SM, each with a row's partial sums of dw in registers
template <int V, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) rms_norm_bwd_kernel(const NormBwdParams p) {
  extern __shared__ float s_dw[];  // [H]
  __shared__ float s_part[2][THREADS / 32];
  const int rows = blockDim.x / p.tpr, lr = threadIdx.x / p.tpr, sub = threadIdx.x % p.tpr;
  const int cpr = p.H / 8;
  const float inv_h = 1.f / (float)p.H;
  pdl_wait();
  const int groups = (p.T + rows - 1) / rows;
  float dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  int buf = 0;
  for (int grp = blockIdx.x; grp < groups; grp += gridDim.x, buf ^= 1) {
    const int t = grp * rows + lr;
    const size_t at = (size_t)t * p.H;
    uint4 rv[V], gv[V], dv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = sub + i * p.tpr;
      const bool ok = t < p.T && c < cpr;
      rv[i] = ok ? reinterpret_cast<const uint4*>(p.r + at)[c] : make_uint4(0, 0, 0, 0);
      gv[i] = ok ? reinterpret_cast<const uint4*>(p.dy + at)[c] : make_uint4(0, 0, 0, 0);
      if (p.dr) dv[i] = ok ? reinterpret_cast<const uint4*>(p.dr + at)[c] : make_uint4(0, 0, 0, 0);
    }
    const float rs = t < p.T ? p.rstd[t] : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = sub + i * p.tpr;
      const uint4 wv = c < cpr ? __ldg(reinterpret_cast<const uint4*>(p.w) + c) : make_uint4(0, 0, 0, 0);
      const uint32_t* wp = reinterpret_cast<const uint32_t*>(&wv);
      const uint32_t *a = reinterpret_cast<const uint32_t*>(&rv[i]), *g = reinterpret_cast<const uint32_t*>(&gv[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p0 = bf16_lo(g[j]) * (bf16_lo(a[j]) * rs), p1 = bf16_hi(g[j]) * (bf16_hi(a[j]) * rs);
        dw[i][2 * j] += p0;
        dw[i][2 * j + 1] += p1;
        dot = fmaf(p0, bf16_lo(wp[j]), dot);
        dot = fmaf(p1, bf16_hi(wp[j]), dot);
      }
    }
    const float mean = row_sum<true>(dot, p.tpr, s_part[buf]) * inv_h;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = sub + i * p.tpr;
      if (t >= p.T || c >= cpr) continue;
      const uint4 wv = __ldg(reinterpret_cast<const uint4*>(p.w) + c);
      const uint32_t* wp = reinterpret_cast<const uint32_t*>(&wv);
      const uint32_t *a = reinterpret_cast<const uint32_t*>(&rv[i]), *g = reinterpret_cast<const uint32_t*>(&gv[i]);
      const uint32_t* d = reinterpret_cast<const uint32_t*>(&dv[i]);
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float d0 = rs * fmaf(-bf16_lo(a[j]) * rs, mean, bf16_lo(g[j]) * bf16_lo(wp[j]));
        float d1 = rs * fmaf(-bf16_hi(a[j]) * rs, mean, bf16_hi(g[j]) * bf16_hi(wp[j]));
        if (p.dr) {
          d0 += bf16_lo(d[j]);
          d1 += bf16_hi(d[j]);
        }
        o[j] = pack2(d0, d1);
      }
      __stcs(reinterpret_cast<uint4*>(p.dx + at) + c, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
  // the block's rows, one after another, into one row of partial sums
  for (int k = 0; k < rows; ++k) {
    if (lr == k) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = sub + i * p.tpr;
        if (c >= cpr) continue;
        float4* s = reinterpret_cast<float4*>(s_dw) + 2 * c;
        float4 lo = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
        float4 hi = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        if (k > 0) {
          const float4 a = s[0], b = s[1];
          lo = make_float4(a.x + lo.x, a.y + lo.y, a.z + lo.z, a.w + lo.w);
          hi = make_float4(b.x + hi.x, b.y + hi.y, b.z + hi.z, b.w + hi.w);
        }
        if (k == rows - 1) {
          float4* o = reinterpret_cast<float4*>(p.part + (size_t)blockIdx.x * p.H) + 2 * c;
          o[0] = lo;
          o[1] = hi;
        } else {
          s[0] = lo;
          s[1] = hi;
        }
      }
    }
    __syncthreads();
  }
}

// dw[h] = sum over the partial rows, in a fixed order: 16 columns a block, four threads
// across them; each of 64 groups of four takes every 64th row, then a tree.
constexpr int kDwCols = 16, kDwGroups = 64;
__global__ void __launch_bounds__(kDwCols / 4 * kDwGroups)
    rms_norm_dw_kernel(const float* __restrict__ part, float* __restrict__ dw, int parts, int H) {
  __shared__ float4 s[kDwGroups][kDwCols / 4];
  const int c = threadIdx.x % (kDwCols / 4), g = threadIdx.x / (kDwCols / 4);
  pdl_wait();
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = g; i < parts; i += kDwGroups) {
    const float4 v = reinterpret_cast<const float4*>(part + (size_t)i * H + blockIdx.x * kDwCols)[c];
    a = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
  }
  s[g][c] = a;
#pragma unroll
  for (int o = kDwGroups / 2; o; o >>= 1) {
    __syncthreads();
    if (g < o) {
      const float4 v = s[g + o][c];
      a = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
      s[g][c] = a;
    }
  }
  if (g == 0) reinterpret_cast<float4*>(dw + blockIdx.x * kDwCols)[c] = a;
}

constexpr int kMaxParts = 608;  // rows of partial sums, and blocks of the gradient

moe_status_t launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) {
    set_error("%s launch: %s", what, cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return check_launch(what);
}

}  // namespace

moe_status_t launch_rms_norm(const moe_layer_desc_t& d, const bf16* x, const bf16* res, const bf16* w,
                             float eps, bf16* r, bf16* y, uint8_t* yq, uint8_t* ys, float* rstd,
                             cudaStream_t st) {
  if (d.T == 0) return MOE_OK;
  // Two groups of 8 columns a thread, four in rows of more than 2048, unless every row has an SM.
  // us with 8-bit rows, two against four against eight groups:
  //   rows                     608             4096            32768
  //   H 320                2.8  3.1  4.2   3.2  3.6  5.3    20   19   30
  //   H 2048               2.9  3.7  5.3  13.4 15.0 15.0    88   90   93
  //   H 4096               4.0  4.3  6.1  26.5 24.7 28.6   190  173  178
  //   H 16384               22   17   21   120   91   96
  // and blocks of 128 threads, or one row: of 32, H 320 4.4 and 20.5, of 256 3.5 and 21.5.
  const int vecs = d.H > 2048 && d.T > device_sm_count() ? 4 : 2;
  // Of the sums, whatever H (2^14 at most), those where mean + eps may be outside of 2^-100 to fp32's
  // largest: at the former the squares that fall below fp32's normal range lose 2^-49 of it.
  NormParams p = {x, res, w, eps, r, y, yq, reinterpret_cast<uint32_t*>(ys), rstd, d.T, d.H,
                  row_threads(d.H, vecs), eps < 0x1p-100f ? 0x1p-86f : 0.f, eps < 0x1p126f ? FLT_MAX : -1.f};
  const int threads = std::max(p.tpr, 128), rows = threads / p.tpr, grid = ceil_div(d.T, rows);
  const size_t smem = yq ? (size_t)rows * ceil_div(d.H, 512) * 4 : 0;
  cudaError_t e;
  {
    LaunchScope _ls(K_NORM, st);
    e = vecs == 2 ? launch_k(rms_norm_kernel<2, 1024, 48>, grid, threads, smem, st, p)
                  : launch_k(rms_norm_kernel<4, 512, 64>, grid, threads, smem, st, p);
  }
  return launched(e, "rms_norm_kernel");
}

size_t rms_norm_bwd_ws_bytes(const moe_layer_desc_t& d) {
  return (size_t)std::min(std::max(d.T, 1), kMaxParts) * d.H * sizeof(float);
}

moe_status_t launch_rms_norm_bwd(const moe_layer_desc_t& d, const bf16* dy, const bf16* dr, const bf16* r,
                                 const bf16* w, const float* rstd, bf16* dx, float* dw, float* part,
                                 cudaStream_t st) {
  int grid = 0;
  cudaError_t e = cudaSuccess;
  if (d.T > 0) {
    // Rows of up to 4096: three blocks of 256 threads with two groups of 8 columns each (4096 x
    // 2048: 17.3 us with the sum over blocks; four groups and two blocks 18.4, one group and
    // four blocks 18.7, four groups in one block, which is what fits unasked, 24.3)
    const bool wide = d.H > 4096;
    NormBwdParams p = {dy, dr, r, w, rstd, dx, part, d.T, d.H, row_threads(d.H, wide ? 4 : 2)};
    const int threads = wide ? 512 : 256, rows = threads / p.tpr;
    grid = std::min({ceil_div(d.T, rows), device_sm_count() * (wide ? 1 : 3), kMaxParts});
    const size_t smem = rows > 1 ? (size_t)d.H * sizeof(float) : 0;
    LaunchScope _ls(K_NORM_BWD, st);
    e = wide ? launch_k(rms_norm_bwd_kernel<4, 512, 1>, grid, threads, smem, st, p)
             : launch_k(rms_norm_bwd_kernel<2, 256, 3>, grid, threads, smem, st, p);
  }
  if (e == cudaSuccess) {
    LaunchScope _ls(K_NORM_DW, st);
    e = launch_k(rms_norm_dw_kernel, d.H / kDwCols, kDwCols / 4 * kDwGroups, 0, st,
                 (const float*)part, dw, grid, d.H);
  }
  return launched(e, "rms_norm_bwd_kernel");
}

}  // namespace moe

using namespace moe;

#define S(st) static_cast<cudaStream_t>(st)
#define BF(p) reinterpret_cast<const bf16*>(p)
#define BFW(p) reinterpret_cast<bf16*>(p)

extern "C" {

moe_status_t moe_rms_norm(const moe_layer_desc_t* d, const moe_bf16* x, const moe_bf16* res,
                          const moe_bf16* w, float eps, moe_bf16* r, moe_bf16* y, moe_e4m3* yq,
                          moe_e8m0* ys, float* rstd, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(x); MOE_PTR_OPT(res); MOE_PTR(w); MOE_PTR_OPT(r); MOE_PTR_OPT(y); MOE_PTR_OPT(yq);
  MOE_PTR_OPT(ys); MOE_PTR_OPT(rstd);
  if (!(eps >= 0.f) || isinf(eps)) { set_error("eps must be finite and not negative"); return MOE_ERR_INVALID_ARG; }
  if (r && !res) { set_error("r is the sum with res, which is NULL"); return MOE_ERR_INVALID_ARG; }
  if (!y && !yq) { set_error("y and yq are both NULL"); return MOE_ERR_INVALID_ARG; }
  if (!yq != !ys) { set_error("yq and ys are given together or not at all"); return MOE_ERR_INVALID_ARG; }
  return launch_rms_norm(*d, BF(x), BF(res), BF(w), eps, BFW(r), BFW(y), yq, ys, rstd, S(stream));
}

size_t moe_rms_norm_bwd_workspace_size(const moe_layer_desc_t* d) {
  return validate(d) == MOE_OK ? rms_norm_bwd_ws_bytes(*d) : 0;
}

moe_status_t moe_rms_norm_bwd(const moe_layer_desc_t* d, const moe_bf16* dy, const moe_bf16* dr,
                              const moe_bf16* r, const moe_bf16* w, const float* rstd, moe_bf16* dx,
                              float* dw, void* ws, size_t ws_bytes, void* stream) {
  MOE_CHECK(validate(d));
  MOE_PTR(dy); MOE_PTR_OPT(dr); MOE_PTR(r); MOE_PTR(w); MOE_PTR(rstd); MOE_PTR(dx); MOE_PTR(dw);
  MOE_PTR(ws);
  if (ws_bytes < rms_norm_bwd_ws_bytes(*d)) {
    set_error("workspace of %zu bytes is smaller than moe_rms_norm_bwd_workspace_size() = %zu",
              ws_bytes, rms_norm_bwd_ws_bytes(*d));
    return MOE_ERR_INVALID_ARG;
  }
  return launch_rms_norm_bwd(*d, BF(dy), BF(dr), BF(r), BF(w), rstd, BFW(dx), dw,
                             static_cast<float*>(ws), S(stream));
}

}  // extern "C"
