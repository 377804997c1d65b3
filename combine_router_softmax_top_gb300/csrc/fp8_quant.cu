// The quantising passes of the 8-bit experts: the weights into e4m3 and 128 x
// 128 block scales, the permute (tokens sorted by expert into the send layout)
// and the gradient of the weighted return, both writing e4m3 rows with one
// scale for each 128 columns. All three are bound by HBM.
#include <algorithm>

#include "fp8_mma.cuh"

namespace moe {

namespace {

__device__ __forceinline__ uint32_t max8(uint32_t m, const uint4& v) {
  m = absmax_bf16x2(m, v.x);
  m = absmax_bf16x2(m, v.y);
  m = absmax_bf16x2(m, v.z);
  return absmax_bf16x2(m, v.w);
}

// ------------------------------------------------------------------ weights
// One CTA per 128 x 128 block. A thread holds 16 columns of 4 rows in registers
// between the pass that finds the block's maximum and the one that rounds, so
// each weight is read once: 2 bytes in, 1 byte out. A row of the block is 256
// contiguous bytes in and 128 out, whole lines both ways. 128 experts of 2048 x 768:
// 1812 MB in 254 us, 7.1 TB/s (more than a copy, as reads outweigh writes).
struct WeightMat {
  const bf16* w;
  uint8_t* q;
  uint8_t* s;
  int R, C, rb, cb;  // rows and columns of a matrix, and their blocks
  long long blocks;  // over all matrices
};

__global__ void __launch_bounds__(256) quantize_weights_kernel(WeightMat m1, WeightMat m2) {
  pdl_wait();
  __shared__ uint32_t s_max[8];
  const bool first = (long long)blockIdx.x < m1.blocks;
  const WeightMat m = first ? m1 : m2;
  const long long blk = (long long)blockIdx.x - (first ? 0 : m1.blocks);
  const int cbi = (int)(blk % m.cb);
  const long long rest = blk / m.cb;
  const int rbi = (int)(rest % m.rb);
  const long long mat = rest / m.rb;
  const int col = cbi * kFp8Block + (threadIdx.x & 7) * 16;
  const int row = rbi * kFp8Block + (threadIdx.x >> 3);
  const size_t at = ((size_t)mat * m.R + row) * m.C + col;
  const bool cok = col < m.C;  // C is a multiple of 64: 16 columns are in or out together
  uint4 v[8];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool ok = cok && row + 32 * i < m.R;
    const uint4* src = reinterpret_cast<const uint4*>(m.w + at + (size_t)32 * i * m.C);
    v[2 * i] = ok ? __ldcs(src) : make_uint4(0, 0, 0, 0);
    v[2 * i + 1] = ok ? __ldcs(src + 1) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = max8(mx, v[i]);
  mx = __reduce_max_sync(0xffffffffu, absmax_bits(mx));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = max(mx, s_max[i]);
  const uint32_t b = fp8_scale_byte(mx);
  const uint32_t inv = fp8_inv_scale2(b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (cok && row + 32 * i < m.R) {
      const uint4 a = v[2 * i], c = v[2 * i + 1];
      *reinterpret_cast<uint4*>(m.q + at + (size_t)32 * i * m.C) =
          make_uint4(fp8x4_of_bf16(a.x, a.y, inv), fp8x4_of_bf16(a.z, a.w, inv),
                     fp8x4_of_bf16(c.x, c.y, inv), fp8x4_of_bf16(c.z, c.w, inv));
    }
  }
  if (threadIdx.x == 0) m.s[blk] = (uint8_t)b;
}

// ------------------------------------------------------------------ permute
// xq[slot[t,j]] = e4m3(x[t] / scale). A warp takes one token's 512 columns
// (four blocks, the four bytes of one scale word): it reads and rounds them
// once and writes them to the token's k rows, so x is read once and only the
// 8-bit rows are written. Lane j holds the token's j-th slot. 4096 tokens of 2048,
// 8 rows each: 84 MB in 13.9 to 14.5 us, 6 TB/s (plain stores 14.9; with the forward behind
// it, which reads the rows, 168.6 us either way); one token 5.5 us, the call itself. (A
// token's blocks need no exchange between warps, so a decode batch has a warp for
// every 512 columns.)
__global__ void __launch_bounds__(256) permute_fp8_kernel(const bf16* __restrict__ x,
                                                          const int32_t* __restrict__ slot,
                                                          uint8_t* __restrict__ xq,
                                                          uint32_t* __restrict__ xs, int T, int H,
                                                          int k, long long N, int nseg) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
  const long long tasks = (long long)T * nseg;
  for (long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < tasks;
       w += warps) {
    const int t = (int)(w / nseg), seg = (int)(w % nseg);
    const int col = seg * 512 + lane * 16;
    const bool ok = col < H;
    const uint4* src = reinterpret_cast<const uint4*>(x + (size_t)t * H + col);
    uint4 a = make_uint4(0, 0, 0, 0), c = a;
    if (ok) {
      a = __ldg(src);
      c = __ldg(src + 1);
    }
    int sl = lane < k ? slot[(size_t)t * k + lane] : -1;
    if (sl >= N) sl = -1;
    uint32_t m = absmax_bits(max8(max8(0, a), c));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t b = fp8_scale_byte(m);
    const uint32_t inv = fp8_inv_scale2(b);
    const uint4 q = make_uint4(fp8x4_of_bf16(a.x, a.y, inv), fp8x4_of_bf16(a.z, a.w, inv),
                               fp8x4_of_bf16(c.x, c.y, inv), fp8x4_of_bf16(c.z, c.w, inv));
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) word |= __shfl_sync(0xffffffffu, b, 8 * i) << (8 * i);
    if (sl >= 0) xs[(size_t)seg * N + sl] = word;
    for (int j = 0; j < k; ++j) {
      const int s = __shfl_sync(0xffffffffu, sl, j);
      if (s >= 0 && ok) __stcs(reinterpret_cast<uint4*>(xq + (size_t)s * H + col), q);
    }
  }
}

// ------------------------------------------------------------------ combine backward
// d_o[slot[t,j]] = bf16(g[t,j] dy[t]), held as e4m3 rows dq with scale words
// ds (and as bf16 when d_o is given); dgates[t,j] = <dy[t], o[slot[t,j]]>.
// Rounding to bf16 and multiplying by |g| both keep order, so a block's largest
// |bf16(g dy)| is bf16(|g| max|dy|): one reduction over dy's block serves all k
// rows. 128 / tpr tokens a group; thread `sub` of a token takes 8 columns, 16
// threads a block. Groups are taken in turn, the next group's routing state
// loaded beside the current rows.
//
// A group's phases (loads, arithmetic and stores, the dot product's reduction) do
// not overlap within a block, so many small blocks do better than few large ones:
// on the 4096-token layer with d_o, 128 threads x 8 blocks an SM with 4 rows in
// flight 63.5 us, 256 x 3 with 8 rows 65.1 us, 256 x 2 78 us, 64 x 12 68 us; one
// token's 8 columns a thread over 256 threads 67 us. 353 MB in 63.2 us, 5.6 TB/s: 0.82
// of the copy rate, as the bf16 gathers of this layer reach.
constexpr int kRowsInFlight = 4;
constexpr int kCombineThreads = 128;
constexpr int kCombineBlocks = 8;  // resident blocks an SM, k <= 8

template <int KMAX>
__global__ void __launch_bounds__(kCombineThreads, KMAX <= 8 ? kCombineBlocks : 1) combine_bwd_fp8_kernel(
    const bf16* __restrict__ dy, const bf16* __restrict__ o, const int32_t* __restrict__ slot,
    const float* __restrict__ gates, bf16* __restrict__ d_o, uint8_t* __restrict__ dq,
    uint32_t* __restrict__ ds, float* __restrict__ dgates, int T, int H, int k, long long N, int tpr,
    int* __restrict__ zero, int nzero) {
  pdl_wait();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < nzero; i += blockDim.x) zero[i] = 0;
  __shared__ float s_part[kCombineThreads / 32][KMAX];
  __shared__ uint32_t s_scale[KMAX * 32];  // the group's scale words [token][j][word]: tokens x words <= 32
  __shared__ int s_slot[2][kCombineThreads / 8 * KMAX];  // tpr >= 8
  __shared__ float s_g[2][kCombineThreads / 8 * KMAX];
  const int tpb = blockDim.x / tpr;
  const int lt = threadIdx.x / tpr, sub = threadIdx.x % tpr;
  const int cpr = H / 8;
  const int nw = (H + 4 * kFp8Block - 1) / (4 * kFp8Block);  // scale words of a row
  const int ngroups = (T + tpb - 1) / tpb;
  const int nent = tpb * k;
  auto stage = [&](int buf, int grp) {
    const long long e0 = (long long)grp * nent;
    for (int i = threadIdx.x; i < nent; i += blockDim.x) {
      const long long e = e0 + i;
      int sv = -1;
      float gv = 0.f;
      if (grp < ngroups && e < N) {
        sv = slot[e];
        gv = gates[e];
      }
      s_slot[buf][i] = sv >= 0 && sv < N ? sv : -1;
      s_g[buf][i] = gv;
    }
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int width = tpr < 32 ? tpr : 32;
  int buf = 0;
  stage(0, blockIdx.x);
  __syncthreads();
  for (int grp = blockIdx.x; grp < ngroups; grp += gridDim.x, buf ^= 1) {
    const int t = grp * tpb + lt;
    const bool active = t < T;
    const int* sl = s_slot[buf] + lt * k;
    const float* gl = s_g[buf] + lt * k;
    float dot[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) dot[j] = 0.f;
    bool next_staged = false;
    // the last word's bytes past the row's blocks stay 0
    for (int j = sub; j < k; j += tpr) s_scale[(lt * k + j) * nw + nw - 1] = 0;
    __syncthreads();
    for (int c0 = 0; c0 < cpr; c0 += tpr) {  // the same trips for every thread: they shuffle
      const int c = c0 + sub;
      const bool ok = active && c < cpr;
      uint4 yv = make_uint4(0, 0, 0, 0);
      if (ok) yv = __ldg(reinterpret_cast<const uint4*>(dy + (size_t)t * H) + c);
      const uint32_t yw[4] = {yv.x, yv.y, yv.z, yv.w};
      uint32_t mb = absmax_bits(max8(0, yv));
#pragma unroll
      for (int i = 1; i < 16; i <<= 1)
        if (i < width) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, i));
      const float ymax = __uint_as_float(mb);
#pragma unroll
      for (int j0 = 0; j0 < KMAX; j0 += kRowsInFlight) {
        uint4 ov[kRowsInFlight];
#pragma unroll
        for (int u = 0; u < kRowsInFlight; ++u) {
          const int j = j0 + u;
          const int sv = (ok && j < KMAX && j < k) ? sl[j] : -1;
          ov[u] = sv >= 0 ? __ldcs(reinterpret_cast<const uint4*>(o + (size_t)sv * H) + c)
                          : make_uint4(0, 0, 0, 0);
        }
        if (!next_staged) {  // the next group's routing state, beside the row loads
          stage(buf ^ 1, grp + gridDim.x);
          next_staged = true;
        }
#pragma unroll
        for (int u = 0; u < kRowsInFlight; ++u) {
          const int j = j0 + u;
          if (!ok || j >= KMAX || j >= k) continue;
          const int sv = sl[j];
          if (sv < 0) continue;
          const float gj = gl[j];
          const uint32_t ow[4] = {ov[u].x, ov[u].y, ov[u].z, ov[u].w};
          uint32_t pw[4];
          float d = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float y0 = bf16_lo(yw[i]), y1 = bf16_hi(yw[i]);
            d = fmaf(y0, bf16_lo(ow[i]), d);
            d = fmaf(y1, bf16_hi(ow[i]), d);
            __nv_bfloat162 p2 = __floats2bfloat162_rn(gj * y0, gj * y1);
            pw[i] = *reinterpret_cast<uint32_t*>(&p2);
          }
          dot[j] += d;
          const float pm = __bfloat162float(__float2bfloat16_rn(fabsf(gj) * ymax));
          const uint32_t b = fp8_scale_byte(__float_as_uint(pm) & 0x7FFFFFFFu);
          const uint32_t inv = fp8_inv_scale2(b);
          *reinterpret_cast<uint2*>(dq + (size_t)sv * H + 8 * c) =
              make_uint2(fp8x4_of_bf16(pw[0], pw[1], inv), fp8x4_of_bf16(pw[2], pw[3], inv));
          if ((c & 15) == 0)
            reinterpret_cast<uint8_t*>(s_scale)[(lt * k + j) * 4 * nw + (c >> 4)] = (uint8_t)b;
          if (d_o)
            __stcs(reinterpret_cast<uint4*>(d_o + (size_t)sv * H) + c,
                   make_uint4(pw[0], pw[1], pw[2], pw[3]));
        }
      }
    }
    if (!next_staged) stage(buf ^ 1, grp + gridDim.x);
    // dot[] over the token's threads, in a fixed tree order
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
#pragma unroll
      for (int i = 16; i; i >>= 1)
        if (i < width) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], i, width);
    }
    if (tpr <= 32) {
      if (active && sub == 0) {
#pragma unroll
        for (int j = 0; j < KMAX; ++j)
          if (j < k) dgates[(size_t)t * k + j] = dot[j];
      }
    } else {
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < KMAX; ++j) s_part[warp][j] = dot[j];
      }
      __syncthreads();
      const int wbase = lt * (tpr / 32);
      if (active && sub < k) {
        float sum = 0.f;
        for (int w = 0; w < tpr / 32; ++w) sum += s_part[wbase + w][sub];
        dgates[(size_t)t * k + sub] = sum;
      }
    }
    if (tpr <= 32) __syncthreads();  // (longer rows have met above)
    // whole scale words: their bytes come from several warps
    for (int i = threadIdx.x; i < nent * nw; i += blockDim.x) {
      const int ent = i / nw, w = i % nw, sv = s_slot[buf][ent];
      if (sv >= 0) ds[(size_t)w * N + sv] = s_scale[i];
    }
    __syncthreads();
  }
}

template <int KMAX>
cudaError_t launch_combine_bwd_fp8_t(const moe_layer_desc_t& d, int groups, const bf16* dy,
                                     const bf16* o, const int32_t* slot, const float* gates,
                                     bf16* d_o, uint8_t* dq, uint8_t* ds, float* dgates, int tpr,
                                     int* zero, int nzero, cudaStream_t st) {
  // one wave of resident blocks, each taking token groups in turn
  const int grid = std::min(groups, (KMAX <= 8 ? kCombineBlocks : 1) * device_sm_count());
  return launch_k(combine_bwd_fp8_kernel<KMAX>, grid, kCombineThreads, 0, st, dy, o, slot, gates, d_o, dq,
                  reinterpret_cast<uint32_t*>(ds), dgates, d.T, d.H, d.k, (long long)d.T * d.k, tpr,
                  zero, nzero);
}

moe_status_t launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) {
    set_error("%s launch: %s", what, cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return check_launch(what);
}

}  // namespace

moe_status_t launch_fp8_quantize_weights(const moe_layer_desc_t& d, const bf16* w1, const bf16* w2,
                                         uint8_t* w1q, uint8_t* w1s, uint8_t* w2q, uint8_t* w2s,
                                         cudaStream_t st) {
  const int nf = fp8_blocks(d.F), nh = fp8_blocks(d.H);
  const WeightMat m1 = {w1, w1q, w1s, d.F, d.H, nf, nh, 2ll * d.E * nf * nh};
  const WeightMat m2 = {w2, w2q, w2s, d.H, d.F, nh, nf, (long long)d.E * nh * nf};
  cudaError_t e;
  {
    LaunchScope _ls(K_FP8_QUANT_W, st);
    e = launch_k(quantize_weights_kernel, dim3((unsigned)(m1.blocks + m2.blocks)), 256, 0, st, m1,
                 m2);
  }
  return launched(e, "quantize_weights_kernel");
}

moe_status_t launch_permute_fp8(const moe_layer_desc_t& d, const bf16* x, const int32_t* slot,
                                uint8_t* xq, uint8_t* xs, cudaStream_t st) {
  const long long N = (long long)d.T * d.k;
  if (N == 0) return MOE_OK;
  const int nseg = ceil_div(d.H, 512);
  const long long blocks = ((long long)d.T * nseg + 7) / 8;
  const int grid = (int)std::min<long long>(blocks, (long long)device_sm_count() * 16);
  cudaError_t e;
  {
    LaunchScope _ls(K_FP8_PERMUTE, st);
    e = launch_k(permute_fp8_kernel, grid, 256, 0, st, x, slot, xq,
                 reinterpret_cast<uint32_t*>(xs), d.T, d.H, d.k, N, nseg);
  }
  return launched(e, "permute_fp8_kernel");
}

moe_status_t launch_combine_bwd_fp8(const moe_layer_desc_t& d, const bf16* dy, const bf16* o,
                                    const int32_t* slot, const float* gates, bf16* d_o,
                                    uint8_t* dq, uint8_t* ds, float* dgates, cudaStream_t st,
                                    int* zero, int nzero) {
  if (d.T == 0) return MOE_OK;
  // threads of a token: a power of two >= H / 16, at most a block, at least the 16
  // that hold a block of 128 columns
  int tpr = d.H > 64 ? 16 : 8;
  while (tpr < d.H / 16 && tpr < kCombineThreads) tpr <<= 1;
  // while all tokens fit one wave, twice the threads: latency counts, not the rate
  if (tpr < d.H / 8 && tpr < kCombineThreads &&
      ceil_div(d.T, kCombineThreads / (2 * tpr)) <= kCombineBlocks * device_sm_count() / 2)
    tpr *= 2;
  const int groups = ceil_div(d.T, kCombineThreads / tpr);
  cudaError_t e;
  {
    LaunchScope _ls(K_FP8_COMBINE_BWD, st);
#define GO(K)                                                                                     \
  launch_combine_bwd_fp8_t<K>(d, groups, dy, o, slot, gates, d_o, dq, ds, dgates, tpr, zero, nzero, \
                              st)
    e = d.k <= 2 ? GO(2) : d.k <= 4 ? GO(4) : d.k <= 8 ? GO(8) : d.k <= 16 ? GO(16) : GO(32);
#undef GO
  }
  return launched(e, "combine_bwd_fp8_kernel");
}

namespace fp8 {

namespace {

// Clears the counters. A kernel rather than a memset, so that the chain's set-up
// overlaps it (programmatic dependent launch).
__global__ void __launch_bounds__(256) zero_counters_kernel(int* dep, int n, int* tile) {
  pdl_wait();
  if (threadIdx.x == 0) *tile = 0;
  if ((int)threadIdx.x < n) dep[threadIdx.x] = 0;
}

}  // namespace

cudaError_t launch_zero_counters(int* dep, int n, int* tile, cudaStream_t st) {
  LaunchScope _ls(K_FP8_ZERO, st);
  return launch_k(zero_counters_kernel, 1, 256, 0, st, dep, n, tile);
}

}  // namespace fp8
}  // namespace moe
