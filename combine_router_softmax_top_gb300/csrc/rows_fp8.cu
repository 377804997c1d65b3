// The 8-bit expert FFN forward for few rows an expert (a batch of single tokens).
//
// With a handful of rows an expert, the products are a stream of weights: bound
// by HBM (604 MB for the 128-expert layer) however few the rows are. The GEMM
// tiles of grouped_gemm_fp8.cu hold 256 rows each; with 4 rows they spend 512
// clocks of the tensor pipe on 16 KB of weights a CTA, which take 700 clocks to
// arrive. Here the weights are the M operand and the rows the N operand:
//   D[128 weight rows, 32 rows of x] += W[128, 128 of K] X[32, 128 of K]^T
// so that a stage of 32 KB of weights costs a fraction of its arrival, and the
// ring holds 6 stages of weights instead of the rows' padding.
//
// One persistent launch, one CTA per SM, both products' tiles as in the GEMM
// chain (claimed in order from a counter, by warp 2; a tile of the second waits
// for its expert's tiles of the first):
//   FC1 tile: (expert, 128 columns of h, 32 rows): 128 gate and 128 up rows of W1
//   FC2 tile: (expert, 256 columns of o, 32 rows): two times 128 rows of W2
//   warp 0      TMA producer: 2 x 16 KB of weights and up to 4 KB of rows a stage
//   warp 1      TMEM allocator + MMA issuer
//   warps 4..7  epilogue: thread = weight row (column of h or o), registers = rows;
//               block maxima by warp reductions and shared memory
//   warps 8..11 scales into TMEM, ahead of the MMAs
//
// 64 tokens of the 128-expert layer (H 2048, F 768, top 8, skewed): 83 to 85 us for the
// 545 MB of the experts that have rows (112 to 118 of them), 6.5 TB/s, 0.96 of a copy's
// rate. One token: 16 us for 38 MB, a chain of latencies (clocks of a
// CTA, weights in L2): set-up and tables 1900, the first tile's claim and loads 2900,
// its 16 K blocks 10700, epilogue and count 2200, the second product's wait and
// scales 3000, its K blocks 3500, epilogue and end 1500. Two CTAs a tile, half of K
// each, were no faster: what the K loop saves, the cluster's barriers and the exchange
// of sums cost again (15.0 against 15.1 us).
#include <algorithm>
#include <atomic>

#include "fp8_mma.cuh"

namespace moe {

using namespace fp8;

namespace {

constexpr int kFc1 = 0, kFc2 = 1;
constexpr int NT = 32;                        // rows of x in a tile
constexpr int kWBytes = 128 * 128;            // one M tile's weights of a stage
constexpr int kStageBytes = 2 * kWBytes + NT * 128;
constexpr int kStages = 6;
constexpr int kThreads = 384;
constexpr int kMaxE = 256;
constexpr int kAccCols = 2 * NT;              // TMEM columns of one accumulator (two M tiles)
constexpr int kTmemScales = 2 * kAccCols;     // buffers of 12: two M tiles, the rows
constexpr int kSf = 4;                        // (two: a buffer's turn-around is not covered)
constexpr int kTmemCols = 256;
constexpr int kSmallBox = 8;                  // rows of the small TMA box
static_assert(kFp8FewRows * kMaxE < 65536, "16-bit tables");
constexpr size_t kDynSmem = (size_t)kStages * kStageBytes + 1024;

struct RowsParams {
  int E, H, F;
  long long N;
  const int32_t* off;
  const uint8_t* xs;
  Fp8Weights w;
  bf16 *a, *h;
  uint8_t *hq, *hs;
  bf16* o;
  int *status, *dep, *tile;
};

struct Tile {
  int e, n0;          // n0: first column of h or o
  long long row;      // first row
  int rows;           // 1..NT
};

struct SmemCtl {
  uint64_t full[kStages], empty[kStages];
  uint64_t sf_full[kSf], sf_empty[kSf], tmem_full[2], tmem_empty[2], drain;
  uint64_t sched_full[2], sched_empty[2], claim;  // claimed tiles
  int sched[2];
  uint32_t tmem_base;
  int abort;
  uint16_t rtile[kMaxE + 1];      // first row tile of each expert
  uint16_t off[kMaxE + 1];
  uint16_t amax[4][NT];           // block maxima of each warp's columns, as bf16 bits
  uint4 h[NT][16];    // the tile's h, bf16 [row][128]
};

template <int G>
__device__ __forceinline__ int kblocks(const RowsParams& p) {
  return ((G == kFc1 ? p.H : p.F) + 127) / 128;
}
template <int G>
__device__ __forceinline__ int ncols(const RowsParams& p) {  // column blocks of an expert
  return G == kFc1 ? (p.F + 127) / 128 : (p.H + 255) / 256;
}

template <int G>
__device__ __forceinline__ Tile tile_at(const RowsParams& p, const SmemCtl& c, int i, int& cursor) {
  const int nc = ncols<G>(p);
  if (c.rtile[cursor + 1] * nc <= i) {  // (most experts may have no rows)
    int lo = cursor + 1, hi = p.E - 1;  // the first expert that ends past i
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (c.rtile[mid + 1] * nc <= i) lo = mid + 1;
      else hi = mid;
    }
    cursor = lo;
  }
  Tile t;
  t.e = cursor;
  const int cnt = c.off[cursor + 1] - c.off[cursor];
  const int local = i - c.rtile[cursor] * nc, nt = (cnt + NT - 1) / NT;
  const int r = (local % nt) * NT;  // row tiles fastest: they share the weights
  t.n0 = (local / nt) * (G == kFc1 ? 128 : 256);
  t.row = (long long)c.off[cursor] + r;
  t.rows = min(NT, cnt - r);
  return t;
}

__device__ __forceinline__ void flag_timeout(SmemCtl& c, int* status, int where) {
  c.abort = 1;
  atomicExch(status + ST_TIMEOUT, where);
}

__device__ __forceinline__ bool wait_expert(SmemCtl& c, const RowsParams& p, int e) {
  const int target = (c.rtile[e + 1] - c.rtile[e]) * ncols<kFc1>(p);
  if (ld_acquire(p.dep + e) < target) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ld_acquire(p.dep + e) < target) {
      if (*(volatile int*)&c.abort || ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
        flag_timeout(c, p.status, 20);
        return false;
      }
    }
  }
  return true;
}

// The n-th tile claimed for this CTA (past the last: none is left; -1: gave up),
// for the 10 warps that read it: producer, MMA issuer, scales, epilogue.
constexpr int kReaders = 10;
__device__ __forceinline__ int next_tile(SmemCtl& c, uint32_t n, int* status, bool warp) {
  bool ok = ptx::mbar_wait(&c.sched_full[n & 1], (n >> 1) & 1, &c.abort, kWaitLimitNs);
  if (warp) ok = __all_sync(0xffffffffu, ok);
  if (!ok) {
    flag_timeout(c, status, 27);
    return -1;
  }
  const int i = *(volatile int*)&c.sched[n & 1];
  if (warp) __syncwarp();
  if (!warp || (threadIdx.x & 31) == 0) ptx::mbar_arrive(&c.sched_empty[n & 1]);
  return i;
}
__device__ __forceinline__ void claim_tiles(SmemCtl& c, const RowsParams& p, int first, int total) {
  for (uint32_t n = 0;; ++n) {
    if ((n == 1 && !ptx::mbar_wait(&c.claim, 0, &c.abort, kWaitLimitNs)) ||
        !ptx::mbar_wait(&c.sched_empty[n & 1], ((n >> 1) & 1) ^ 1, &c.abort, kWaitLimitNs)) {
      flag_timeout(c, p.status, 28);
      return;
    }
    const int i = min(n > 0 ? atomicAdd(p.tile, 1) : first, total);
    *(volatile int*)&c.sched[n & 1] = i;
    ptx::mbar_arrive(&c.sched_full[n & 1]);
    if (i == total) return;
  }
}

// M tiles of a tile: the second one is past the edge when 128 columns or fewer are left
template <int G>
__device__ __forceinline__ int mtiles(const RowsParams& p, const Tile& t) {
  return G == kFc1 || t.n0 + 128 < p.H ? 2 : 1;
}

template <int G>
__device__ __forceinline__ bool producer_tile(SmemCtl& c, uint8_t* smem, const RowsParams& p,
                                              const CUtensorMap* tmW, const CUtensorMap* tmX,
                                              const CUtensorMap* tmS, const Tile& t, int& stage,
                                              uint32_t& phase) {
  const int nk = kblocks<G>(p), mt = mtiles<G>(p, t);
  const int w0 = G == kFc1 ? t.e * 2 * p.F + t.n0 : t.e * p.H + t.n0;
  const int w1 = w0 + (G == kFc1 ? p.F : 128);
  const bool small = t.rows <= NT / 2;
  const int xrows = small ? (t.rows + kSmallBox - 1) / kSmallBox * kSmallBox : NT;
  bool ready = G == kFc1, ok = true;
  for (int kt = 0; kt < nk && ok; ++kt) {
    if (!ptx::mbar_wait(&c.empty[stage], phase ^ 1, &c.abort, kWaitLimitNs)) {
      flag_timeout(c, p.status, 21);
      return false;
    }
    if (kt == nk / 4) ptx::mbar_arrive(&c.claim);
    uint8_t* s = smem + stage * kStageBytes;
    uint64_t* bar = &c.full[stage];
    const int k0 = kt * 128;
    ptx::mbar_arrive_expect_tx(bar, mt * kWBytes + xrows * 128);
    ptx::tma_load_2d(s, tmW, bar, k0, w0);
    if (mt == 2) ptx::tma_load_2d(s + kWBytes, tmW, bar, k0, w1);
    if (!ready) {  // the weights do not wait for the first product, its rows do
      // (after an abort the stage is still loaded whole: drain_loads waits for stages)
      ok = wait_expert(c, p, t.e);
      asm volatile("fence.proxy.async.global;" ::: "memory");
      ready = true;
    }
    uint8_t* sx = s + 2 * kWBytes;
    if (!small) ptx::tma_load_2d(sx, tmX, bar, k0, (int)t.row);
    else
      for (int r = 0; r < xrows; r += kSmallBox)
        ptx::tma_load_2d(sx + r * 128, tmS, bar, k0, (int)t.row + r);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
  return ok;
}

// Scale byte of weight block (K block kb, M tile i).
template <int G>
__device__ __forceinline__ uint32_t weight_scale(const RowsParams& p, const Tile& t, int kb,
                                                 int i) {
  const int nh = (p.H + 127) / 128, nf = (p.F + 127) / 128;
  const size_t e = t.e;
  if (G == kFc1) return kb < nh ? p.w.w1s[((e * 2 + i) * nf + t.n0 / 128) * nh + kb] : 0;
  const int hb = t.n0 / 128 + i;
  return kb < nf && hb < nh ? p.w.w2s[(e * nh + hb) * nf + kb] : 0;
}

__device__ __forceinline__ void arrive(uint64_t* bar, int lane) {
  ptx::tc_fence_before();
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(bar);
}

template <int G>
__device__ __forceinline__ bool scales_tile(SmemCtl& c, const RowsParams& p, const Tile& t,
                                            uint32_t tmem, uint32_t& group, int quarter, int lane) {
  const int nk = kblocks<G>(p);
  const uint32_t* words = reinterpret_cast<const uint32_t*>(G == kFc1 ? p.xs : p.hs);
  if (G == kFc2) {
    bool ok = true;
    if (lane == 0) ok = wait_expert(c, p, t.e);
    if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
    __syncwarp();  // what lane 0 acquired, for all lanes
  }
  for (int g = 0; g * 4 < nk; ++g, ++group) {
    const uint32_t x = lane < t.rows ? __ldcg(words + (size_t)g * p.N + t.row + lane) : 0;
    const uint32_t b = lane < 8 ? weight_scale<G>(p, t, 4 * g + (lane & 3), lane >> 2) : 0;
    uint32_t wb[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) wb[i >> 2] |= __shfl_sync(0xffffffffu, b, i) << (8 * (i & 3));
    const int buf = group % kSf;
    const bool got =
        ptx::mbar_wait(&c.sf_empty[buf], ((group / kSf) & 1) ^ 1, &c.abort, kWaitLimitNs);
    if (!__all_sync(0xffffffffu, got)) {
      if (lane == 0) flag_timeout(c, p.status, 22);
      return false;
    }
    ptx::tc_fence_after();
    const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + kTmemScales + buf * 12;
    const uint32_t w0[4] = {wb[0], wb[0], wb[0], wb[0]}, w1[4] = {wb[1], wb[1], wb[1], wb[1]};
    const uint32_t wx[4] = {x, x, x, x};  // (32 rows: the first column alone is read)
    tmem_st_x4(at, w0);
    tmem_st_x4(at + 4, w1);
    tmem_st_x4(at + 8, wx);
    tmem_st_wait();
    arrive(&c.sf_full[buf], lane);
  }
  return true;
}

struct MmaState {
  int stage = 0;
  uint32_t phase = 0, group = 0, tiles = 0;
};
template <int G>
__device__ __forceinline__ bool mma_tile(SmemCtl& c, uint32_t smem, const RowsParams& p,
                                         const Tile& t, uint32_t tmem, MmaState& m) {
  constexpr uint32_t idesc = idesc_mxf8(128, NT, 0);
  const uint64_t desc0 = ptx::sdesc_sw128(0, 16, 1024);
  const int nk = kblocks<G>(p), mt = mtiles<G>(p, t);
  const int acc = m.tiles & 1;
  auto wait = [&](uint64_t* bar, uint32_t parity, int where) {
    const bool got = ptx::mbar_wait(bar, parity, &c.abort, kWaitLimitNs);
    if (__all_sync(0xffffffffu, got)) return true;
    flag_timeout(c, p.status, where);
    return false;
  };
  if (!wait(&c.tmem_empty[acc], ((m.tiles >> 1) & 1) ^ 1, 23)) return false;
  ptx::tc_fence_after();
  const uint32_t d = tmem + acc * kAccCols;
  constexpr uint32_t kSel = (1u << 4) | (1u << 29);  // scale byte kb of both operands
  // One lane waits and issues for the whole tile: the eight MMAs of a K block take the
  // tensor pipe 400 to 500 clocks, and waits of the whole warp as long again (one token
  // of the 128-expert layer: 16.9 -> 15.9 us).
  int where = 0;
  if (elect_one()) {
    int stage = m.stage;
    uint32_t phase = m.phase, group = m.group;
    for (int k0 = 0; k0 < nk && !where; k0 += 4, ++group) {
      const int buf = group % kSf;
      if (!ptx::mbar_wait(&c.sf_full[buf], (group / kSf) & 1, &c.abort, kWaitLimitNs)) where = 24;
      const uint32_t sf = tmem + kTmemScales + buf * 12;
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        if (k0 + kb >= nk || where) break;
        if (!ptx::mbar_wait(&c.full[stage], phase, &c.abort, kWaitLimitNs)) {
          where = 25;
          break;
        }
        ptx::tc_fence_after();
        const uint64_t a0 = desc0 | ((smem + stage * kStageBytes) >> 4);
        const uint64_t x = a0 + (2 * kWBytes >> 4);
        const uint32_t on = (k0 + kb) != 0;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          umma_mxf8(d, a0 + kk * 2, x + kk * 2, idesc | kb * kSel, sf, sf + 8, on | (kk != 0));
          if (mt == 2)
            umma_mxf8(d + NT, a0 + (kWBytes >> 4) + kk * 2, x + kk * 2, idesc | kb * kSel, sf + 4,
                      sf + 8, on | (kk != 0));
        }
        ptx::umma_commit(&c.empty[stage]);
        if (kb == 3 || k0 + kb == nk - 1) ptx::umma_commit(&c.sf_empty[buf]);
        if (k0 + kb == nk - 1) ptx::umma_commit(&c.tmem_full[acc]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  }
  where = __reduce_max_sync(0xffffffffu, where);
  if (where) {
    flag_timeout(c, p.status, where);
    return false;
  }
  m.group += (nk + 3) / 4;
  const int at = m.stage + nk;
  m.phase ^= (at / kStages) & 1;
  m.stage = at % kStages;
  ++m.tiles;
  return true;
}

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int G>
__device__ __forceinline__ bool epilogue_tile(SmemCtl& c, const RowsParams& p, const Tile& t,
                                              uint32_t tmem, uint32_t& tiles, int q, int lane) {
  const int acc = tiles & 1, col = q * 32 + lane;  // this thread's weight row
  const bool got = ptx::mbar_wait(&c.tmem_full[acc], (tiles >> 1) & 1, &c.abort, kWaitLimitNs);
  // (after an abort the tile is gone through all the same: the others wait below)
  if (!__all_sync(0xffffffffu, got) && lane == 0) flag_timeout(c, p.status, 26);
  ptx::tc_fence_after();
  const uint32_t tbase = tmem + acc * kAccCols + ((uint32_t)(q * 32) << 16);
  if (G == kFc1) {
    const int f = t.n0 + col;
    const bool ok = f < p.F;  // uniform in the warp: F is a multiple of 64
    for (int r0 = 0; r0 < t.rows; r0 += 8) {
      uint32_t g[8], u[8];
      tmem_ld_x8(tbase + r0, g);
      tmem_ld_x8(tbase + NT + r0, u);
      tmem_ld_wait_x8(g);
      tmem_ld_wait_x8(u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (r0 + j >= t.rows) break;
        const bf16 gb = __float2bfloat16_rn(__uint_as_float(g[j]));
        const bf16 ub = __float2bfloat16_rn(__uint_as_float(u[j]));
        const float gf = __bfloat162float(gb);
        const bf16 hb = __float2bfloat16_rn(gf * sigmoid_f(gf) * __bfloat162float(ub));
        const uint16_t bits = __bfloat16_as_ushort(hb);
        if (p.a && ok) {
          bf16* a = p.a + (size_t)(t.row + r0 + j) * (2 * p.F) + f;
          a[0] = gb;
          a[p.F] = ub;
        }
        reinterpret_cast<uint16_t*>(c.h[r0 + j])[col] = bits;
        const uint32_t mx = __reduce_max_sync(0xffffffffu, ok ? (uint32_t)(bits & 0x7FFFu) : 0u);
        if (lane == 0) c.amax[q][r0 + j] = (uint16_t)mx;
      }
    }
    arrive(&c.tmem_empty[acc], lane);
    epilogue_sync();  // the tile's h and maxima are in shared memory
    const int fb = t.n0 / 128;
    for (int i = col; i < t.rows * 8; i += 128) {  // 16 columns of a row
      const int r = i >> 3, cc = (i & 7) * 16;
      const uint32_t m = max(max((uint32_t)c.amax[0][r], (uint32_t)c.amax[1][r]),
                             max((uint32_t)c.amax[2][r], (uint32_t)c.amax[3][r]));
      const uint32_t b = fp8_scale_byte(m << 16);
      const uint32_t inv = fp8_inv_scale2(b);
      const size_t row = (size_t)(t.row + r);
      if (t.n0 + cc < p.F) {
        const uint4 v0 = c.h[r][(i & 7) * 2], v1 = c.h[r][(i & 7) * 2 + 1];
        *reinterpret_cast<uint4*>(p.hq + row * p.F + t.n0 + cc) =
            make_uint4(fp8x4_of_bf16(v0.x, v0.y, inv), fp8x4_of_bf16(v0.z, v0.w, inv),
                       fp8x4_of_bf16(v1.x, v1.y, inv), fp8x4_of_bf16(v1.z, v1.w, inv));
        if (p.h) {
          uint4* hp = reinterpret_cast<uint4*>(p.h + row * p.F + t.n0 + cc);
          hp[0] = v0;
          hp[1] = v1;
        }
      }
      if (cc == 0) p.hs[((size_t)(fb >> 2) * p.N + row) * 4 + (fb & 3)] = (uint8_t)b;
    }
    epilogue_sync();  // every store issued, and the shared buffers free again
    if (col == 0) {
      __threadfence();
      atomicAdd(p.dep + t.e, 1);
    }
  } else {
    const int mt = mtiles<G>(p, t);
    for (int m = 0; m < mt; ++m) {
      const int h = t.n0 + 128 * m + col;
      for (int r0 = 0; r0 < t.rows; r0 += 8) {
        uint32_t v[8];
        tmem_ld_x8(tbase + NT * m + r0, v);
        tmem_ld_wait_x8(v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (r0 + j < t.rows && h < p.H)
            p.o[(size_t)(t.row + r0 + j) * p.H + h] = __float2bfloat16_rn(__uint_as_float(v[j]));
      }
    }
    arrive(&c.tmem_empty[acc], lane);
  }
  ++tiles;
  return *(volatile int*)&c.abort == 0;
}

__global__ void __launch_bounds__(kThreads, 1)
    rows_ffn_fp8_kernel(const __grid_constant__ CUtensorMap tmW1,
                        const __grid_constant__ CUtensorMap tmX1,
                        const __grid_constant__ CUtensorMap tmS1,
                        const __grid_constant__ CUtensorMap tmW2,
                        const __grid_constant__ CUtensorMap tmX2,
                        const __grid_constant__ CUtensorMap tmS2, const RowsParams p) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ SmemCtl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) &
                                             ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&ctl.full[s], 1);
      ptx::mbar_init(&ctl.empty[s], 1);
    }
    for (int b = 0; b < kSf; ++b) {
      ptx::mbar_init(&ctl.sf_full[b], 4);
      ptx::mbar_init(&ctl.sf_empty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&ctl.tmem_full[b], 1);
      ptx::mbar_init(&ctl.tmem_empty[b], 4);
      ptx::mbar_init(&ctl.sched_full[b], 1);
      ptx::mbar_init(&ctl.sched_empty[b], kReaders);
    }
    ptx::mbar_init(&ctl.drain, 1);
    ptx::mbar_init(&ctl.claim, 1);
    ctl.abort = 0;
    ptx::fence_mbar_init();
    for (const CUtensorMap* m : {&tmW1, &tmX1, &tmS1, &tmW2, &tmX2, &tmS2})
      ptx::tma_prefetch_desc(m);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&ctl.tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  }
  pdl_wait();
  int first = 0;  // the first tile, claimed while the tables are made
  if (warp == 2 && lane == 0) first = atomicAdd(p.tile, 1);
  // offsets outside 0..N would send stores out of the buffers
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x)
    ctl.off[e] = (uint16_t)min(max((long long)p.off[e], 0ll), p.N);
  __syncthreads();
  if (warp == 0) {  // row tiles of the experts -> exclusive prefix, 8 experts a lane
    int n[kMaxE / 32], sum = 0;
#pragma unroll
    for (int k = 0; k < kMaxE / 32; ++k) {
      const int e = lane * (kMaxE / 32) + k;
      n[k] = sum;
      if (e < p.E) sum += max(0, (ctl.off[e + 1] - ctl.off[e] + NT - 1) / NT);
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
#pragma unroll
    for (int k = 0; k < kMaxE / 32; ++k) {
      const int e = lane * (kMaxE / 32) + k;
      if (e < p.E) ctl.rtile[e] = (uint16_t)(incl - sum + n[k]);
    }
    if (lane == 31) ctl.rtile[p.E] = (uint16_t)incl;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  const int total1 = ctl.rtile[p.E] * ncols<kFc1>(p);
  const int total = total1 + ctl.rtile[p.E] * ncols<kFc2>(p);
  int cur1 = 0, cur2 = 0;
  auto tile1 = [&](int i) { return tile_at<kFc1>(p, ctl, i, cur1); };
  auto tile2 = [&](int i) { return tile_at<kFc2>(p, ctl, i - total1, cur2); };
  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (uint32_t n = 0; ok; ++n) {
        const int i = next_tile(ctl, n, p.status, false);
        ok = i >= 0;
        if (!ok || i >= total) break;
        ok = i < total1
                 ? producer_tile<kFc1>(ctl, smem, p, &tmW1, &tmX1, &tmS1, tile1(i), stage, phase)
                 : producer_tile<kFc2>(ctl, smem, p, &tmW2, &tmX2, &tmS2, tile2(i), stage, phase);
      }
      if (!ok) drain_loads(ctl.full, kStages, stage, phase);
    }
    __syncwarp();
  } else if (warp == 1) {
    MmaState m;
    for (uint32_t n = 0; ok; ++n) {
      const int i = next_tile(ctl, n, p.status, true);
      ok = i >= 0;
      if (!ok || i >= total) break;
      ok = i < total1 ? mma_tile<kFc1>(ctl, ptx::smem_u32(smem), p, tile1(i), tmem, m)
                      : mma_tile<kFc2>(ctl, ptx::smem_u32(smem), p, tile2(i), tmem, m);
    }
    __syncwarp();
    if (elect_one()) ptx::umma_commit(&ctl.drain);  // no MMA may still run when TMEM is released
    if (!ptx::mbar_wait(&ctl.drain, 0, &ctl.abort, kWaitLimitNs)) {
      int dummy = 0;
      ptx::mbar_wait(&ctl.drain, 0, &dummy, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) claim_tiles(ctl, p, first, total);
    __syncwarp();
  } else if (warp >= 8) {
    uint32_t group = 0;
    for (uint32_t n = 0; ok; ++n) {
      const int i = next_tile(ctl, n, p.status, true);
      ok = i >= 0;
      if (!ok || i >= total) break;
      ok = i < total1 ? scales_tile<kFc1>(ctl, p, tile1(i), tmem, group, warp - 8, lane)
                      : scales_tile<kFc2>(ctl, p, tile2(i), tmem, group, warp - 8, lane);
    }
  } else if (warp >= 4) {
    uint32_t tiles = 0;
    for (uint32_t n = 0;; ++n) {
      const int i = next_tile(ctl, n, p.status, true);
      // the four warps enter a tile together or not at all: they meet at barriers in it
      int stop;
      asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                   "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
                   : "=r"(stop)
                   : "r"((int)(i < 0 || i >= total || !ok))
                   : "memory");
      if (stop) break;
      ok = i < total1 ? epilogue_tile<kFc1>(ctl, p, tile1(i), tmem, tiles, warp - 4, lane)
                      : epilogue_tile<kFc2>(ctl, p, tile2(i), tmem, tiles, warp - 4, lane);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, kTmemCols);
}

// Sets the kernel's shared memory up, once for each device.
cudaError_t set_up() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (ready.load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(rows_ffn_fp8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kDynSmem);
  if (e == cudaSuccess) ready.fetch_or(bit);
  return e;
}

}  // namespace

moe_status_t launch_ffn_rows_fp8(const moe_layer_desc_t& d, const uint8_t* xq, const uint8_t* xs,
                                 const int32_t* off, const Fp8Weights& w, bf16* a, bf16* h,
                                 uint8_t* hq, uint8_t* hs, bf16* o, int* status, int* dep,
                                 cudaStream_t st) {
  const long long N = (long long)d.T * d.k;
  CUtensorMap m[6];
  if (!make_map(&m[0], w.w1q, 2, d.H, 2ll * d.E * d.F, 1, 128, 1) ||
      !make_map(&m[1], xq, 2, d.H, N, 1, NT, 1) || !make_map(&m[2], xq, 2, d.H, N, 1, kSmallBox, 1) ||
      !make_map(&m[3], w.w2q, 2, d.F, (long long)d.E * d.H, 1, 128, 1) ||
      !make_map(&m[4], hq, 2, d.F, N, 1, NT, 1) || !make_map(&m[5], hq, 2, d.F, N, 1, kSmallBox, 1))
    return MOE_ERR_CUDA;
  const RowsParams p = {d.E, d.H, d.F, N, off, xs, w, a, h, hq, hs, o, status, dep,
                        tile_counter(status)};
  cudaError_t e = set_up();
  if (e == cudaSuccess) e = launch_zero_counters(dep, d.E, p.tile, st);
  // one CTA per SM, fewer when there cannot be as many tiles
  const long long rows = N / NT + std::min<long long>(N, d.E);
  const long long tiles = rows * (fp8_blocks(d.F) + fp8_blocks(d.H));
  const int grid = (int)std::min<long long>(device_sm_count(), tiles);
  if (e == cudaSuccess) {
    LaunchScope _ls(K_FP8_ROWS_FFN, st);
    e = launch_k(rows_ffn_fp8_kernel, grid, kThreads, kDynSmem, st, m[0], m[1], m[2], m[3], m[4],
                 m[5], p);
  }
  if (e != cudaSuccess) {
    set_error("rows_ffn_fp8_kernel launch: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return check_launch("rows_ffn_fp8_kernel");
}

}  // namespace moe
