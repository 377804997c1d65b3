// The 4-bit expert FFN forward for few rows an expert (a batch of single tokens).
//
// With a handful of rows an expert the products are a stream of weights, bound by HBM
// however few the rows are. As in rows_fp8.cu the weights are the M operand and 32 rows
// the N operand:
//   D[128 weight rows, 32 rows of x] += W[128, 256 of K] X[32, 256 of K]^T
// with 256 K values to a stage (128 bytes), two M tiles a stage.
//
// One persistent launch, one CTA per SM, both products' tiles claimed in order from a
// counter; a tile of the second waits for its expert's tiles of the first:
//   FC1 tile: (expert, 128 columns of h, 32 rows): 128 gate and 128 up rows of W1
//   FC2 tile: (expert, 256 columns of o, 32 rows): two times 128 rows of W2
//   warp 0      producer: a stage's weights and rows by TMA, their scales beside them as
//               contiguous copies, on the same barrier
//   warp 1      TMEM allocator + MMA issuer
//   warp 2      claims tiles
//   warps 4..7  epilogue: thread = weight row (column of h or o), registers = rows; then, by
//               way of shared memory, thread = a block (32 columns) of a row of h
//   warps 8..11 a stage's scales from shared memory into TMEM, ahead of its MMAs
//
// 64 tokens of the 128-expert layer (H 2048, F 768, top 8, skewed): 50.7 us for the 304 MB that
// it reads, 0.9 of a copy's rate; 6.1 TB/s while its CTAs are active, the launches before and the
// last tiles are the rest. An MMA takes the tensor pipe some 130 clocks however small its N (the
// 8-bit ones 55), so a stage's eight are 1040 clocks, and its 37 KB arrive in 1700: with 32
// rows an expert the call still takes 59 us. One token: 12.5 us for 20 MB, a chain of latencies
// (ns): set-up and tables 1200, claim 800, first stage 800, K loop 3700 (20 MB at 5.6 TB/s, the
// second product's weights on their way beside the first's), epilogue 400, count 700, seen
// by the second product 300, its rows and scales 900, its 3 stages 1450, o and end 1000. Tiles
// half as wide on twice the SMs were slower there (17.6 us: both products' tiles no longer
// fit the SMs at once, so that some weights are asked for late); a second set of scale
// warps made no difference.
#include <algorithm>
#include <atomic>

#include "fp4_mma.cuh"

namespace moe {

using namespace fp8;
using namespace fp4;

namespace {

constexpr int kFc1 = 0, kFc2 = 1;
constexpr int NT = 32;                        // rows of x in a tile
constexpr int BK = kFp4Group;                 // K values of a stage
constexpr int kWBytes = 128 * BK / 2;         // one M tile's weights of a stage
constexpr int kXAt = 2 * kWBytes;
constexpr int kSwAt = kXAt + NT * BK / 2;     // scales: two M tiles' ...
constexpr int kSwBytes = 128 * 8;
constexpr int kSxAt = kSwAt + 2 * kSwBytes;   // ... and the rows', from an even row on
constexpr int kStageBytes = (kSxAt + (NT + 2) * 8 + 1023) / 1024 * 1024;
constexpr int kStages = 5;
constexpr int kThreads = 384;
constexpr int kMaxE = 256;
constexpr int kAccCols = 2 * NT;              // TMEM columns of one accumulator (two M tiles)
constexpr int kTmemScales = 2 * kAccCols;     // buffers of 24: for each half of a stage two M tiles, the rows
constexpr int kSf = 4, kSfCols = 24;
constexpr int kTmemCols = 256;
constexpr int kSmallBox = 8;                  // rows of the small TMA box
static_assert(kTmemScales + kSf * kSfCols <= kTmemCols, "TMEM columns");
static_assert(kFp4FewRows * kMaxE < 65536, "16-bit offsets");
constexpr size_t kDynSmem = (size_t)kStages * kStageBytes + 1024;

// The tile's h between the epilogue's two views: a thread writes its column of every row,
// then takes a block (32 columns) of one row. Blocks 36 floats apart and rows 144: neither
// the writes nor the 16-byte reads of 8 lanes (two rows' four blocks) meet in a bank.
constexpr int kHBlock = 36, kHRow = 4 * kHBlock;
constexpr int kORow = 264;  // and of a tile of o, bf16
static_assert(kORow % 8 == 0 && NT * kORow * 2 <= NT * kHRow * 4, "o's rows in h's room");

struct RowsParams {
  int E, H, F;
  long long N;
  const int32_t* off;
  const uint8_t* xs;
  Fp4Weights w;
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
  uint64_t claim_full[2], claim_empty[2], claim;  // claimed tiles
  int claimed[2];
  uint32_t tmem_base;
  int abort;
  int rtile[kMaxE + 1];           // first row tile of each expert
  uint16_t off[kMaxE + 1];
  alignas(16) float h[NT * kHRow];  // read 16 bytes at a time
};
static_assert(kHBlock % 4 == 0 && kHRow % 4 == 0, "16-byte reads of a row's blocks");

template <int G>
__device__ __forceinline__ int kvalues(const RowsParams& p) { return G == kFc1 ? p.H : p.F; }
template <int G>
__device__ __forceinline__ int kstages(const RowsParams& p) { return (kvalues<G>(p) + BK - 1) / BK; }
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

__device__ __forceinline__ void give_up(SmemCtl& c, int* status, int where) {
  c.abort = 1;
  atomicExch(status + ST_TIMEOUT, where);
}

__device__ __forceinline__ bool wait_expert(SmemCtl& c, const RowsParams& p, int e) {
  const int target = (c.rtile[e + 1] - c.rtile[e]) * ncols<kFc1>(p);
  if (ld_acquire(p.dep + e) < target) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ld_acquire(p.dep + e) < target) {
      if (*(volatile int*)&c.abort || ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
        give_up(c, p.status, 40);
        return false;
      }
    }
  }
  return true;
}

// The n-th tile claimed for this CTA (at or past the total: none is left; -1: gave up), for the
// 10 warps that read it: producer, MMA issuer, scales, epilogue. A reader's arrival
// (release) comes after its read, the slot is overwritten after all of them.
constexpr int kReaders = 10;
__device__ __forceinline__ int claimed_tile(SmemCtl& c, uint32_t n, int* status, bool warp) {
  bool ok = ptx::mbar_wait(&c.claim_full[n & 1], (n >> 1) & 1, &c.abort, kWaitLimitNs);
  if (warp) ok = __all_sync(0xffffffffu, ok);
  if (!ok) {
    give_up(c, status, 41);
    return -1;
  }
  const int i = *(volatile int*)&c.claimed[n & 1];
  if (warp) __syncwarp();
  if (!warp || (threadIdx.x & 31) == 0) ptx::mbar_arrive(&c.claim_empty[n & 1]);
  return i;
}
__device__ __forceinline__ void publish(SmemCtl& c, uint32_t n, int i) {
  *(volatile int*)&c.claimed[n & 1] = i;
  ptx::mbar_arrive(&c.claim_full[n & 1]);
}
// The tiles after the first, which has been published while the tables were made.
__device__ __forceinline__ void claim_tiles(SmemCtl& c, const RowsParams& p, int first, int total) {
  for (uint32_t n = 1; first < total; ++n) {
    if ((n == 1 && !ptx::mbar_wait(&c.claim, 0, &c.abort, kWaitLimitNs)) ||
        !ptx::mbar_wait(&c.claim_empty[n & 1], ((n >> 1) & 1) ^ 1, &c.abort, kWaitLimitNs)) {
      give_up(c, p.status, 42);
      return;
    }
    const int i = atomicAdd(p.tile, 1);
    publish(c, n, i);
    if (i >= total) return;
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
  const int nk = kstages<G>(p), mt = mtiles<G>(p, t);
  const int w0 = G == kFc1 ? t.e * 2 * p.F + t.n0 : t.e * p.H + t.n0;
  const int w1 = w0 + (G == kFc1 ? p.F : 128);
  const bool small = t.rows <= NT / 2;
  const int xrows = small ? (t.rows + kSmallBox - 1) / kSmallBox * kSmallBox : NT;
  // scales: of a matrix's rows in this tile (the edge may cut one M tile in half) ...
  const int R = G == kFc1 ? p.F : p.H;
  const uint32_t sb0 = min(128, R - t.n0) * 8;
  const uint32_t sb1 = G == kFc1 ? sb0 : mt == 2 ? min(128, R - t.n0 - 128) * 8 : 0;
  const uint8_t* ws = G == kFc1 ? p.w.w1s : p.w.w2s;
  const uint8_t* s0 = ws + ((size_t)(G == kFc1 ? 2 * t.e : t.e) * nk * R + t.n0) * 8;
  const uint8_t* s1 = s0 + (G == kFc1 ? (size_t)nk * R : 128) * 8;
  // ... and of the rows of x, from an even one on
  const long long np = scale_rows(p.N), sr = t.row & ~1ll;
  const uint32_t sbx = (((int)(t.row & 1) + t.rows + 1) & ~1) * 8;
  const uint8_t* sx = (G == kFc1 ? p.xs : p.hs) + sr * 8;
  const uint32_t bytes = mt * kWBytes + xrows * (BK / 2) + sb0 + sb1 + sbx;
  bool ready = G == kFc1, ok = true;
  for (int kt = 0; kt < nk && ok; ++kt) {
    if (!ptx::mbar_wait(&c.empty[stage], phase ^ 1, &c.abort, kWaitLimitNs)) {
      give_up(c, p.status, 43);
      return false;
    }
    if (kt == nk / 4) ptx::mbar_arrive(&c.claim);
    uint8_t* s = smem + stage * kStageBytes;
    uint64_t* bar = &c.full[stage];
    const int k0 = kt * (BK / 2);  // bytes
    ptx::mbar_arrive_expect_tx(bar, bytes);
    ptx::tma_load_2d(s, tmW, bar, k0, w0);
    if (mt == 2) ptx::tma_load_2d(s + kWBytes, tmW, bar, k0, w1);
    bulk_load(s + kSwAt, s0 + (size_t)kt * R * 8, sb0, bar);
    if (mt == 2) bulk_load(s + kSwAt + kSwBytes, s1 + (size_t)kt * R * 8, sb1, bar);
    if (!ready) {  // the weights do not wait for the first product, its rows do
      // (after an abort the stage is still loaded whole: drain_loads waits for stages)
      ok = wait_expert(c, p, t.e);
      asm volatile("fence.proxy.async.global;" ::: "memory");
      ready = true;
    }
    if (!small) ptx::tma_load_2d(s + kXAt, tmX, bar, k0, (int)t.row);
    else
      for (int r = 0; r < xrows; r += kSmallBox)
        ptx::tma_load_2d(s + kXAt + r * (BK / 2), tmS, bar, k0, (int)t.row + r);
    bulk_load(s + kSxAt, sx + (size_t)kt * np * 8, sbx, bar);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
  return ok;
}

__device__ __forceinline__ void arrive(uint64_t* bar, int lane) {
  ptx::tc_fence_before();
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(bar);
}

struct ScaleState {
  int stage = 0;
  uint32_t phase = 0, group = 0;
};
// A cell (lane r % 32, column r / 32) holds four scales of a row: two words a row and stage.
template <int G>
__device__ __forceinline__ bool scales_tile(SmemCtl& c, const uint8_t* smem, const RowsParams& p,
                                            const Tile& t, uint32_t tmem, ScaleState& m, int quarter,
                                            int lane) {
  const int nk = kstages<G>(p);
  const int odd = (int)(t.row & 1);
  for (int kt = 0; kt < nk; ++kt, ++m.group) {
    const int buf = m.group % kSf;
    bool got = ptx::mbar_wait(&c.full[m.stage], m.phase, &c.abort, kWaitLimitNs);
    const uint8_t* s = smem + m.stage * kStageBytes;
    uint32_t w[2][8];  // [half of the stage][two M tiles x 4]
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint2 v = *reinterpret_cast<const uint2*>(s + kSwAt + (i * 32 + lane) * 8);
      w[0][i] = v.x;
      w[1][i] = v.y;
    }
    const uint2 x = *reinterpret_cast<const uint2*>(s + kSxAt + (odd + lane) * 8);
    got = got && ptx::mbar_wait(&c.sf_empty[buf], ((m.group / kSf) & 1) ^ 1, &c.abort, kWaitLimitNs);
    if (!__all_sync(0xffffffffu, got)) {
      if (lane == 0) give_up(c, p.status, 44);
      return false;
    }
    ptx::tc_fence_after();
    const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + kTmemScales + buf * kSfCols;
    const uint32_t wx[8] = {x.x, x.x, x.x, x.x, x.y, x.y, x.y, x.y};  // (32 rows: the first column is read)
    tmem_st_x8(at, w[0]);
    tmem_st_x8(at + 8, w[1]);
    tmem_st_x8(at + 16, wx);
    tmem_st_wait();
    arrive(&c.sf_full[buf], lane);
    if (++m.stage == kStages) {
      m.stage = 0;
      m.phase ^= 1;
    }
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
  constexpr uint32_t idesc = idesc_mxf4(128, NT);
  const uint64_t desc0 = ptx::sdesc_sw128(0, 16, 1024);
  const int K = kvalues<G>(p), nk = kstages<G>(p), mt = mtiles<G>(p, t);
  const int acc = m.tiles & 1;
  const bool got =
      ptx::mbar_wait(&c.tmem_empty[acc], ((m.tiles >> 1) & 1) ^ 1, &c.abort, kWaitLimitNs);
  if (!__all_sync(0xffffffffu, got)) {
    give_up(c, p.status, 45);
    return false;
  }
  ptx::tc_fence_after();
  const uint32_t d = tmem + acc * kAccCols;
  int where = 0;
  if (elect_one()) {  // one lane waits and issues for the whole tile
    int stage = m.stage;
    uint32_t phase = m.phase, group = m.group;
    for (int kt = 0; kt < nk; ++kt, ++group) {
      const int buf = group % kSf;
      if (!ptx::mbar_wait(&c.full[stage], phase, &c.abort, kWaitLimitNs)) {
        where = 46;
        break;
      }
      if (!ptx::mbar_wait(&c.sf_full[buf], (group / kSf) & 1, &c.abort, kWaitLimitNs)) {
        where = 47;
        break;
      }
      ptx::tc_fence_after();
      const uint32_t sf = tmem + kTmemScales + buf * kSfCols;
      const uint64_t a0 = desc0 | ((smem + stage * kStageBytes) >> 4);
      const uint64_t x = a0 + (kXAt >> 4);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {  // 64 K values each; past the edge there are none
        if (kt * BK + kk * 64 >= K) break;
        const uint32_t id = idesc | (kk & 1 ? kUpperPair : 0), on = (kt | kk) != 0;
        const uint32_t sw = sf + 8 * (kk >> 1), sx = sf + 16 + 4 * (kk >> 1);
        umma_mxf4(d, a0 + kk * 2, x + kk * 2, id, sw, sx, on);
        if (mt == 2) umma_mxf4(d + NT, a0 + (kWBytes >> 4) + kk * 2, x + kk * 2, id, sw + 4, sx, on);
      }
      ptx::umma_commit(&c.empty[stage]);
      ptx::umma_commit(&c.sf_empty[buf]);
      if (kt == nk - 1) ptx::umma_commit(&c.tmem_full[acc]);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
  where = __reduce_max_sync(0xffffffffu, where);
  if (where) {
    give_up(c, p.status, where);
    return false;
  }
  m.group += nk;
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
  if (!__all_sync(0xffffffffu, got) && lane == 0) give_up(c, p.status, 48);
  ptx::tc_fence_after();
  const uint32_t tbase = tmem + acc * kAccCols + ((uint32_t)(q * 32) << 16);
  if (G == kFc1) {
    const int f = t.n0 + col;
    const bool ok = f < p.F;  // uniform in the warp: F is a multiple of 64
    for (int r0 = 0; r0 < t.rows && ok; r0 += 8) {
      uint32_t g[8], u[8];
      tmem_ld_x8(tbase + r0, g);
      tmem_ld_x8(tbase + NT + r0, u);
      tmem_ld_wait_x8(g);
      tmem_ld_wait_x8(u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (r0 + j >= t.rows) break;
        const float gf = __uint_as_float(g[j]), uf = __uint_as_float(u[j]);
        const float hf = gf * sigmoid_f(gf) * uf;
        const size_t row = (size_t)(t.row + r0 + j);
        if (p.a) {
          bf16* a = p.a + row * (2 * p.F) + f;
          a[0] = __float2bfloat16_rn(gf);
          a[p.F] = __float2bfloat16_rn(uf);
        }
        if (p.h) p.h[row * p.F + f] = __float2bfloat16_rn(hf);
        c.h[(r0 + j) * kHRow + q * kHBlock + lane] = hf;
      }
    }
    arrive(&c.tmem_empty[acc], lane);
    epilogue_sync();  // the tile's h is in shared memory
    const int r = col >> 2, fb = t.n0 + 32 * (col & 3);  // this thread's row and block
    if (r < t.rows && fb < p.F) {
      const float4* hp = reinterpret_cast<const float4*>(&c.h[r * kHRow + (col & 3) * kHBlock]);
      float v[32], mx = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = hp[i];
        v[4 * i] = x.x;
        v[4 * i + 1] = x.y;
        v[4 * i + 2] = x.z;
        v[4 * i + 3] = x.w;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) mx = absmax_nan(mx, v[i]);
      const uint32_t b = fp4_scale_byte(__float_as_uint(mx));
      const float inv = fp4_inv_scale(b);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= inv;
      const size_t row = (size_t)(t.row + r);
      const int blk = fb >> 5;
      *reinterpret_cast<uint4*>(p.hq + (row * p.F + fb) / 2) =
          make_uint4(fp4x8(v), fp4x8(v + 8), fp4x8(v + 16), fp4x8(v + 24));
      p.hs[((size_t)(blk >> 3) * scale_rows(p.N) + row) * 8 + (blk & 7)] = (uint8_t)b;
    }
    epilogue_sync();  // every store issued, and c.h free again
    if (col == 0) {
      __threadfence();
      atomicAdd(p.dep + t.e, 1);
    }
  } else {
    // by way of shared memory too, so that rows leave 16 bytes a thread
    const int mt = mtiles<G>(p, t);
    bf16* buf = reinterpret_cast<bf16*>(c.h);
    for (int m = 0; m < mt; ++m) {
      for (int r0 = 0; r0 < t.rows; r0 += 8) {
        uint32_t v[8];
        tmem_ld_x8(tbase + NT * m + r0, v);
        tmem_ld_wait_x8(v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (r0 + j < t.rows)
            buf[(r0 + j) * kORow + 128 * m + col] = __float2bfloat16_rn(__uint_as_float(v[j]));
      }
    }
    arrive(&c.tmem_empty[acc], lane);
    epilogue_sync();
    for (int i = col; i < t.rows * 32; i += 128) {
      const int r = i >> 5, x = (i & 31) * 8;
      if (t.n0 + x < p.H)
        *reinterpret_cast<uint4*>(p.o + (size_t)(t.row + r) * p.H + t.n0 + x) =
            *reinterpret_cast<const uint4*>(buf + r * kORow + x);
    }
    epilogue_sync();  // c.h is free again
  }
  ++tiles;
  return *(volatile int*)&c.abort == 0;
}

__global__ void __launch_bounds__(kThreads, 1)
    rows_ffn_fp4_kernel(const __grid_constant__ CUtensorMap tmW1,
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
      ptx::mbar_init(&ctl.claim_full[b], 1);
      ptx::mbar_init(&ctl.claim_empty[b], kReaders);
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
  __syncthreads();  // warp 2 arrives on claim_full below: initialised for every warp (beside the launch before)
  pdl_wait();
  int first = 0;  // the first tile, claimed while the tables are made
  if (warp == 2 && lane == 0) {
    first = atomicAdd(p.tile, 1);
    publish(ctl, 0, first);
  }
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
      if (e < p.E) ctl.rtile[e] = incl - sum + n[k];
    }
    if (lane == 31) ctl.rtile[p.E] = incl;
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
        const int i = claimed_tile(ctl, n, p.status, false);
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
      const int i = claimed_tile(ctl, n, p.status, true);
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
    ScaleState m;
    for (uint32_t n = 0; ok; ++n) {
      const int i = claimed_tile(ctl, n, p.status, true);
      ok = i >= 0;
      if (!ok || i >= total) break;
      ok = i < total1 ? scales_tile<kFc1>(ctl, smem, p, tile1(i), tmem, m, warp - 8, lane)
                      : scales_tile<kFc2>(ctl, smem, p, tile2(i), tmem, m, warp - 8, lane);
    }
  } else if (warp >= 4) {
    uint32_t tiles = 0;
    for (uint32_t n = 0;; ++n) {
      const int i = claimed_tile(ctl, n, p.status, true);
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
  e = cudaFuncSetAttribute(rows_ffn_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kDynSmem);
  if (e == cudaSuccess) ready.fetch_or(bit);
  return e;
}

}  // namespace

moe_status_t launch_ffn_rows_fp4(const moe_layer_desc_t& d, const uint8_t* xq, const uint8_t* xs,
                                 const int32_t* off, const Fp4Weights& w, bf16* a, bf16* h,
                                 uint8_t* hq, uint8_t* hs, bf16* o, int* status, int* dep,
                                 cudaStream_t st, bool counters_zeroed) {
  const long long N = (long long)d.T * d.k;
  CUtensorMap m[6];
  if (!make_map(&m[0], w.w1q, 2, d.H / 2, 2ll * d.E * d.F, 1, 128, 1) ||
      !make_map(&m[1], xq, 2, d.H / 2, N, 1, NT, 1) ||
      !make_map(&m[2], xq, 2, d.H / 2, N, 1, kSmallBox, 1) ||
      !make_map(&m[3], w.w2q, 2, d.F / 2, (long long)d.E * d.H, 1, 128, 1) ||
      !make_map(&m[4], hq, 2, d.F / 2, N, 1, NT, 1) ||
      !make_map(&m[5], hq, 2, d.F / 2, N, 1, kSmallBox, 1))
    return MOE_ERR_CUDA;
  const RowsParams p = {d.E, d.H, d.F, N, off, xs, w, a, h, hq, hs, o, status, dep,
                        tile_counter(status)};
  cudaError_t e = set_up();
  if (e == cudaSuccess && !counters_zeroed) e = launch_zero_counters(dep, d.E, p.tile, st);
  // one CTA per SM, fewer when there cannot be as many tiles
  const long long rows = N / NT + std::min<long long>(N, d.E);
  const long long tiles = rows * (ceil_div(d.F, 128) + ceil_div(d.H, 256));
  const int grid = (int)std::min<long long>(device_sm_count(), tiles);
  if (e == cudaSuccess) {
    LaunchScope _ls(K_FP4_ROWS_FFN, st);
    e = launch_k(rows_ffn_fp4_kernel, grid, kThreads, kDynSmem, st, m[0], m[1], m[2], m[3], m[4],
                 m[5], p);
  }
  if (e != cudaSuccess) {
    set_error("rows_ffn_fp4_kernel launch: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return check_launch("rows_ffn_fp4_kernel");
}

}  // namespace moe
