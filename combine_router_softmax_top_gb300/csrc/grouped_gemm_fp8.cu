// Grouped expert GEMMs on e4m3 operands with block scales (see fp8.cuh): the
// SwiGLU expert FFN forward (FC1 -> FC2) and its activation gradient (FC2
// dgrad -> FC1 dgrad).
//
//   D[r, c] = sum over 128-wide K blocks b of
//             2^(sa[r,b]-127) 2^(sb[c,b]-127) sum_{i in b} A[r,i] B[c,i]
//
// The tensor cores apply both scales themselves (tcgen05.mma kind::mxf8f6f4,
// one scale per 32 K values: the four K = 32 steps of a block use the same
// bytes), so the fp32 accumulator needs no pass over it between blocks.
//
// One persistent launch per chain, a CTA pair (tcgen05 cta_group::2, M = 256,
// N = 256) per two SMs, warp-specialised:
//   warp 0      TMA producer of the operand ring: this CTA's 128 rows of A and its
//               half of B, 128 bytes of K, 32 KB a stage, 6 stages
//   warp 1      TMEM allocator + (even CTA) single-thread MMA issuer for the pair
//   warp 2      counts first-GEMM tiles for their experts (below)
//   warp 3      gradient: loads the saved pre-activations for the epilogue
//   warps 12..15 scales: each writes the scale bytes of four K blocks (the four
//               bytes of a TMEM cell) into its 32 TMEM lanes (tcgen05.st), ahead of
//               the MMA issuer. Copying them from shared memory (tcgen05.cp) in the
//               MMA issuer's order instead drains the tensor pipe: 647 clocks a
//               stage of four MMAs against 512 without.
//   warps 4..11 epilogue: TMEM -> registers -> SwiGLU (or its gradient),
//               rounding, block maxima, e4m3 -> global; two warps per TMEM lane
//               quarter, each owning 64 of every 128 columns
// Tiles are claimed in order from a counter, the first GEMM's before the second's
// (the odd CTA's warp 1 claims for the pair, up to two ahead of what its slowest
// warp works on; the second once the first is under way, or with few tiles half of
// the pairs would take two each). A tile of the second GEMM starts once every tile
// of its expert in the first has been stored (per-expert counters): those have been
// claimed before it by pairs that are running, so the wait ends however many pairs
// are resident beside other work. (Tiles dealt out by CTA number would need every
// CTA resident, and are little faster: 163 against 166 us for the forward below.)
//
// TMEM: two 256-column accumulators and four buffers of 12 scale columns do not
// fit 512 columns, so the accumulators share 64: columns 0..255 and 192..447.
// The epilogue reads the shared columns first and releases them (ovl), so the
// next tile's MMAs start while it works on the rest. (Two scale buffers would
// need only 32 shared columns, but a buffer's turn-around through both CTAs -
// MMAs done, scale warps, MMA issuer - takes 2000 clocks and more, as long as
// the four K blocks of the other buffer: the K loop ran at 595 clocks a block
// instead of 512.)
//
// What bounds it, 128 experts of H 2048, F 768 at 4096 tokens, top 8, balanced: the
// forward that keeps a and h moves 956 MB in 160 to 169 us (5.7 to 6.0 TB/s, the copy
// rate being 6.8), the gradient 1007 MB in 180 us. Its second product lands 64 KB of
// operands in a pair for each 256 x 256 x 128 step, at the 9 to 10 TB/s that L2 gives all
// SMs together. Skewed loads (95 to 4096 rows an expert) cost the gradient 234 to 248
// us: half as many 256-row tiles again, their last rows empty, and a first product at
// the pace of its epilogue (22000 clocks a tile, the K loop 14000). 64 experts of F 1408 at
// 8192 tokens, nothing kept: 1134 GFLOP in 410 us for the first launches at 2070 MHz (2.8
// PFLOP/s, tensor pipe 73% active); after a second of them 1365 W, the power cap active and
// 1560 MHz, 477 us (484 to 500 from box to box).
//
// Ragged groups as in the bf16 GEMMs: expert e owns rows off[e]..off[e+1]-1; a
// tile's rows past the expert's end are computed on whatever TMA loaded and
// not stored (rows of A do not mix). Columns past a matrix edge likewise. K past
// an edge must add nothing: maps whose K dimension ends with the expert (or the
// gate or up half) zero-fill it.
#include <algorithm>
#include <atomic>

#include "fp8_mma.cuh"

namespace moe {

using namespace fp8;

namespace {

enum Fp8Mode {
  FC1_FWD = 0,   // a, h, hq = SwiGLU(xq @ W1q^T)
  FC2_FWD = 1,   // o = hq @ W2q^T
  FC2_DGRAD = 2, // da, daq = SwiGLU'(dq @ W2q, a)
  FC1_DGRAD = 3  // dx_perm = daq @ W1q
};

constexpr int BM = 128, BN = 256, BK = 128;   // BM: rows of one CTA of the pair
constexpr int kABytes = BM * BK, kBBytes = BN / 2 * BK;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kAuxBytes = 4 * 8192;           // one step: gate and up, 128 rows x 2 x 32 columns
constexpr int kEpiBytes = 8 * 2048;           // a 32 x 32 bf16 box for each epilogue warp
constexpr int kABoxRows = 16;                 // tiles of 64 rows or fewer load boxes of 16
constexpr int kTmemCols = 512;
constexpr int kAccStep = 192;                 // second accumulator's first column
constexpr int kTmemScales = 448;              // buffers of 4 columns for A, 8 for B
constexpr int kSf = 4;                        // scale buffers
constexpr int kThreads = 512;
// registers a thread: 128 at launch; the epilogue's two warpgroups take what the
// control and scale warpgroups give up (2 * 72 + 2 * 184 = 4 * 128). At 128 the forward
// chain is compiled with two words spilled (8 bytes stored, 56 loaded), the gradient's
// with none.
constexpr int kRegsControl = 72, kRegsEpilogue = 184;
constexpr int kMaxE = 256;

// Launch-wide constants. The gradient's first GEMM gives two of the six operand
// stages up for two steps of the saved pre-activations (asking L2 for them ahead
// instead was slower: 204 against 196 us, and 184 so); its second GEMM gets them
// back as a ring of its own (kSecond: its first barrier).
template <int M1>
struct Chain {
  static constexpr bool kAux = M1 == 2;
  static constexpr int kStages1 = kAux ? 4 : 6, kStages2 = 6;
  static constexpr int kSecond = kAux ? kStages1 : 0;
  static constexpr int kBars = kSecond + kStages2;
  static constexpr int kAuxAt = kStages1 * kStageBytes;
  static constexpr int kEpiAt = kStages2 * kStageBytes;
  static constexpr size_t kDynSmem = kEpiAt + kEpiBytes + 1024;
  static_assert(!kAux || kAuxAt + 2 * kAuxBytes <= kEpiAt, "the pre-activations' room");
};
constexpr int kMaxBars = 10;
constexpr int kHalf = 8;  // slots of half a mailbox (below)

struct Maps {
  CUtensorMap a1, s1, b1, a2, s2, b2;  // operands: A, A in small boxes, B of both GEMMs
  CUtensorMap o1, o2, o3;              // a | da, h | daq, o | dx_perm
  CUtensorMap aux;                     // the saved pre-activation
};

struct KParams {
  int E, H, F;
  long long N;
  const int32_t* off;
  const uint8_t* sa;  // scale words of the A rows
  const uint8_t* sb;  // scale bytes of the weight blocks
  bf16* out0;         // a | o | da | dx_perm (a and da may be NULL)
  bf16* out1;         // h (may be NULL)
  uint8_t* q;         // hq | daq
  uint8_t* s;         // hs | das
  int* status;
  int* dep;           // per-expert count of first-GEMM tiles stored, by CTA
  int* tile;          // tiles claimed
  int halves;         // FC2 dgrad: 128-column halves that a tile's epilogue stores (set on the device)
};

template <int MODE>
struct Mode {
  static constexpr bool kBMn = MODE == FC2_DGRAD || MODE == FC1_DGRAD;  // N contiguous in B
  static constexpr bool kFirst = MODE == FC1_FWD || MODE == FC2_DGRAD;
  __device__ static int kblocks(const KParams& p) {
    const int nh = (p.H + 127) / 128, nf = (p.F + 127) / 128;
    return MODE == FC1_FWD || MODE == FC2_DGRAD ? nh : MODE == FC2_FWD ? nf : 2 * nf;
  }
  __device__ static int ntiles(const KParams& p) {
    return MODE == FC1_FWD     ? (p.F + 127) / 128
           : MODE == FC2_DGRAD ? (p.F + 128 * p.halves - 1) / (128 * p.halves)
                               : (p.H + BN - 1) / BN;
  }
};

struct Tile {
  int e, m0, n0, rows, row0;  // m0: first row of this CTA's 128 in the expert; rows <= 0: none
  int rows_odd;               // even CTA: rows left for the odd one
};

struct SmemCtl {
  uint64_t full[kMaxBars], empty[kMaxBars];
  uint64_t aux_full[2], aux_empty[2], aux_done;
  uint64_t paired[4];  // both warps of a quarter have left their block maxima
  uint64_t sf_full[kSf], sf_empty[kSf];
  uint64_t tmem_full[2], tmem_empty[2], ovl, drain;
  uint64_t mail_full[2 * kHalf], mail_empty[2];  // claimed tiles, from the odd CTA to both producers
  uint64_t sched_full[2], sched_empty[2];  // and from the producer to the others of its CTA
  uint64_t claim;                          // odd CTA: time to claim the second tile
  int mail[2 * kHalf], sched[2];
  uint64_t stored[2], counted[2];  // a first-GEMM tile's stores issued; counted for its expert
  uint32_t tmem_base;
  int abort;
  int tstart[2][kMaxE + 1];  // tile prefixes of the two GEMMs
  int off[kMaxE + 1];
  uint32_t amax[2][8][32];   // block maxima handed between the two warps of a quarter
};

template <int MODE>
__device__ __forceinline__ Tile tile_at(const KParams& p, const SmemCtl& c, int tile, int& cursor,
                                        uint32_t rank) {
  const int* tstart = c.tstart[Mode<MODE>::kFirst ? 0 : 1];
  while (tstart[cursor + 1] <= tile) ++cursor;
  Tile t;
  t.e = cursor;
  t.row0 = c.off[cursor];
  const int cnt = c.off[cursor + 1] - t.row0;
  const int local = tile - tstart[cursor];
  const int mt = (cnt + 2 * BM - 1) / (2 * BM);
  t.m0 = (local % mt) * 2 * BM + (int)rank * BM;
  t.n0 = (local / mt) * (MODE == FC1_FWD ? 128 : MODE == FC2_DGRAD ? 128 * p.halves : BN);
  t.rows = min(BM, cnt - t.m0);
  t.rows_odd = rank == 0 ? cnt - t.m0 - BM : 0;
  return t;
}

__device__ __forceinline__ void flag_timeout(SmemCtl& c, int* status, int where) {
  c.abort = 1;
  atomicExch(status + ST_TIMEOUT, where);
}

// ---------------------------------------------------------------- tcgen05, block-scaled
// The pair's MMA: A rows, the scales of A and D are each CTA's own, B's N rows
// are half in each CTA, B's scales whole in both.
__device__ __forceinline__ void umma_mxf8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X "
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
template <int REGS>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int32_t c0, int32_t c1,
                                                 int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// ---------------------------------------------------------------- stores
// 32 rows (thread i holds row i) x 32 bf16 columns (16 packed words). Whole boxes
// leave through this warp's 2 KB buffer as one TMA store, in whole lines; a box
// that ends with the expert's rows is written by its threads, a 32-byte sector at
// a time (256-bit stores): slower, as every sector is a request of its own (the
// gradient's epilogue takes 31000 clocks a tile that way, 18000 without stores).
__device__ __forceinline__ void st_sector(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
struct Out {       // one warp's slab of an output
  uint4* buf;      // its shared buffer
  int lane, rows;  // valid rows of the slab
};
__device__ __forceinline__ void store_box(const Out& o, const CUtensorMap* map, const uint32_t* w,
                                          bf16* base, size_t row, int ld, int x) {
  if (o.rows >= 32) {
    if (o.lane == 0) ptx::bulk_wait_group_read0();  // the last box has left the buffer
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q)  // 64-byte swizzle
      o.buf[o.lane * 4 + (q ^ ((o.lane >> 1) & 3))] =
          make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (o.lane == 0) {
      ptx::tma_store_2d(map, o.buf, x, (int)row);
      ptx::bulk_commit_group();
    }
  } else if (o.lane < o.rows) {
    bf16* p = base + (row + o.lane) * (size_t)ld + x;
    st_sector(p, w);
    st_sector(p + 16, w + 8);
  }
}
// 16 bf16 columns (8 packed words) rounded to e4m3
__device__ __forceinline__ uint4 fp8x16(const uint32_t* w, uint32_t inv) {
  return make_uint4(fp8x4_of_bf16(w[0], w[1], inv), fp8x4_of_bf16(w[2], w[3], inv),
                    fp8x4_of_bf16(w[4], w[5], inv), fp8x4_of_bf16(w[6], w[7], inv));
}
// 32 bf16 columns (16 packed words) rounded to e4m3
__device__ __forceinline__ void store_fp8(uint8_t* p, const uint32_t* w, uint32_t inv) {
  uint32_t v[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = fp8x4_of_bf16(w[2 * q], w[2 * q + 1], inv);
  st_sector(p, v);
}

// ================================================================ dependences
// A second-GEMM tile of expert e: wait (bounded) until the expert's first-GEMM
// tiles have all stored their output.
__device__ __forceinline__ bool wait_expert(SmemCtl& c, const KParams& p, int e) {
  const int target = 2 * (c.tstart[0][e + 1] - c.tstart[0][e]);  // both CTAs of the pair
  if (ld_acquire(p.dep + e) < target) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ld_acquire(p.dep + e) < target) {
      __nanosleep(64);
      if (*(volatile int*)&c.abort || ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
        flag_timeout(c, p.status, 10);
        return false;
      }
    }
  }
  return true;
}

// ================================================================ tiles
// The odd CTA claims for the pair and leaves the tile in a mailbox in each CTA; that
// CTA's producer, which needs it first, takes it out and hands it to the others of its
// CTA. So one thread of the even CTA, with no stores in flight, releases what it read
// to the odd one, and as a release at cluster scope takes some 3000 clocks with stores
// in flight on the SM, it does so once in kHalf tiles: the mailbox has two halves of as
// many slots. (Once a tile: the balanced forward 180 us against 160 so, the gradient 191
// against 180, prefill 515 against 499, in turn on one GPU; by every warp of the pair, as
// slow.)
//
// What reads the tiles of a CTA beside the producer: counting warp, scale and epilogue
// warps, the MMA issuer in the even one (and the gradient's aux loader).
__device__ __forceinline__ int readers(uint32_t rank, bool aux) {
  return 1 + 4 + 8 + (rank == 0) + aux;
}
// Relaxed: for accesses to TMEM alone, which the tcgen05 fences on both sides order.
__device__ __forceinline__ void arrive_remote(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster)
               : "memory");
}
// The producer: takes the n-th tile claimed for this pair (past the last: none is left; -1:
// gave up) out of the mailbox and hands it on.
__device__ __forceinline__ int take_tile(SmemCtl& c, uint32_t n, int* status) {
  const int slot = n % (2 * kHalf);
  const uint32_t round = n / (2 * kHalf);
  if (!mbar_wait_cluster(&c.mail_full[slot], round & 1, &c.abort)) {
    flag_timeout(c, status, 14);
    return -1;
  }
  const int i = *(volatile int*)&c.mail[slot];
  if (slot % kHalf == kHalf - 1)  // the half has been read
    ptx::mbar_arrive_cluster(ptx::mapa_shared(&c.mail_empty[slot / kHalf], 1));
  if (!ptx::mbar_wait(&c.sched_empty[n & 1], ((n >> 1) & 1) ^ 1, &c.abort, kWaitLimitNs)) {
    flag_timeout(c, status, 18);
    return -1;
  }
  *(volatile int*)&c.sched[n & 1] = i;
  ptx::mbar_arrive(&c.sched_full[n & 1]);
  return i;
}
// The others: the n-th tile. Every lane of a warp that passes warp = true calls it together.
__device__ __forceinline__ int next_tile(SmemCtl& c, uint32_t n, int* status, bool warp) {
  bool ok = ptx::mbar_wait(&c.sched_full[n & 1], (n >> 1) & 1, &c.abort, kWaitLimitNs);
  if (warp) ok = __all_sync(0xffffffffu, ok);
  if (!ok) {
    flag_timeout(c, status, 19);
    return -1;
  }
  const int i = *(volatile int*)&c.sched[n & 1];
  if (warp) __syncwarp();
  if (!warp || (threadIdx.x & 31) == 0) ptx::mbar_arrive(&c.sched_empty[n & 1]);
  return i;
}
// Claims tiles for the pair until none is left (one thread of the odd CTA): each once
// this CTA's warps have read the last but one, and both producers, for the first of a
// half, what that half held.
__device__ __forceinline__ void claim_tiles(SmemCtl& c, const KParams& p, int first, int total) {
  for (uint32_t n = 0;; ++n) {
    const int slot = n % (2 * kHalf);
    const uint32_t round = n / (2 * kHalf);
    if ((n == 1 && !ptx::mbar_wait(&c.claim, 0, &c.abort, kWaitLimitNs)) ||
        !ptx::mbar_wait(&c.sched_empty[n & 1], ((n >> 1) & 1) ^ 1, &c.abort, kWaitLimitNs) ||
        (slot % kHalf == 0 &&
         !mbar_wait_cluster(&c.mail_empty[slot / kHalf], (round & 1) ^ 1, &c.abort))) {
      flag_timeout(c, p.status, 15);
      return;
    }
    const int i = min(n > 0 ? atomicAdd(p.tile, 1) : first, total);
    c.mail[slot] = i;
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(ptx::mapa_shared(&c.mail[slot], 0)),
                 "r"(i)
                 : "memory");
    ptx::mbar_arrive_cluster(ptx::mapa_shared(&c.mail_full[slot], 0));
    ptx::mbar_arrive_cluster(ptx::mapa_shared(&c.mail_full[slot], 1));
    if (i == total) return;
  }
}

// ================================================================ producer
// Bytes of A loaded for a CTA's `rows` valid rows: rows that no expert has are not
// fetched (what the buffer held stays in the unused rows of the product).
__device__ __forceinline__ int a_bytes(int rows) {
  return rows <= 0 ? 0 : rows > 64 ? kABytes : (rows + kABoxRows - 1) / kABoxRows * kABoxRows * BK;
}
template <int MODE>
__device__ __forceinline__ void load_a(uint8_t* dst, const CUtensorMap* big,
                                       const CUtensorMap* small, uint32_t bar, int x, int half,
                                       int row, int rows) {
  if (rows <= 0) return;
  if (rows > 64) {
    if (MODE == FC1_DGRAD) tma_load_3d_pair(dst, big, bar, x, half, row);
    else ptx::tma_load_2d_pair(dst, big, bar, x, row);
    return;
  }
  for (int r = 0; r < rows; r += kABoxRows) {
    if (MODE == FC1_DGRAD) tma_load_3d_pair(dst + r * BK, small, bar, x, half, row + r);
    else ptx::tma_load_2d_pair(dst + r * BK, small, bar, x, row + r);
  }
}

template <int MODE, int KS>
__device__ __forceinline__ bool producer_tile(SmemCtl& c, int ring, uint8_t* smem, const KParams& p,
                                              const CUtensorMap* tmA, const CUtensorMap* tmS,
                                              const CUtensorMap* tmB, const Tile& t, uint32_t rank,
                                              int& stage, uint32_t& phase) {
  // (the even CTA announces both CTAs' bytes)
  const uint32_t bytes = 2 * kBBytes + a_bytes(t.rows) + a_bytes(min(BM, t.rows_odd));
  const int row = t.row0 + t.m0;
  const int nk = Mode<MODE>::kblocks(p), nf = (p.F + 127) / 128;
  if (!Mode<MODE>::kFirst) {
    if (!wait_expert(c, p, t.e)) return false;
    // the generic writes it waited for, before the TMA (async-proxy) reads
    asm volatile("fence.proxy.async.global;" ::: "memory");
  }
  for (int kt = 0; kt < nk; ++kt) {
    if (!ptx::mbar_wait(&c.empty[ring + stage], phase ^ 1, &c.abort, kWaitLimitNs)) {
      flag_timeout(c, p.status, 1);
      return false;
    }
    if (rank == 1 && kt == nk / 4) ptx::mbar_arrive(&c.claim);
    uint8_t* sA = smem + stage * kStageBytes;
    uint8_t* sB = sA + kABytes;
    const int k0 = kt * BK;
    // both CTAs' loads complete on the even CTA's full[stage]
    uint64_t* bar = &c.full[ring + stage];
    const uint32_t fb = ptx::mapa_shared(bar, 0);
    if (rank == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
    if (MODE == FC1_FWD) {  // even CTA: 128 gate rows of W1, odd CTA: 128 up rows
      load_a<MODE>(sA, tmA, tmS, fb, k0, 0, row, t.rows);
      ptx::tma_load_2d_pair(sB, tmB, fb, k0, (2 * t.e + rank) * p.F + t.n0);
    } else if (MODE == FC2_FWD) {
      load_a<MODE>(sA, tmA, tmS, fb, k0, 0, row, t.rows);
      ptx::tma_load_2d_pair(sB, tmB, fb, k0, t.e * p.H + t.n0 + 128 * rank);
    } else if (MODE == FC2_DGRAD) {
      load_a<MODE>(sA, tmA, tmS, fb, k0, 0, row, t.rows);
      tma_load_3d_pair(sB, tmB, fb, t.n0 + 128 * rank, k0, t.e);
    } else {
      const int half = kt >= nf, kb = (kt - half * nf) * BK;
      load_a<MODE>(sA, tmA, tmS, fb, kb, half, row, t.rows);
      tma_load_3d_pair(sB, tmB, fb, t.n0 + 128 * rank, kb, 2 * t.e + half);
    }
    if (++stage == KS) {
      stage = 0;
      phase ^= 1;
    }
  }
  return true;
}

// ================================================================ scales
// One arrival on the even CTA's barrier, after this warp's TMEM accesses. Those are
// complete when their waits return: no earlier memory operation needs to be
// released to the other CTA.
__device__ __forceinline__ void release(uint64_t* bar, uint32_t rank, int lane) {
  ptx::tc_fence_before();
  __syncwarp();
  if (lane == 0) {
    if (rank == 0) ptx::mbar_arrive(bar);
    else arrive_remote(ptx::mapa_shared(bar, 0));
  }
}

// Scale byte of weight block (K block kb, 128-column half i of the tile).
template <int MODE>
__device__ __forceinline__ uint32_t weight_scale(const KParams& p, const Tile& t, int kb, int i) {
  const int nh = (p.H + 127) / 128, nf = (p.F + 127) / 128;
  const size_t e = t.e;
  if (MODE == FC1_FWD) {
    return kb < nh ? p.sb[((e * 2 + i) * nf + t.n0 / 128) * nh + kb] : 0;
  } else if (MODE == FC2_FWD) {
    const int hb = t.n0 / 128 + i;
    return kb < nf && hb < nh ? p.sb[(e * nh + hb) * nf + kb] : 0;
  } else if (MODE == FC2_DGRAD) {
    const int fb = t.n0 / 128 + i;
    return kb < nh && fb < nf ? p.sb[(e * nh + kb) * nf + fb] : 0;
  } else {
    const int hb = t.n0 / 128 + i;
    return kb < 2 * nf && hb < nh ? p.sb[(e * 2 * nf + kb) * nh + hb] : 0;
  }
}

template <int MODE>
__device__ __forceinline__ bool scales_tile(SmemCtl& c, const KParams& p, const Tile& t,
                                            uint32_t tmem, uint32_t rank, uint32_t& group, int quarter,
                                            int lane) {
  const int nk = Mode<MODE>::kblocks(p);
  const uint32_t* words = reinterpret_cast<const uint32_t*>(p.sa);
  const long long r0 = (long long)t.row0 + t.m0;
  if (!Mode<MODE>::kFirst) {
    bool ok = true;
    if (lane == 0) ok = wait_expert(c, p, t.e);
    if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
    __syncwarp();  // what lane 0 acquired, for all lanes
  }
  for (int g = 0; g * 4 < nk; ++g, ++group) {
    // row r of the tile: lane r % 32, column r / 32
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = r0 + lane + 32 * i;
      w[i] = r < p.N ? __ldcg(words + (size_t)g * p.N + r) : 0;
    }
    // lanes 0..7 fetch the weight bytes of (half, K block), every lane packs them
    const uint32_t b = lane < 8 ? weight_scale<MODE>(p, t, 4 * g + (lane & 3), lane >> 2) : 0;
    uint32_t wb[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) wb[i >> 2] |= __shfl_sync(0xffffffffu, b, i) << (8 * (i & 3));
    const int buf = group % kSf;
    if (!ptx::mbar_wait(&c.sf_empty[buf], ((group / kSf) & 1) ^ 1, &c.abort, kWaitLimitNs)) {
      if (lane == 0) flag_timeout(c, p.status, 2);
      return false;
    }
    __syncwarp();
    ptx::tc_fence_after();  // the MMAs that read this buffer are done
    const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + kTmemScales + buf * 12;
    const uint32_t w0[4] = {wb[0], wb[0], wb[0], wb[0]}, w1[4] = {wb[1], wb[1], wb[1], wb[1]};
    tmem_st_x4(at, w);
    tmem_st_x4(at + 4, w0);
    tmem_st_x4(at + 8, w1);
    tmem_st_wait();
    release(&c.sf_full[buf], rank, lane);
  }
  return true;
}

// ================================================================ MMA issuer
// The whole warp runs this, so that addresses and descriptors stay in uniform
// registers; one elected lane issues.
struct MmaState {
  int stage = 0;
  uint32_t phase = 0, group = 0, tiles = 0;
};
template <int MODE, int KS>
__device__ __forceinline__ bool mma_tile(SmemCtl& c, int ring, uint32_t smem, const KParams& p,
                                         uint32_t tmem, MmaState& m) {
  constexpr uint32_t idesc = idesc_mxf8(2 * BM, BN, Mode<MODE>::kBMn);
  // one 128-byte atom wide in N (no second atom: LBO unused), or K-major
  const uint64_t desc0 = ptx::sdesc_sw128(0, 16, 1024);
  constexpr uint32_t b_adv = Mode<MODE>::kBMn ? (4096 >> 4) : (32 >> 4);
  const int nk = Mode<MODE>::kblocks(p);
  const int acc = m.tiles & 1;
  auto wait = [&](uint64_t* bar, uint32_t parity, int where) {
    const bool got = ptx::mbar_wait(bar, parity, &c.abort, kWaitLimitNs);
    if (__all_sync(0xffffffffu, got)) return true;
    flag_timeout(c, p.status, where);
    return false;
  };
  // the first stage and scales, then this accumulator (free since the tile before
  // the last), and last the columns it shares with the previous tile's, which come
  // free last: only they delay the first MMA
  if (!wait(&c.sf_full[m.group % kSf], (m.group / kSf) & 1, 4)) return false;
  if (!wait(&c.full[ring + m.stage], m.phase, 5)) return false;
  if (!wait(&c.tmem_empty[acc], ((m.tiles >> 1) & 1) ^ 1, 3)) return false;
  if (m.tiles > 0 && !wait(&c.ovl, (m.tiles - 1) & 1, 3)) return false;
  ptx::tc_fence_after();
  const uint32_t d = tmem + acc * kAccStep;
  for (int k0 = 0; k0 < nk; k0 += 4) {  // four K blocks: one buffer of scales
    const int buf = m.group % kSf;
    if (k0 && !wait(&c.sf_full[buf], (m.group / kSf) & 1, 4)) return false;
    const uint32_t sfa = tmem + kTmemScales + buf * 12;
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      if (k0 + kb >= nk) break;
      if (k0 + kb) {
        if (!wait(&c.full[ring + m.stage], m.phase, 5)) return false;
        ptx::tc_fence_after();
      }
      const uint64_t adesc = desc0 | ((smem + m.stage * kStageBytes) >> 4);
      const uint64_t bdesc = adesc + (kABytes >> 4);
      constexpr uint32_t kSel = (1u << 4) | (1u << 29);  // scale byte kb of both operands
      const uint32_t acc_on = (k0 + kb) != 0;
      if (elect_one()) {
        umma_mxf8_pair(d, adesc, bdesc, idesc | kb * kSel, sfa, sfa + 4, acc_on);
#pragma unroll
        for (int kk = 1; kk < 4; ++kk)
          umma_mxf8_pair(d, adesc + kk * 2, bdesc + kk * b_adv, idesc | kb * kSel, sfa, sfa + 4, 1);
        ptx::umma_commit_pair(&c.empty[ring + m.stage], 3);
        if (kb == 3 || k0 + kb == nk - 1) ptx::umma_commit_pair(&c.sf_empty[buf], 3);
        if (k0 + kb == nk - 1) ptx::umma_commit_pair(&c.tmem_full[acc], 3);
      }
      __syncwarp();
      if (++m.stage == KS) {
        m.stage = 0;
        m.phase ^= 1;
      }
    }
    ++m.group;
  }
  ++m.tiles;
  return true;
}

// ================================================================ epilogue
// Larger of this thread's and its partner warp's block maximum (the same row,
// the other 64 columns), as fp32 bits. buf alternates between calls, so that a
// warp never overwrites a value that its partner has yet to read: it passes the
// next call's barrier only after the partner has read this call's. (An mbarrier, as
// its wait ends after an abort when the partner does not come. n counts the calls.)
__device__ __forceinline__ uint32_t pair_max(SmemCtl& c, const KParams& p, uint32_t m, int ew,
                                             int lane, uint32_t& n) {
  const int buf = n & 1;
  uint64_t* bar = &c.paired[ew & 3];
  c.amax[buf][ew][lane] = m;
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(bar);
  if (!ptx::mbar_wait(bar, buf, &c.abort, kWaitLimitNs)) flag_timeout(c, p.status, 16);
  ++n;
  return max(m, c.amax[buf][ew ^ 4][lane]);
}

// Hands a first-GEMM tile, the n-th of this CTA, to the counting warp, which has
// counted the one before the last. The gradient's only once the next tile is known
// (and before anything is waited for that could depend on this one): daq leaves by
// TMA, and the stores' completion, waited for here, takes 1000 clocks and more.
template <int MODE>
__device__ __forceinline__ void hand_over(SmemCtl& c, const KParams& p, uint32_t n, int lane) {
  __syncwarp();
  if (lane == 0) {
    if (MODE == FC2_DGRAD) ptx::bulk_wait_group0();
    if (!ptx::mbar_wait(&c.counted[n & 1], ((n >> 1) & 1) ^ 1, &c.abort, kWaitLimitNs))
      flag_timeout(c, p.status, 7);
    ptx::mbar_arrive(&c.stored[n & 1]);
  }
  __syncwarp();
}

// ================================================================ aux loader
// FC2 dgrad: the saved pre-activations of a tile, in the epilogue's four steps:
// for each 128 columns (half) and each 32 of a warp's 64 columns (i), the gate and
// up boxes of both warps of a quarter.
__device__ __forceinline__ bool aux_tile(SmemCtl& c, uint8_t* aux, const KParams& p,
                                         const CUtensorMap* map, const Tile& t, uint32_t& tiles,
                                         uint32_t& step) {
  const int rev = p.halves == 2 ? (tiles & 1) ^ 1 : 0;
  ++tiles;
  if (t.rows <= 0) return true;
  for (int n = 0; n < 2 * p.halves; ++n, ++step) {
    const int b = step & 1;
    if (!ptx::mbar_wait(&c.aux_empty[b], ((step >> 1) & 1) ^ 1, &c.abort, kWaitLimitNs)) {
      flag_timeout(c, p.status, 9);
      return false;
    }
    uint8_t* dst = aux + b * kAuxBytes;
    uint64_t* bar = &c.aux_full[b];
    ptx::mbar_arrive_expect_tx(bar, kAuxBytes);
    const int x = t.n0 + 128 * ((n >> 1) ^ rev) + 32 * (n & 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ptx::tma_load_2d(dst + 16384 * h, map, bar, x + 64 * h, t.row0 + t.m0);
      ptx::tma_load_2d(dst + 16384 * h + 8192, map, bar, p.F + x + 64 * h, t.row0 + t.m0);
    }
  }
  return true;
}

// The columns that the two accumulators share are the first one's last 64 and
// the second one's first 64. An epilogue therefore starts with the higher half of
// its columns on the first accumulator (rev = 1) and with the lower half on the
// second; the warps that hold the shared columns (hf == rev) release them as soon
// as they are in registers.
template <int MODE>
__device__ __forceinline__ bool epilogue_tile(SmemCtl& c, const uint8_t* aux, uint4* buf,
                                              const KParams& p, const Maps& m, const Tile& t,
                                              uint32_t tmem, uint32_t rank, uint32_t& tiles,
                                              uint32_t& step, uint32_t& pairs, int ew, int lane) {
  const int q = ew & 3, hf = ew >> 2;
  const int acc = tiles & 1, rev = acc ^ 1;
  const size_t row0 = (size_t)t.row0 + t.m0 + q * 32, row = row0 + lane;  // this warp's, thread's
  const bool rok = q * 32 + lane < t.rows;
  const Out out = {buf, lane, t.rows - q * 32};
  if (!ptx::mbar_wait(&c.tmem_full[acc], (tiles >> 1) & 1, &c.abort, kWaitLimitNs)) {
    if (lane == 0) flag_timeout(c, p.status, 6);
    return false;
  }
  __syncwarp();
  ptx::tc_fence_after();
  const uint32_t tbase = tmem + acc * kAccStep + ((uint32_t)(q * 32) << 16);
  if (q * 32 >= t.rows) {  // nothing to store (both warps of the quarter)
    if (hf == rev) release(&c.ovl, rank, lane);
    release(&c.tmem_empty[acc], rank, lane);
    if (MODE == FC2_DGRAD && t.rows > 0) {  // the other quarters' pre-activations pass by
      for (int n = 0; n < 2 * p.halves; ++n, ++step) {
        if (!ptx::mbar_wait(&c.aux_full[step & 1], (step >> 1) & 1, &c.abort, kWaitLimitNs)) {
          if (lane == 0) flag_timeout(c, p.status, 11);
          return false;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&c.aux_empty[step & 1]);
      }
    }
  } else if (MODE == FC1_FWD) {
    // columns 0..127 gate, 128..255 up of one 128-wide block of h; this warp's 64
    // of each, the shared ones (up 64..127 of the first accumulator, gate 0..63 of
    // the second) first
    uint32_t hw[32], s0[32], s1[32], o[32];
    uint32_t mx = 0;
    const uint32_t sbase = tbase + 128 * rev + 64 * hf, obase = tbase + 128 * (rev ^ 1) + 64 * hf;
    ptx::tmem_ld_32x32b_x32(sbase, s0);
    ptx::tmem_ld_32x32b_x32(sbase + 32, s1);
    ptx::tmem_ld_wait(s0, s1);
    if (hf == rev) release(&c.ovl, rank, lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int f = t.n0 + 64 * hf + 32 * i;
      const bool ok = f < p.F;
      uint32_t(&sh)[32] = i ? s1 : s0;
      ptx::tmem_ld_32x32b_x32(obase + 32 * i, o);
      ptx::tmem_ld_wait(o);
      if (i == 1) release(&c.tmem_empty[acc], rank, lane);
      uint32_t gw[16], uw[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t ws = pack_bf16x2(__uint_as_float(sh[2 * j]), __uint_as_float(sh[2 * j + 1]));
        const uint32_t wo = pack_bf16x2(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1]));
        gw[j] = rev ? wo : ws;
        uw[j] = rev ? ws : wo;
        const float g0 = bf16_lo(gw[j]), g1 = bf16_hi(gw[j]);
        const uint32_t h2 = pack_bf16x2(g0 * sigmoid_f(g0) * bf16_lo(uw[j]),
                                        g1 * sigmoid_f(g1) * bf16_hi(uw[j]));
        hw[16 * i + j] = h2;
        if (ok) mx = absmax_bf16x2(mx, h2);  // columns past F are not part of the block
      }
      if (ok) {
        if (p.out0) {
          store_box(out, &m.o1, gw, p.out0, row0, 2 * p.F, f);
          store_box(out, &m.o1, uw, p.out0, row0, 2 * p.F, p.F + f);
        }
        if (p.out1) store_box(out, &m.o2, hw + 16 * i, p.out1, row0, p.F, f);
      }
    }
    const uint32_t b = fp8_scale_byte(pair_max(c, p, absmax_bits(mx), ew, lane, pairs));
    const uint32_t inv = fp8_inv_scale2(b);
    const int f = t.n0 + 64 * hf, fb = t.n0 / 128;
    if (rok && f < p.F) {
      uint8_t* qp = p.q + row * (size_t)p.F + f;
      store_fp8(qp, hw, inv);
      store_fp8(qp + 32, hw + 16, inv);
    }
    if (hf == 0 && rok) p.s[((size_t)(fb >> 2) * p.N + row) * 4 + (fb & 3)] = (uint8_t)b;
  } else if (MODE == FC2_DGRAD) {
    const int nf = (p.F + 127) / 128;
    int held = -1;  // lane 0: the buffer that da is still being stored from
    auto free_held = [&] {
      if (held >= 0) {
        ptx::bulk_wait_group_read0();
        ptx::mbar_arrive(&c.aux_empty[held]);
        held = -1;
      }
    };
    uint32_t v[2][32];
    // 128 columns: one block of da_gate, one of da_up; a 128-column tile's are the lower
    // half, in which the first accumulator shares nothing
    if (p.halves == 1 && rev && hf == rev) release(&c.ovl, rank, lane);
#pragma unroll 1
    for (int hi = 0; hi < p.halves; ++hi) {
      const int half = p.halves == 2 ? hi ^ rev : 0;
      uint32_t gw[32], uw[32];
      uint32_t mg = 0, mu = 0;
      const uint32_t vbase = tbase + 128 * half + 64 * hf;
      ptx::tmem_ld_32x32b_x32(vbase, v[0]);
      ptx::tmem_ld_32x32b_x32(vbase + 32, v[1]);
      ptx::tmem_ld_wait(v[0], v[1]);
      if (hi == 0 && hf == rev && (p.halves == 2 || !rev)) release(&c.ovl, rank, lane);
      if (hi == p.halves - 1) release(&c.tmem_empty[acc], rank, lane);
#pragma unroll
      for (int i = 0; i < 2; ++i, ++step) {
        const int f = t.n0 + 128 * half + 64 * hf + 32 * i;
        const bool ok = f < p.F;
        free_held();
        // the step's gate and up boxes: 64-byte rows, 16-byte chunk j of row r at j ^ ((r >> 1) & 3)
        const int b = step & 1;
        if (!ptx::mbar_wait(&c.aux_full[b], (step >> 1) & 1, &c.abort, kWaitLimitNs)) {
          if (lane == 0) flag_timeout(c, p.status, 12);
          return false;
        }
        uint4 gc[4], uc[4];
        const int r = q * 32 + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = b * kAuxBytes + 16384 * hf + r * 64 + ((j ^ ((r >> 1) & 3)) * 16);
          gc[j] = *reinterpret_cast<const uint4*>(aux + at);
          uc[j] = *reinterpret_cast<const uint4*>(aux + 8192 + at);
        }
        __syncwarp();
        // da leaves from where the pre-activations were (this warp's rows of the gate and
        // up boxes): the buffer is free once the stores have read it, at the next step.
        // Through the 2 KB buffer the second box of a step would wait for the first one's
        // store, 700 clocks; unstored, or with rows of another expert, it is free now.
        const bool whole = ok && out.rows >= 32, inplace = p.out0 && whole;
        // the half's last step stays for daq's boxes (below)
        if (lane == 0) {
          if (whole && (inplace || i == 1)) held = b;
          else ptx::mbar_arrive(&c.aux_empty[b]);
        }
        const uint32_t* ag = reinterpret_cast<const uint32_t*>(gc);
        const uint32_t* au = reinterpret_cast<const uint32_t*>(uc);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float d0 = __uint_as_float(v[i][2 * j]), d1 = __uint_as_float(v[i][2 * j + 1]);
          const float a0 = bf16_lo(ag[j]), a1 = bf16_hi(ag[j]);
          const float s0 = sigmoid_f(a0), s1 = sigmoid_f(a1);
          const float e0 = d0 * s0, e1 = d1 * s1;
          const uint32_t u2 = pack_bf16x2(e0 * a0, e1 * a1);
          const uint32_t g2 = pack_bf16x2(e0 * bf16_lo(au[j]) * fmaf(a0, 1.f - s0, 1.f),
                                          e1 * bf16_hi(au[j]) * fmaf(a1, 1.f - s1, 1.f));
          uw[16 * i + j] = u2;
          gw[16 * i + j] = g2;
          if (ok) {
            mu = absmax_bf16x2(mu, u2);
            mg = absmax_bf16x2(mg, g2);
          }
        }
        if (inplace) {
          uint8_t* slab = const_cast<uint8_t*>(aux) + b * kAuxBytes + 16384 * hf + q * 2048;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16);
            const uint32_t *g = gw + 16 * i + 4 * j, *u = uw + 16 * i + 4 * j;
            *reinterpret_cast<uint4*>(slab + at) = make_uint4(g[0], g[1], g[2], g[3]);
            *reinterpret_cast<uint4*>(slab + 8192 + at) = make_uint4(u[0], u[1], u[2], u[3]);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::tma_store_2d(&m.o1, slab, f, (int)row0);
            ptx::tma_store_2d(&m.o1, slab + 8192, p.F + f, (int)row0);
            ptx::bulk_commit_group();
          }
        } else if (p.out0 && ok && rok) {
          bf16* da = p.out0 + row * (size_t)(2 * p.F) + f;
          st_sector(da, gw + 16 * i);
          st_sector(da + 16, gw + 16 * i + 8);
          st_sector(da + p.F, uw + 16 * i);
          st_sector(da + p.F + 16, uw + 16 * i + 8);
        }
      }
      const uint32_t bg = fp8_scale_byte(pair_max(c, p, absmax_bits(mg), ew, lane, pairs));
      const uint32_t bu = fp8_scale_byte(pair_max(c, p, absmax_bits(mu), ew, lane, pairs));
      const uint32_t ig = fp8_inv_scale2(bg), iu = fp8_inv_scale2(bu);
      const int f = t.n0 + 128 * half + 64 * hf;
      if (f < p.F && out.rows >= 32) {
        // daq's 64-byte rows, in place of the last step's da once that has been read (as
        // 32-byte sectors from registers every row is a request of its own: 182 -> 177 us
        // on the balanced layer, 234 -> 229 on the skewed one)
        uint8_t* slab = const_cast<uint8_t*>(aux) + ((step - 1) & 1) * kAuxBytes + 16384 * hf +
                        q * 2048;
        if (lane == 0) ptx::bulk_wait_group_read0();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16);
          *reinterpret_cast<uint4*>(slab + at) = fp8x16(gw + 8 * j, ig);
          *reinterpret_cast<uint4*>(slab + 8192 + at) = fp8x16(uw + 8 * j, iu);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::tma_store_2d(&m.o2, slab, f, (int)row0);
          ptx::tma_store_2d(&m.o2, slab + 8192, p.F + f, (int)row0);
          ptx::bulk_commit_group();
        }
      } else if (rok && f < p.F) {
        uint8_t* qp = p.q + row * (size_t)(2 * p.F) + f;
        store_fp8(qp, gw, ig);
        store_fp8(qp + 32, gw + 16, ig);
        store_fp8(qp + p.F, uw, iu);
        store_fp8(qp + p.F + 32, uw + 16, iu);
      }
      if (rok && t.n0 + 128 * half < p.F) {
        const int kb = hf * nf + t.n0 / 128 + half;  // the gate's byte or the up half's
        p.s[((size_t)(kb >> 2) * p.N + row) * 4 + (kb & 3)] = (uint8_t)(hf ? bu : bg);
      }
    }
    free_held();
  } else {
    // plain fp32 tile -> bf16; the other half's TMEM loads run beside the stores
    uint32_t v[2][32];
    const uint32_t vbase = tbase + 64 * hf;
    ptx::tmem_ld_32x32b_x32(vbase + 128 * rev, v[0]);
    ptx::tmem_ld_32x32b_x32(vbase + 128 * rev + 32, v[1]);
    ptx::tmem_ld_wait(v[0], v[1]);
    if (hf == rev) release(&c.ovl, rank, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int half = (i >> 1) ^ rev;
      if (i == 2) {
        ptx::tmem_ld_wait(v[0], v[1]);
        release(&c.tmem_empty[acc], rank, lane);
      }
      const int col = 128 * half + 64 * hf + 32 * (i & 1);
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        w[j] = pack_bf16x2(__uint_as_float(v[i & 1][2 * j]), __uint_as_float(v[i & 1][2 * j + 1]));
      if (i < 2) ptx::tmem_ld_32x32b_x32(vbase + 128 * (rev ^ 1) + 32 * i, v[i]);
      if (t.n0 + col < p.H) store_box(out, &m.o3, w, p.out0, row0, p.H, t.n0 + col);
    }
  }
  if (MODE == FC1_FWD) hand_over<MODE>(c, p, tiles, lane);
  ++tiles;
  return true;
}

// ================================================================ counting
// Counts a first-GEMM tile for its expert once the epilogue's stores are visible
// device-wide: the fence takes 3000 to 4000 clocks with stores in flight, which
// the epilogue warps spend on the next tile. (Their stores are ordered before
// their arrivals, the arrivals before this fence, the fence before the count.)
__device__ __forceinline__ bool count_tile(SmemCtl& c, const KParams& p, int e, uint32_t& tiles) {
  const int acc = tiles & 1;
  if (!ptx::mbar_wait(&c.stored[acc], (tiles >> 1) & 1, &c.abort, kWaitLimitNs)) {
    flag_timeout(c, p.status, 8);
    return false;
  }
  __threadfence();
  atomicAdd(p.dep + e, 1);
  ptx::mbar_arrive(&c.counted[acc]);
  ++tiles;
  return true;
}

template <int M1, int M2>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_fp8_kernel(const __grid_constant__ Maps m, const KParams args1, const KParams p2) {
  using C = Chain<M1>;
  KParams p1 = args1;
  extern __shared__ uint8_t dyn_smem[];
  __shared__ SmemCtl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) &
                                             ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p1.E;
  const uint32_t rank = ptx::cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kBars; ++s) {
      ptx::mbar_init(&ctl.full[s], 1);
      ptx::mbar_init(&ctl.empty[s], 1);
    }
    for (int b = 0; b < kSf; ++b) {
      ptx::mbar_init(&ctl.sf_full[b], 8);  // both CTAs' scale warps
      ptx::mbar_init(&ctl.sf_empty[b], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&ctl.sched_full[a], 1);
      ptx::mbar_init(&ctl.sched_empty[a], readers(rank, C::kAux));
      ptx::mbar_init(&ctl.mail_empty[a], 2);  // (the odd CTA's) both producers
      ptx::mbar_init(&ctl.stored[a], 8);  // this CTA's epilogue warps
      ptx::mbar_init(&ctl.counted[a], 1);
      ptx::mbar_init(&ctl.aux_full[a], 1);
      ptx::mbar_init(&ctl.aux_empty[a], 8);
      ptx::mbar_init(&ctl.tmem_full[a], 1);
      ptx::mbar_init(&ctl.tmem_empty[a], 16);  // both CTAs' epilogue warps
    }
    for (int i = 0; i < 2 * kHalf; ++i) ptx::mbar_init(&ctl.mail_full[i], 1);
    for (int q = 0; q < 4; ++q) ptx::mbar_init(&ctl.paired[q], 2);
    ptx::mbar_init(&ctl.ovl, 8);  // the four warps of each CTA that hold the shared columns
    ptx::mbar_init(&ctl.drain, 1);
    ptx::mbar_init(&ctl.claim, 1);
    ptx::mbar_init(&ctl.aux_done, 1);
    ctl.abort = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  ptx::cluster_sync();  // barriers are live in both CTAs before TMEM is allocated for the pair
  if (warp == 1) {
    ptx::tmem_alloc_pair(&ctl.tmem_base, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  if (threadIdx.x == 0) {
    for (const CUtensorMap* t : {&m.a1, &m.s1, &m.b1, &m.a2, &m.s2, &m.b2})
      ptx::tma_prefetch_desc(t);
  }
  pdl_wait();
  int first = 0;  // the first tile, claimed while the tables are made
  if (warp == 1 && lane == 0 && rank == 1) first = atomicAdd(p1.tile, 1);
  // offsets outside 0..N would send stores out of the buffers
  for (int e = threadIdx.x; e <= E; e += blockDim.x)
    ctl.off[e] = (int)min(max((long long)p1.off[e], 0ll), p1.N);
  __syncthreads();
  p1.halves = 2;
  if (C::kAux) {
    // a tile's epilogue is the longest part of a small gradient: with tiles for half
    // of the pairs or fewer, tiles of one 128-column half (8 experts: 64 tokens, H
    // 320, F 448 21.2 -> 18.6 us; 256 tokens, H 1024, F 768 27.9 -> 24.9 us)
    int tiles = 0;
    for (int e = lane; e < E; e += 32)
      tiles += max(0, (ctl.off[e + 1] - ctl.off[e] + 2 * BM - 1) / (2 * BM));
    tiles = __reduce_add_sync(0xffffffffu, tiles) * Mode<M1>::ntiles(p1);
    if (2 * tiles <= (int)ptx::cluster_count_x()) p1.halves = 1;
  }
  if (warp < 2) {  // pair tiles per expert -> exclusive prefix, one warp for each GEMM
    const int nt = warp == 0 ? Mode<M1>::ntiles(p1) : Mode<M2>::ntiles(p2);
    int carry = 0;
    for (int base = 0; base < E; base += 32) {
      const int e = base + lane;
      int n = 0;
      if (e < E) {
        const int cnt = ctl.off[e + 1] - ctl.off[e];
        n = cnt > 0 ? (cnt + 2 * BM - 1) / (2 * BM) * nt : 0;
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (e < E) ctl.tstart[warp][e] = carry + incl - n;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) ctl.tstart[warp][E] = carry;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  const int total1 = ctl.tstart[0][E], total = total1 + ctl.tstart[1][E];
  int cur1 = 0, cur2 = 0;
  auto tile1 = [&](int i) { return tile_at<M1>(p1, ctl, i, cur1, rank); };
  auto tile2 = [&](int i) { return tile_at<M2>(p2, ctl, i - total1, cur2, rank); };
  if (warp < 4) {
    regs_dec<kRegsControl>();
    if (warp == 0 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, second = !C::kAux;
      int ring = 0, ring_stages = C::kStages1;
      for (uint32_t n = 0; ok; ++n) {
        const int i = take_tile(ctl, n, p1.status);
        ok = i >= 0;
        if (!ok || i >= total) break;
        if (i < total1) {
          ok = producer_tile<M1, C::kStages1>(ctl, 0, smem, p1, &m.a1, &m.s1, &m.b1, tile1(i),
                                              rank, stage, phase);
          continue;
        }
        if (!second) {
          // the second ring takes the first one's memory and the pre-activations':
          // wait until every stage and every step have been read (the aux loader knows:
          // the epilogue may be more than a tile behind this warp)
          for (int s = 0; ok && s < C::kStages1; ++s)
            ok = ptx::mbar_wait(&ctl.empty[s], s < stage ? phase : phase ^ 1, &ctl.abort,
                                kWaitLimitNs);
          ok = ok && ptx::mbar_wait(&ctl.aux_done, 0, &ctl.abort, kWaitLimitNs);
          if (!ok) {
            flag_timeout(ctl, p1.status, 13);
            break;
          }
          second = true;
          ring = C::kSecond;
          ring_stages = C::kStages2;
          stage = 0;
          phase = 0;
        }
        ok = producer_tile<M2, C::kStages2>(ctl, C::kSecond, smem, p2, &m.a2, &m.s2, &m.b2,
                                            tile2(i), rank, stage, phase);
      }
      if (!ok && rank == 0) drain_loads(ctl.full + ring, ring_stages, stage, phase);  // both CTAs'
    } else if (warp == 1 && rank == 0) {
      MmaState st;
      bool ok = true, second = !C::kAux;
      for (uint32_t n = 0; ok; ++n) {
        const int i = next_tile(ctl, n, p1.status, true);
        ok = i >= 0;
        if (!ok || i >= total) break;
        if (i >= total1 && !second) {
          second = true;
          st.stage = 0;
          st.phase = 0;
        }
        ok = i < total1 ? mma_tile<M1, C::kStages1>(ctl, 0, ptx::smem_u32(smem), p1, tmem, st)
                        : mma_tile<M2, C::kStages2>(ctl, C::kSecond, ptx::smem_u32(smem), p2, tmem,
                                                    st);
      }
      // no MMA may still run when TMEM is released (the same lane is elected as above)
      __syncwarp();
      if (elect_one()) ptx::umma_commit_pair(&ctl.drain, 1);
      if (!ptx::mbar_wait(&ctl.drain, 0, &ctl.abort, kWaitLimitNs)) {
        int dummy = 0;
        ptx::mbar_wait(&ctl.drain, 0, &dummy, kWaitLimitNs);
      }
    } else if (warp == 1 && lane == 0) {
      claim_tiles(ctl, p1, first, total);
    } else if (C::kAux && warp == 3 && lane == 0) {
      ptx::tma_prefetch_desc(&m.aux);
      uint32_t tiles = 0, step = 0;
      bool ok = true, done = false;
      for (uint32_t n = 0; ok; ++n) {
        const int i = next_tile(ctl, n, p1.status, false);
        ok = i >= 0;
        if (!ok || i >= total) break;
        if (i < total1) {
          ok = aux_tile(ctl, smem + C::kAuxAt, p1, &m.aux, tile1(i), tiles, step);
        } else if (!done) {  // the last two steps have been read: the producer may have the room
          for (uint32_t b = step > 2 ? step - 2 : 0; ok && b < step; ++b)
            ok = ptx::mbar_wait(&ctl.aux_empty[b & 1], (b >> 1) & 1, &ctl.abort, kWaitLimitNs);
          if (!ok) flag_timeout(ctl, p1.status, 17);
          ptx::mbar_arrive(&ctl.aux_done);
          done = true;
        }
      }
      // after an abort: the loads of the last two steps have landed
      for (uint32_t n = step > 2 ? step - 2 : 0; !ok && n < step; ++n) {
        int none = 0;
        ptx::mbar_wait(&ctl.aux_full[n & 1], (n >> 1) & 1, &none, kWaitLimitNs);
      }
    } else if (warp == 2 && lane == 0) {
      uint32_t tiles = 0;
      bool ok = true;
      for (uint32_t n = 0; ok; ++n) {
        const int i = next_tile(ctl, n, p1.status, false);
        ok = i >= 0;
        if (!ok || i >= total) break;
        if (i < total1) ok = count_tile(ctl, p1, tile1(i).e, tiles);
      }
    }
    __syncwarp();
  } else if (warp < 12) {
    regs_inc<kRegsEpilogue>();
    uint32_t tiles = 0, step = 0, pairs = 0;
    bool ok = true, pending = false;
    const int ew = warp - 4;
    const uint8_t* aux = smem + C::kAuxAt;
    uint4* buf = reinterpret_cast<uint4*>(smem + C::kEpiAt) + ew * 128;
    for (uint32_t n = 0; ok; ++n) {
      const int i = next_tile(ctl, n, p1.status, true);
      if (pending) hand_over<M1>(ctl, p1, tiles - 1, lane);
      pending = M1 == FC2_DGRAD && i < total1;
      ok = i >= 0;
      if (!ok || i >= total) break;
      ok = i < total1 ? epilogue_tile<M1>(ctl, aux, buf, p1, m, tile1(i), tmem, rank, tiles, step,
                                          pairs, ew, lane)
                      : epilogue_tile<M2>(ctl, aux, buf, p2, m, tile2(i), tmem, rank, tiles, step,
                                          pairs, ew, lane);
    }
    // the buffers and the outputs must outlive the TMA stores
    if (lane == 0) ptx::bulk_wait_group0();
    __syncwarp();
  } else {
    regs_dec<kRegsControl>();
    uint32_t group = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      const int i = next_tile(ctl, n, p1.status, true);
      ok = i >= 0;
      if (!ok || i >= total) break;
      ok = i < total1 ? scales_tile<M1>(ctl, p1, tile1(i), tmem, rank, group, warp - 12, lane)
                      : scales_tile<M2>(ctl, p2, tile2(i), tmem, rank, group, warp - 12, lane);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::cluster_sync();  // the peer may still arrive on this CTA's barriers
  if (warp == 1) ptx::tmem_dealloc_pair(tmem, kTmemCols);
}

// ------------------------------------------------------------------ host side
// How many pairs can be resident at once on the current device, after setting
// the kernel's shared memory up there (once for each device).
template <int M1, int M2>
cudaError_t resident_pairs(int* pairs) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*pairs = known[dev].load()) > 0) return cudaSuccess;
  e = cudaFuncSetAttribute(grouped_gemm_fp8_kernel<M1, M2>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Chain<M1>::kDynSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(device_sm_count() / 2 * 2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Chain<M1>::kDynSmem;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(pairs, grouped_gemm_fp8_kernel<M1, M2>, &cfg);
  if (e == cudaSuccess && *pairs < 1) e = cudaErrorLaunchOutOfResources;
  if (e == cudaSuccess && dev < 64) known[dev].store(*pairs);
  return e;
}

template <int M1, int M2>
moe_status_t launch_chain(const moe_layer_desc_t& d, const Maps& m, const KParams& p1,
                          const KParams& p2, int kernel_id, cudaStream_t st) {
  int pairs = 0;
  cudaError_t e = resident_pairs<M1, M2>(&pairs);
  if (e == cudaSuccess) e = launch_zero_counters(p1.dep, d.E, p1.tile, st);
  if (e != cudaSuccess) {
    set_error("grouped_gemm_fp8_kernel set-up: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  // one pair for every two SMs, and no more than there can be tiles
  const long long n1 = ceil_div(d.F, 128);
  const long long rows = p1.N / (2 * BM) + std::min<long long>(p1.N, d.E);
  pairs = (int)std::min<long long>(pairs, rows * (n1 + ceil_div(d.H, BN)));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = MOE_PDL;
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Chain<M1>::kDynSmem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  {
    LaunchScope _ls(kernel_id, st);
    e = cudaLaunchKernelEx(&cfg, grouped_gemm_fp8_kernel<M1, M2>, m, p1, p2);
  }
  if (e != cudaSuccess) {
    set_error("grouped_gemm_fp8_kernel launch: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return check_launch("grouped_gemm_fp8_kernel");
}

KParams params(const moe_layer_desc_t& d, const int32_t* off, int* status, int* dep) {
  KParams p = {};
  p.E = d.E;
  p.H = d.H;
  p.F = d.F;
  p.N = (long long)d.T * d.k;
  p.off = off;
  p.status = status;
  p.dep = dep;
  p.tile = tile_counter(status);
  p.halves = 2;
  return p;
}

}  // namespace

moe_status_t launch_ffn_fwd_fp8(const moe_layer_desc_t& d, const uint8_t* xq, const uint8_t* xs,
                                const int32_t* off, const Fp8Weights& w, bf16* a, bf16* h,
                                uint8_t* hq, uint8_t* hs, bf16* o, int* status, int* dep,
                                cudaStream_t st) {
  const long long N = (long long)d.T * d.k;
  if (N == 0) return MOE_OK;
  if (N <= kFp8FewRows * d.E)
    return launch_ffn_rows_fp8(d, xq, xs, off, w, a, h, hq, hs, o, status, dep, st);
  Maps m = {};
  if (!make_map(&m.a1, xq, 2, d.H, N, 1, BM, 1) || !make_map(&m.s1, xq, 2, d.H, N, 1, kABoxRows, 1) ||
      !make_map(&m.b1, w.w1q, 2, d.H, 2ll * d.E * d.F, 1, 128, 1) ||
      !make_map(&m.a2, hq, 2, d.F, N, 1, BM, 1) || !make_map(&m.s2, hq, 2, d.F, N, 1, kABoxRows, 1) ||
      !make_map(&m.b2, w.w2q, 2, d.F, (long long)d.E * d.H, 1, 128, 1) ||
      !make_rows_map(&m.o3, o, N, d.H, 32) || (a && !make_rows_map(&m.o1, a, N, 2 * d.F, 32)) ||
      (h && !make_rows_map(&m.o2, h, N, d.F, 32)))
    return MOE_ERR_CUDA;
  KParams p1 = params(d, off, status, dep), p2 = p1;
  p1.sa = xs;
  p1.sb = w.w1s;
  p1.out0 = a;
  p1.out1 = h;
  p1.q = hq;
  p1.s = hs;
  p2.sa = hs;
  p2.sb = w.w2s;
  p2.out0 = o;
  return launch_chain<FC1_FWD, FC2_FWD>(d, m, p1, p2, K_FP8_FFN_FWD, st);
}

moe_status_t launch_ffn_dgrad_fp8(const moe_layer_desc_t& d, const uint8_t* dq, const uint8_t* ds,
                                  const bf16* a, const int32_t* off, const Fp8Weights& w, bf16* da,
                                  uint8_t* daq, uint8_t* das, bf16* dx_perm, int* status, int* dep,
                                  cudaStream_t st) {
  const long long N = (long long)d.T * d.k;
  if (N == 0) return MOE_OK;
  Maps m = {};
  if (!make_map(&m.a1, dq, 2, d.H, N, 1, BM, 1) || !make_map(&m.s1, dq, 2, d.H, N, 1, kABoxRows, 1) ||
      !make_map(&m.b1, w.w2q, 3, d.F, d.H, d.E, 128, 1) ||
      !make_map(&m.a2, daq, 3, d.F, 2, N, 1, BM) || !make_map(&m.s2, daq, 3, d.F, 2, N, 1, kABoxRows) ||
      !make_map(&m.b2, w.w1q, 3, d.H, d.F, 2ll * d.E, 128, 1) ||
      !make_rows_map(&m.o3, dx_perm, N, d.H, 32) || !make_rows_map(&m.aux, a, N, 2 * d.F, BM) ||
      !make_rows_map(&m.o2, daq, N, 2 * d.F, 32, true) ||
      (da && !make_rows_map(&m.o1, da, N, 2 * d.F, 32)))
    return MOE_ERR_CUDA;
  KParams p1 = params(d, off, status, dep), p2 = p1;
  p1.sa = ds;
  p1.sb = w.w2s;
  p1.out0 = da;
  p1.q = daq;
  p1.s = das;
  p2.sa = das;
  p2.sb = w.w1s;
  p2.out0 = dx_perm;
  return launch_chain<FC2_DGRAD, FC1_DGRAD>(d, m, p1, p2, K_FP8_FFN_DGRAD, st);
}

}  // namespace moe
