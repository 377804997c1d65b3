// Grouped expert GEMMs on microscaled 4-bit operands (see fp4.cuh): the SwiGLU expert FFN
// forward, FC1 -> FC2.
//
//   D[r, c] = sum over 32-wide K blocks b of
//             2^(sa[r,b]-127) 2^(sb[c,b]-127) sum_{i in b} A[r,i] B[c,i]
//
// The tensor cores apply both scales (tcgen05.mma kind::mxf4, 64 K values an
// instruction, two scales a row). One persistent launch for both products, a CTA pair
// (cta_group::2, M = 256, N = 256) per two SMs, as in grouped_gemm_fp8.cu:
//   warp 0      TMA producer: this CTA's 128 rows of A, once for a strip of tiles beside each
//               other, and its half of B, 256 K values (128 bytes) a stage. Twelve slots of 16
//               KB: as many for A as the longer product has stages (up to 8), the others B's
//   warp 1      TMEM allocator + (even CTA) MMA issuer; (odd CTA) claims tiles
//   warp 2      counts FC1 tiles for their experts
//   warp 3      producer of the scales' ring: contiguous copies of the rows' and the weights'
//               scale bytes, 3 KB a stage, 4 stages
//   warps 12..15 scales: shared memory -> TMEM (tcgen05.st), ahead of the MMAs: for each stage
//               16 columns of B's, and in a strip's first tile 8 of A's, which stay
//   warps 4..11 epilogue: TMEM -> registers -> SwiGLU, block scales, e2m1 -> global; two
//               warps per TMEM lane quarter, each owning 64 of every 128 columns. A block of
//               h (32 columns) lies in one thread.
// FC2 tiles wait for their expert's FC1 tiles through per-expert counters. Strips are
// claimed in order from a counter, FC1's first, so a wait is always for a tile that a
// running pair holds.
//
// TMEM: two 256-column accumulators that share 128 (columns 0..255 and 128..383), the
// scales of A's slots and four buffers of B's. The epilogue reads the shared columns first
// and releases them (ovl), so the next tile's MMAs start while it works on the rest.
//
// What bounds it. 64 experts of H 2048, F 1408 at 8192 tokens, top 8, skewed, nothing kept: 1134
// GFLOP in 244 us, 4.6 PFLOP/s, at 1330 W and 2070 MHz (the limit is 1400 W; before the
// strips 272 us at 2032 to 2062 MHz with the power cap active). A stage's four MMAs alone take
// some 600 clocks (512 at the nominal rate of this form, 64 K values an instruction), and what
// shares shared memory or TMEM with them adds its time: B's loads 95 clocks, scales 70, the
// epilogue's TMEM reads and boxes 190 (each found by leaving it out). A's loads were 85 more,
// hence the strips; tiles of N = 192, which would need no shared columns, take as long as N =
// 256. 128 experts of F 768 at 4096 tokens, balanced, a and h kept: 620 MB of DRAM traffic in 113
// us, 5.5 TB/s, 0.82 of a copy's rate: 8 us of set-up and last tiles, then 5.9.
//
// Ragged groups: expert e owns rows off[e]..off[e+1]-1; a tile's rows past the
// expert's end are computed on whatever was loaded and not stored (rows do not mix).
// Columns past a matrix edge likewise. K past an edge is not computed: H and F are
// multiples of an instruction's 64.
#include <algorithm>
#include <atomic>

#include "fp4_mma.cuh"

namespace moe {

using namespace fp8;
using namespace fp4;

namespace {

enum Fp4Mode {
  FC1 = 0,  // a, h, hq = SwiGLU(xq @ W1q^T)
  FC2 = 1   // o = hq @ W2q^T
};

constexpr int BM = 128, BN = 256, BK = kFp4Group;  // BM: rows of one CTA of the pair
constexpr int kRowBytes = BK / 2;                  // of a stage
constexpr int kSlotBytes = 128 * kRowBytes;        // a stage of A's rows, or of half of B's
constexpr int kSlots = 12;                         // shared by A and B (below)
constexpr int kMaxA = 8, kMaxB = 8;
constexpr int kEpiBytes = 8 * 2048;           // a 32 x 32 bf16 box for each epilogue warp
constexpr int kScA = 1152;                    // scales of a stage: 128 rows of A from an even one on ...
constexpr int kScBytes = kScA + BN * 8;       // ... and all of B's
constexpr int kSc = 4;                        // stages of scales in shared memory
static_assert((BM + 2) * 8 <= kScA && kScA % 16 == 0, "room for A's scales");
constexpr int kABoxRows = 16;                 // tiles of 64 rows or fewer load boxes of 16
constexpr int kTmemCols = 512;
constexpr int kAccStep = 128;                 // second accumulator's first column
// scale columns: 8 for each slot of A (4 for each half of a stage), buffers of 16 for B
constexpr int kTmemA = 384, kTmemB = kTmemA + 8 * kMaxA;
constexpr int kSf = 4;
static_assert(kTmemB + 16 * kSf <= kTmemCols, "TMEM columns");
constexpr int kThreads = 512;
// registers a thread: 128 at launch; the epilogue's two warpgroups take what the
// control and scale warpgroups give up (2 * 72 + 2 * 184 = 4 * 128)
constexpr int kRegsControl = 72, kRegsEpilogue = 184;
constexpr int kMaxE = 256;
constexpr int kEpiAt = kSlots * kSlotBytes, kScAt = kEpiAt + kEpiBytes;
constexpr size_t kDynSmem = kScAt + kSc * kScBytes + 1024;
constexpr int kHalf = 8;  // slots of half a mailbox (below)
// Strips (below) that a pair should get of each product, if they can be as many: few of the
// first, which the second follows, and more of the second, whose last ones are the end. us of
// the products, tiles of a strip in the first and the second:
//   prefill (11 and 8 tiles across)  11, 4 243   6, 4 244   11, 2 249   4, 4 249   2, 2 272   1, 1 328
//   train (6 and 8)                   6, 2 112   2, 2 111    3, 2 113   6, 4 118   3, 3 114   1, 1 124
// and these numbers, 2 and 4 against 2 and 6, 1 and 6, 4 and 6: 2048 tokens of the 64 experts, skewed,
// 99 / 107 / 106 / 109; 8000 of 16 experts of H, F 1024, top 4, 65 / 72 / 69 / 74; 20480 of one
// expert of H 2048, F 1408 97 / 97 / 112 / 93; train, a pass, 126.2 / 125.4 / 124.2 / 124.7.
constexpr int kStrips[2] = {2, 4};

struct Maps {
  CUtensorMap a1, s1, b1, a2, s2, b2;  // operands: A, A in small boxes, B of both GEMMs
  CUtensorMap o1, o2, o3;              // a, h, o
};

struct KParams {
  int E, H, F;
  long long N;
  const int32_t* off;
  const uint8_t *xs, *w1s, *w2s;
  bf16 *a, *h, *o;    // a and h may be NULL
  uint8_t *hq, *hs;
  int* status;
  int* dep;           // per-expert count of FC1 tiles stored, by CTA
  int* tile;          // strips claimed
  int na, nb;         // slots of A and of B
  int strip[2];       // tiles of a strip, in both products
};

template <int MODE>
__device__ __forceinline__ int kvalues(const KParams& p) { return MODE == FC1 ? p.H : p.F; }
template <int MODE>
__device__ __forceinline__ int kstages(const KParams& p) { return (kvalues<MODE>(p) + BK - 1) / BK; }
template <int MODE>
__device__ __forceinline__ int ntiles(const KParams& p) {
  return MODE == FC1 ? (p.F + 127) / 128 : (p.H + BN - 1) / BN;
}

// A strip: up to p.strip tiles side by side, over the same rows.
struct Strip {
  int e, m0, rows, row0;  // m0: first row of this CTA's 128 in the expert; rows <= 0: none
  int rows_odd;           // even CTA: rows left for the odd one
  int n0, n1;             // tiles
};

struct SmemCtl {
  uint64_t a_empty[kMaxA], full[kMaxB], empty[kMaxB];
  uint64_t sc_full[kSc], sc_empty[kSc];    // scales in shared memory (each CTA its own)
  uint64_t sf_full[kSf], sf_empty[kSf];    // scales in TMEM
  uint64_t tmem_full[2], tmem_empty[2], ovl, drain;
  uint64_t mail_full[2 * kHalf], mail_empty[2];  // claimed tiles, from the odd CTA to both producers
  uint64_t hand_full[2], hand_empty[2];    // and from the producer to the others of its CTA
  uint64_t claim;                          // odd CTA: time to claim the second tile
  int mail[2 * kHalf], hand[2];
  uint64_t stored[2], counted[2];  // an FC1 tile's stores issued; counted for its expert
  uint32_t tmem_base;
  int abort;
  int tstart[2][kMaxE + 1];  // strip prefixes of the two GEMMs
  int off[kMaxE + 1];
};
static_assert(kDynSmem + sizeof(SmemCtl) <= 232448, "shared memory of a CTA");

template <int MODE>
__device__ __forceinline__ int strips(const KParams& p) {  // across an expert
  return (ntiles<MODE>(p) + p.strip[MODE] - 1) / p.strip[MODE];
}
template <int MODE>
__device__ __forceinline__ Strip strip_at(const KParams& p, const SmemCtl& c, int i, int& cursor,
                                          uint32_t rank) {
  const int* tstart = c.tstart[MODE];
  if (tstart[cursor + 1] <= i) {
    int lo = cursor + 1, hi = p.E - 1;  // the first expert that ends past i
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (tstart[mid + 1] <= i) lo = mid + 1;
      else hi = mid;
    }
    cursor = lo;
  }
  Strip t;
  t.e = cursor;
  t.row0 = c.off[cursor];
  const int cnt = c.off[cursor + 1] - t.row0;
  const int local = i - tstart[cursor];
  const int mt = (cnt + 2 * BM - 1) / (2 * BM);
  t.m0 = (local % mt) * 2 * BM + (int)rank * BM;  // row tiles fastest: they share the weights
  t.n0 = (local / mt) * p.strip[MODE];
  t.n1 = min(t.n0 + p.strip[MODE], ntiles<MODE>(p));
  t.rows = min(BM, cnt - t.m0);
  t.rows_odd = rank == 0 ? cnt - t.m0 - BM : 0;
  return t;
}
// First column of h or o of a tile
template <int MODE>
__device__ __forceinline__ int column(int n) { return n * (MODE == FC1 ? 128 : BN); }

__device__ __forceinline__ void give_up(SmemCtl& c, int* status, int where) {
  c.abort = 1;
  atomicExch(status + ST_TIMEOUT, where);
}
template <int REGS>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// ---------------------------------------------------------------- stores
__device__ __forceinline__ void st_sector(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
struct Out {       // one warp's slab of an output
  uint4* buf;      // its shared buffer
  int lane, rows;  // valid rows of the slab
};
// 32 rows (thread i holds row i) x 32 bf16 columns (16 packed words): whole boxes by TMA
// through this warp's buffer, a box that ends with the expert's rows by its threads.
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

// ================================================================ dependences
// An FC2 tile of expert e: wait (bounded) until the expert's FC1 tiles have all stored
// their output.
__device__ __forceinline__ bool wait_expert(SmemCtl& c, const KParams& p, int e) {
  // tiles of the first product, by both CTAs of the pair
  const int target = 2 * ((c.off[e + 1] - c.off[e] + 2 * BM - 1) / (2 * BM)) * ntiles<FC1>(p);
  if (ld_acquire(p.dep + e) < target) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ld_acquire(p.dep + e) < target) {
      if (*(volatile int*)&c.abort || ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
        give_up(c, p.status, 60);
        return false;
      }
    }
  }
  return true;
}

// ================================================================ tiles
// The odd CTA claims for the pair and leaves the tile in a mailbox in each CTA; that CTA's
// producer takes it out and hands it to the others of its CTA. What a mailbox's slot held
// is released to the odd CTA by halves (a release at cluster scope waits for the stores in
// flight on the SM).
//
// What reads the handed tiles of a CTA: counting warp, scale producer, scale and epilogue
// warps, the MMA issuer in the even one.
__device__ __forceinline__ int readers(uint32_t rank) { return 2 + 4 + 8 + (rank == 0); }
// Relaxed: for accesses to TMEM alone, which the tcgen05 fences on both sides order.
__device__ __forceinline__ void arrive_remote(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster)
               : "memory");
}
// The producer: the n-th tile of this pair (at or past the total: none is left; -1: gave up).
__device__ __forceinline__ int mailed_tile(SmemCtl& c, uint32_t n, int* status) {
  const int slot = n % (2 * kHalf);
  const uint32_t round = n / (2 * kHalf);
  if (!mbar_wait_cluster(&c.mail_full[slot], round & 1, &c.abort)) {
    give_up(c, status, 61);
    return -1;
  }
  const int i = *(volatile int*)&c.mail[slot];
  if (slot % kHalf == kHalf - 1)  // the half has been read
    ptx::mbar_arrive_cluster(ptx::mapa_shared(&c.mail_empty[slot / kHalf], 1));
  if (!ptx::mbar_wait(&c.hand_empty[n & 1], ((n >> 1) & 1) ^ 1, &c.abort, kWaitLimitNs)) {
    give_up(c, status, 62);
    return -1;
  }
  *(volatile int*)&c.hand[n & 1] = i;
  ptx::mbar_arrive(&c.hand_full[n & 1]);
  return i;
}
// The others: the n-th tile. Every lane of a warp that passes warp = true calls it together.
__device__ __forceinline__ int handed_tile(SmemCtl& c, uint32_t n, int* status, bool warp) {
  bool ok = ptx::mbar_wait(&c.hand_full[n & 1], (n >> 1) & 1, &c.abort, kWaitLimitNs);
  if (warp) ok = __all_sync(0xffffffffu, ok);
  if (!ok) {
    give_up(c, status, 63);
    return -1;
  }
  const int i = *(volatile int*)&c.hand[n & 1];
  if (warp) __syncwarp();
  if (!warp || (threadIdx.x & 31) == 0) ptx::mbar_arrive(&c.hand_empty[n & 1]);
  return i;
}
__device__ __forceinline__ void mail_tile(SmemCtl& c, int slot, int i) {
  c.mail[slot] = i;
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(ptx::mapa_shared(&c.mail[slot], 0)), "r"(i)
               : "memory");
  ptx::mbar_arrive_cluster(ptx::mapa_shared(&c.mail_full[slot], 0));
  ptx::mbar_arrive_cluster(ptx::mapa_shared(&c.mail_full[slot], 1));
}
// Claims tiles for the pair until none is left (one thread of the odd CTA): those after the
// first, which has been mailed while the tables were made.
__device__ __forceinline__ void claim_tiles(SmemCtl& c, const KParams& p, int first, int total) {
  for (uint32_t n = 1; first < total; ++n) {
    const int slot = n % (2 * kHalf);
    const uint32_t round = n / (2 * kHalf);
    if ((n == 1 && !ptx::mbar_wait(&c.claim, 0, &c.abort, kWaitLimitNs)) ||
        !ptx::mbar_wait(&c.hand_empty[n & 1], ((n >> 1) & 1) ^ 1, &c.abort, kWaitLimitNs) ||
        (slot % kHalf == 0 &&
         !mbar_wait_cluster(&c.mail_empty[slot / kHalf], (round & 1) ^ 1, &c.abort))) {
      give_up(c, p.status, 64);
      return;
    }
    const int i = atomicAdd(p.tile, 1);
    mail_tile(c, slot, i);
    if (i >= total) return;
  }
}

// ================================================================ producer
// The rows of a strip stay in shared memory while its tiles pass: A is loaded, a slot a
// stage, with the first tile's B, and its slots are released by the last tile's MMAs.
// (Rows of more than kMaxA stages stream: a strip is then one tile.) A pair lands 64 KB of
// operands in 512 clocks of MMAs otherwise, and every byte of it takes shared memory's time
// from the tensor cores' own reads.
//
// Bytes of A loaded for a CTA's `rows` valid rows: rows that no expert has are not
// fetched (what the buffer held stays in the unused rows of the product).
__device__ __forceinline__ int a_bytes(int rows) {
  return rows <= 0 ? 0
         : rows > 64 ? kSlotBytes
                     : (rows + kABoxRows - 1) / kABoxRows * kABoxRows * kRowBytes;
}

struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == n) {
      at = 0;
      phase ^= 1;
    }
  }
};

template <int MODE>
__device__ __forceinline__ bool producer_strip(SmemCtl& c, uint8_t* smem, const KParams& p,
                                               const CUtensorMap* tmA, const CUtensorMap* tmS,
                                               const CUtensorMap* tmB, const Strip& t, uint32_t rank,
                                               Ring& ra, Ring& rb) {
  // (the even CTA announces both CTAs' bytes)
  const uint32_t bytes = a_bytes(t.rows) + a_bytes(min(BM, t.rows_odd));
  const int row = t.row0 + t.m0, nk = kstages<MODE>(p);
  // FC1: even CTA 128 gate rows of W1, odd CTA 128 up rows
  const int brow = MODE == FC1 ? (2 * t.e + (int)rank) * p.F : t.e * p.H + 128 * (int)rank;
  if (MODE == FC2) {
    if (!wait_expert(c, p, t.e)) return false;
    // the generic writes it waited for, before the TMA (async-proxy) reads
    asm volatile("fence.proxy.async.global;" ::: "memory");
  }
  for (int n = t.n0; n < t.n1; ++n) {
    for (int kt = 0; kt < nk; ++kt) {
      const int k0 = kt * kRowBytes;
      const bool first = n == t.n0;
      if (!ptx::mbar_wait(&c.empty[rb.at], rb.phase ^ 1, &c.abort, kWaitLimitNs) ||
          (first && !ptx::mbar_wait(&c.a_empty[ra.at], ra.phase ^ 1, &c.abort, kWaitLimitNs))) {
        give_up(c, p.status, 65);
        return false;
      }
      if (rank == 1 && first && kt == nk / 4) ptx::mbar_arrive(&c.claim);
      // both CTAs' loads complete on the even CTA's barrier
      uint64_t* bar = &c.full[rb.at];
      const uint32_t fb = ptx::mapa_shared(bar, 0);
      if (rank == 0) ptx::mbar_arrive_expect_tx(bar, 2 * kSlotBytes + (first ? bytes : 0));
      if (first) {
        uint8_t* sA = smem + ra.at * kSlotBytes;
        if (t.rows > 64) ptx::tma_load_2d_pair(sA, tmA, fb, k0, row);
        else
          for (int r = 0; r < t.rows; r += kABoxRows)
            ptx::tma_load_2d_pair(sA + r * kRowBytes, tmS, fb, k0, row + r);
        ra.next(p.na);
      }
      ptx::tma_load_2d_pair(smem + (p.na + rb.at) * kSlotBytes, tmB, fb, k0, brow + column<MODE>(n));
      rb.next(p.nb);
    }
  }
  return true;
}

// ================================================================ scales
// Into shared memory: the scales of this CTA's rows of A, beside the first tile's, and of
// all 256 rows of B, which the pair's MMA wants whole in both CTAs.
template <int MODE>
__device__ __forceinline__ bool scale_loads(SmemCtl& c, uint8_t* smem, const KParams& p,
                                            const Strip& t, Ring& slot) {
  const int nk = kstages<MODE>(p), R = MODE == FC1 ? p.F : p.H;
  const long long row = (long long)t.row0 + t.m0, np = scale_rows(p.N), r0 = row & ~1ll;
  const uint32_t rows = t.rows <= 0 ? 0 : (((int)(row & 1) + t.rows + 1) & ~1) * 8;
  const uint8_t* sa = (MODE == FC1 ? p.xs : p.hs) + r0 * 8;
  const uint8_t* sb = (MODE == FC1 ? p.w1s : p.w2s) + (size_t)(MODE == FC1 ? 2 * t.e : t.e) * nk * R * 8;
  const size_t up = (size_t)nk * R * 8;
  if (MODE == FC2) {
    if (!wait_expert(c, p, t.e)) return false;
    asm volatile("fence.proxy.async.global;" ::: "memory");
  }
  for (int n = t.n0; n < t.n1; ++n) {
    const int n0 = column<MODE>(n);
    const uint32_t ba = n == t.n0 ? rows : 0;
    // the edge of a matrix may cut its 128 (FC1: of both halves) or 256 rows short
    const uint32_t bb = min(MODE == FC1 ? 128 : 256, R - n0) * 8;
    for (int kt = 0; kt < nk; ++kt) {
      if (!ptx::mbar_wait(&c.sc_empty[slot.at], slot.phase ^ 1, &c.abort, kWaitLimitNs)) {
        give_up(c, p.status, 66);
        return false;
      }
      uint8_t* s = smem + kScAt + slot.at * kScBytes;
      uint64_t* bar = &c.sc_full[slot.at];
      const uint8_t* b = sb + ((size_t)kt * R + n0) * 8;
      ptx::mbar_arrive_expect_tx(bar, ba + (MODE == FC1 ? 2 : 1) * bb);
      if (ba) bulk_load(s, sa + (size_t)kt * np * 8, ba, bar);
      bulk_load(s + kScA, b, bb, bar);
      if (MODE == FC1) bulk_load(s + kScA + 128 * 8, b + up, bb, bar);
      slot.next(kSc);
    }
  }
  return true;
}

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

struct ScaleState {
  Ring slot, a;
  uint32_t group = 0;
};
// Into TMEM: row r of an operand is lane r % 32, column r / 32; a cell holds four scales,
// half a stage's. A's stay for the strip, as its rows do.
template <int MODE>
__device__ __forceinline__ bool scales_strip(SmemCtl& c, const uint8_t* smem, const KParams& p,
                                             const Strip& t, uint32_t tmem, uint32_t rank,
                                             ScaleState& m, int quarter, int lane) {
  const int nk = kstages<MODE>(p);
  const int odd = (t.row0 + t.m0) & 1;
  const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
  for (int n = t.n0; n < t.n1; ++n) {
    for (int kt = 0; kt < nk; ++kt, ++m.group) {
      const int buf = m.group % kSf;
      bool got = ptx::mbar_wait(&c.sc_full[m.slot.at], m.slot.phase, &c.abort, kWaitLimitNs);
      const uint8_t* s = smem + kScAt + m.slot.at * kScBytes;
      uint32_t a[8], b[16];  // the first half's cells, the second's
      if (n == t.n0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint2 v = *reinterpret_cast<const uint2*>(s + (odd + 32 * i + lane) * 8);
          a[i] = v.x;
          a[4 + i] = v.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint2 v = *reinterpret_cast<const uint2*>(s + kScA + (32 * i + lane) * 8);
        b[i] = v.x;
        b[8 + i] = v.y;
      }
      got = got && ptx::mbar_wait(&c.sf_empty[buf], ((m.group / kSf) & 1) ^ 1, &c.abort, kWaitLimitNs);
      if (n == t.n0)
        got = got && ptx::mbar_wait(&c.a_empty[m.a.at], m.a.phase ^ 1, &c.abort, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, got)) {
        if (lane == 0) give_up(c, p.status, 67);
        return false;
      }
      __syncwarp();  // every lane has read the slot
      if (lane == 0) ptx::mbar_arrive(&c.sc_empty[m.slot.at]);
      ptx::tc_fence_after();  // the MMAs that read these columns are done
      if (n == t.n0) {
        tmem_st_x8(lanes + kTmemA + 8 * m.a.at, a);
        m.a.next(p.na);
      }
      tmem_st_x16(lanes + kTmemB + 16 * buf, b);
      tmem_st_wait();
      release(&c.sf_full[buf], rank, lane);
      m.slot.next(kSc);
    }
  }
  return true;
}

// ================================================================ MMA issuer
struct MmaState {
  Ring a, b;
  uint32_t group = 0, tiles = 0;
};
template <int MODE>
__device__ __forceinline__ bool mma_strip(SmemCtl& c, uint32_t smem, const KParams& p, const Strip& t,
                                          uint32_t tmem, MmaState& m) {
  constexpr uint32_t idesc = idesc_mxf4(2 * BM, BN);
  const uint64_t desc0 = ptx::sdesc_sw128(0, 16, 1024);
  const int K = kvalues<MODE>(p), nk = kstages<MODE>(p);
  int where = 0;
  // One lane waits and issues for the whole strip. Last it waits for the columns that an
  // accumulator shares with the previous tile's, which come free last.
  if (elect_one()) {
    MmaState s = m;
    for (int n = t.n0; n < t.n1 && !where; ++n, ++s.tiles) {
      const int acc = s.tiles & 1;
      const uint32_t d = tmem + acc * kAccStep;
      Ring a = m.a;  // the strip's rows, for every tile from the first stage on
      for (int kt = 0; kt < nk; ++kt, ++s.group) {
        const int buf = s.group % kSf;
        if (!ptx::mbar_wait(&c.sf_full[buf], (s.group / kSf) & 1, &c.abort, kWaitLimitNs)) where = 68;
        else if (!ptx::mbar_wait(&c.full[s.b.at], s.b.phase, &c.abort, kWaitLimitNs)) where = 69;
        else if (kt == 0 &&
                 (!ptx::mbar_wait(&c.tmem_empty[acc], ((s.tiles >> 1) & 1) ^ 1, &c.abort, kWaitLimitNs) ||
                  (s.tiles > 0 && !ptx::mbar_wait(&c.ovl, (s.tiles - 1) & 1, &c.abort, kWaitLimitNs))))
          where = 70;
        if (where) break;
        ptx::tc_fence_after();
        const uint32_t sa = tmem + kTmemA + 8 * a.at, sb = tmem + kTmemB + 16 * buf;
        const uint64_t ad = desc0 | ((smem + a.at * kSlotBytes) >> 4);
        const uint64_t bd = desc0 | ((smem + (p.na + s.b.at) * kSlotBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {  // 64 K values each; past the edge there are none
          if (kt * BK + kk * 64 >= K) break;
          umma_mxf4_pair(d, ad + kk * 2, bd + kk * 2, idesc | (kk & 1 ? kUpperPair : 0),
                         sa + 4 * (kk >> 1), sb + 8 * (kk >> 1), (kt | kk) != 0);
        }
        ptx::umma_commit_pair(&c.empty[s.b.at], 3);
        ptx::umma_commit_pair(&c.sf_empty[buf], 3);
        if (n == t.n1 - 1) ptx::umma_commit_pair(&c.a_empty[a.at], 3);
        if (kt == nk - 1) ptx::umma_commit_pair(&c.tmem_full[acc], 3);
        a.next(p.na);
        s.b.next(p.nb);
      }
    }
  }
  where = __reduce_max_sync(0xffffffffu, where);
  if (where) {
    give_up(c, p.status, where);
    return false;
  }
  // where the issuing lane stands, for all
  const int tiles = t.n1 - t.n0, steps = tiles * nk;
  m.group += steps;
  m.tiles += tiles;
  const int b = m.b.at + steps, a = m.a.at + nk;
  m.b.phase ^= (b / p.nb) & 1;
  m.b.at = b % p.nb;
  m.a.phase ^= (a / p.na) & 1;
  m.a.at = a % p.na;
  return true;
}

// ================================================================ epilogue
// 32 columns of h from g and u (fp32): a, h in bf16 where kept, codes and their scale byte.
struct HOut {
  const Out& out;
  const Maps& m;
  const KParams& p;
  size_t row0;  // the slab's first row
};
__device__ __forceinline__ uint32_t swiglu_block(const HOut& ho, const uint32_t (&g)[32],
                                                 const uint32_t (&u)[32], int f, uint32_t* q) {
  const KParams& p = ho.p;
  float h[32], mx = 0.f;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float gf = __uint_as_float(g[j]);
    h[j] = gf * sigmoid_f(gf) * __uint_as_float(u[j]);
    mx = absmax_nan(mx, h[j]);
  }
  uint32_t w[16];
  if (p.a) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      w[j] = pack_bf16x2(__uint_as_float(g[2 * j]), __uint_as_float(g[2 * j + 1]));
    store_box(ho.out, &ho.m.o1, w, p.a, ho.row0, 2 * p.F, f);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      w[j] = pack_bf16x2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
    store_box(ho.out, &ho.m.o1, w, p.a, ho.row0, 2 * p.F, p.F + f);
  }
  if (p.h) {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(h[2 * j], h[2 * j + 1]);
    store_box(ho.out, &ho.m.o2, w, p.h, ho.row0, p.F, f);
  }
  const uint32_t b = fp4_scale_byte(__float_as_uint(mx));
  const float inv = fp4_inv_scale(b);
#pragma unroll
  for (int j = 0; j < 32; ++j) h[j] *= inv;
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = fp4x8(h + 8 * j);
  return b;
}

// Hands an FC1 tile, the n-th of this CTA, to the counting warp, which has counted the one
// before the last.
__device__ __forceinline__ void hand_over(SmemCtl& c, const KParams& p, uint32_t n, int lane) {
  __syncwarp();
  if (lane == 0) {
    if (!ptx::mbar_wait(&c.counted[n & 1], ((n >> 1) & 1) ^ 1, &c.abort, kWaitLimitNs))
      give_up(c, p.status, 71);
    ptx::mbar_arrive(&c.stored[n & 1]);
  }
  __syncwarp();
}

// The columns that the two accumulators share are the first one's last 128 and the
// second one's first 128: an epilogue starts with the higher half of its columns on the
// first accumulator (rev = 1) and with the lower half on the second, and releases them as
// soon as they are in registers.
template <int MODE>
__device__ __forceinline__ bool epilogue_tile(SmemCtl& c, uint4* buf, const KParams& p,
                                              const Maps& m, const Strip& t, int n0, uint32_t tmem,
                                              uint32_t rank, uint32_t& tiles, int ew, int lane) {
  const int q = ew & 3, hf = ew >> 2;
  const int acc = tiles & 1, rev = acc ^ 1;
  const size_t row0 = (size_t)t.row0 + t.m0 + q * 32, row = row0 + lane;  // this warp's, thread's
  const bool rok = q * 32 + lane < t.rows;
  const Out out = {buf, lane, t.rows - q * 32};
  if (!ptx::mbar_wait(&c.tmem_full[acc], (tiles >> 1) & 1, &c.abort, kWaitLimitNs)) {
    if (lane == 0) give_up(c, p.status, 72);
    return false;
  }
  __syncwarp();
  ptx::tc_fence_after();
  const uint32_t tbase = tmem + acc * kAccStep + ((uint32_t)(q * 32) << 16) + 64 * hf;
  if (q * 32 >= t.rows) {  // nothing to store (both warps of the quarter)
    release(&c.ovl, rank, lane);
    release(&c.tmem_empty[acc], rank, lane);
  } else if (MODE == FC1) {
    // columns 0..127 gate, 128..255 up of one 128-wide block of h; this warp's 64 of each,
    // the shared ones (up on the first accumulator, gate on the second) first
    uint32_t s0[32], s1[32], o[32], codes[8], b[2];
    const int f = n0 + 64 * hf;
    const bool ok = f < p.F;  // F is a multiple of 64
    const HOut ho = {out, m, p, row0};
    ptx::tmem_ld_32x32b_x32(tbase + 128 * rev, s0);
    ptx::tmem_ld_32x32b_x32(tbase + 128 * rev + 32, s1);
    ptx::tmem_ld_wait(s0, s1);
    release(&c.ovl, rank, lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t(&s)[32] = i ? s1 : s0;
      ptx::tmem_ld_32x32b_x32(tbase + 128 * (rev ^ 1) + 32 * i, o);
      ptx::tmem_ld_wait(o);
      if (i == 1) release(&c.tmem_empty[acc], rank, lane);
      if (!ok) continue;
      b[i] = rev ? swiglu_block(ho, o, s, f + 32 * i, codes + 4 * i)
                 : swiglu_block(ho, s, o, f + 32 * i, codes + 4 * i);
    }
    if (ok && rok) {
      const int blk = f >> 5;
      st_sector(p.hq + (row * p.F + f) / 2, codes);
      *reinterpret_cast<uint16_t*>(p.hs + ((size_t)(blk >> 3) * scale_rows(p.N) + row) * 8 + (blk & 7)) =
          (uint16_t)(b[0] | b[1] << 8);
    }
  } else {
    // plain fp32 tile -> bf16; the other half's TMEM loads run beside the stores
    uint32_t v[2][32];
    ptx::tmem_ld_32x32b_x32(tbase + 128 * rev, v[0]);
    ptx::tmem_ld_32x32b_x32(tbase + 128 * rev + 32, v[1]);
    ptx::tmem_ld_wait(v[0], v[1]);
    release(&c.ovl, rank, lane);
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
      if (i < 2) ptx::tmem_ld_32x32b_x32(tbase + 128 * (rev ^ 1) + 32 * i, v[i]);
      if (n0 + col < p.H) store_box(out, &m.o3, w, p.o, row0, p.H, n0 + col);
    }
  }
  if (MODE == FC1) hand_over(c, p, tiles, lane);
  ++tiles;
  return true;
}

// ================================================================ counting
// Counts an FC1 tile for its expert once the epilogue's stores are visible device-wide:
// the fence takes thousands of clocks with stores in flight, which the epilogue warps
// spend on the next tile.
__device__ __forceinline__ bool count_tile(SmemCtl& c, const KParams& p, int e, uint32_t& tiles) {
  const int acc = tiles & 1;
  if (!ptx::mbar_wait(&c.stored[acc], (tiles >> 1) & 1, &c.abort, kWaitLimitNs)) {
    give_up(c, p.status, 73);
    return false;
  }
  __threadfence();
  atomicAdd(p.dep + e, 1);
  ptx::mbar_arrive(&c.counted[acc]);
  ++tiles;
  return true;
}

__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_fp4_kernel(const __grid_constant__ Maps m, const KParams p) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ SmemCtl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) &
                                             ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E;
  const uint32_t rank = ptx::cluster_ctarank();
  if (warp == 0) {  // a lane inits the barriers of its number
    auto init = [&](uint64_t* b, int n, uint32_t count) {
      if (lane < n) ptx::mbar_init(b + lane, count);
    };
    init(ctl.a_empty, kMaxA, 1);
    init(ctl.full, kMaxB, 1);
    init(ctl.empty, kMaxB, 1);
    init(ctl.sc_full, kSc, 1);
    init(ctl.sc_empty, kSc, 4);   // this CTA's scale warps
    init(ctl.sf_full, kSf, 8);    // both CTAs' scale warps
    init(ctl.sf_empty, kSf, 1);
    init(ctl.tmem_full, 2, 1);
    init(ctl.tmem_empty, 2, 16);  // both CTAs' epilogue warps
    init(&ctl.ovl, 1, 16);
    init(&ctl.drain, 1, 1);
    init(ctl.mail_full, 2 * kHalf, 1);
    init(ctl.mail_empty, 2, 2);   // (the odd CTA's) both producers
    init(ctl.hand_full, 2, 1);
    init(ctl.hand_empty, 2, readers(rank));
    init(&ctl.claim, 1, 1);
    init(ctl.stored, 2, 8);       // this CTA's epilogue warps
    init(ctl.counted, 2, 1);
    if (lane == 0) ctl.abort = 0;
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
  if (warp == 1 && lane == 0 && rank == 1) {
    first = atomicAdd(p.tile, 1);
    mail_tile(ctl, 0, first);
  }
  // offsets outside 0..N would send stores out of the buffers
  for (int e = threadIdx.x; e <= E; e += blockDim.x)
    ctl.off[e] = (int)min(max((long long)p.off[e], 0ll), p.N);
  __syncthreads();
  if (warp < 2) {  // strips per expert -> exclusive prefix, one warp for each GEMM
    const int nt = warp == 0 ? strips<FC1>(p) : strips<FC2>(p);
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
  auto strip1 = [&](int i) { return strip_at<FC1>(p, ctl, i, cur1, rank); };
  auto strip2 = [&](int i) { return strip_at<FC2>(p, ctl, i - total1, cur2, rank); };
  bool ok = true;
  if (warp < 4) {
    regs_dec<kRegsControl>();
    if (warp == 0 && lane == 0) {
      Ring ra, rb;
      for (uint32_t n = 0; ok; ++n) {
        const int i = mailed_tile(ctl, n, p.status);
        ok = i >= 0;
        if (!ok || i >= total) break;
        ok = i < total1
                 ? producer_strip<FC1>(ctl, smem, p, &m.a1, &m.s1, &m.b1, strip1(i), rank, ra, rb)
                 : producer_strip<FC2>(ctl, smem, p, &m.a2, &m.s2, &m.b2, strip2(i), rank, ra, rb);
      }
      if (!ok && rank == 0) drain_loads(ctl.full, p.nb, rb.at, rb.phase);  // both CTAs'
    } else if (warp == 1 && rank == 0) {
      MmaState st;
      for (uint32_t n = 0; ok; ++n) {
        const int i = handed_tile(ctl, n, p.status, true);
        ok = i >= 0;
        if (!ok || i >= total) break;
        ok = i < total1 ? mma_strip<FC1>(ctl, ptx::smem_u32(smem), p, strip1(i), tmem, st)
                        : mma_strip<FC2>(ctl, ptx::smem_u32(smem), p, strip2(i), tmem, st);
      }
      // no MMA may still run when TMEM is released (the same lane is elected as above)
      __syncwarp();
      if (elect_one()) ptx::umma_commit_pair(&ctl.drain, 1);
      if (!ptx::mbar_wait(&ctl.drain, 0, &ctl.abort, kWaitLimitNs)) {
        int dummy = 0;
        ptx::mbar_wait(&ctl.drain, 0, &dummy, kWaitLimitNs);
      }
    } else if (warp == 1 && lane == 0) {
      claim_tiles(ctl, p, first, total);
    } else if (warp == 2 && lane == 0) {
      uint32_t tiles = 0;
      for (uint32_t n = 0; ok; ++n) {
        const int i = handed_tile(ctl, n, p.status, false);
        ok = i >= 0;
        if (!ok || i >= total) break;
        if (i >= total1) continue;
        const Strip t = strip1(i);
        for (int j = t.n0; j < t.n1 && ok; ++j) ok = count_tile(ctl, p, t.e, tiles);
      }
    } else if (warp == 3 && lane == 0) {
      Ring slot;
      for (uint32_t n = 0; ok; ++n) {
        const int i = handed_tile(ctl, n, p.status, false);
        ok = i >= 0;
        if (!ok || i >= total) break;
        ok = i < total1 ? scale_loads<FC1>(ctl, smem, p, strip1(i), slot)
                        : scale_loads<FC2>(ctl, smem, p, strip2(i), slot);
      }
      if (!ok) drain_loads(ctl.sc_full, kSc, slot.at, slot.phase);
    }
    __syncwarp();
  } else if (warp < 12) {
    regs_inc<kRegsEpilogue>();
    uint32_t tiles = 0;
    const int ew = warp - 4;
    uint4* buf = reinterpret_cast<uint4*>(smem + kEpiAt) + ew * 128;
    for (uint32_t n = 0; ok; ++n) {
      const int i = handed_tile(ctl, n, p.status, true);
      ok = i >= 0;
      if (!ok || i >= total) break;
      const Strip t = i < total1 ? strip1(i) : strip2(i);
      for (int j = t.n0; j < t.n1 && ok; ++j)
        ok = i < total1
                 ? epilogue_tile<FC1>(ctl, buf, p, m, t, column<FC1>(j), tmem, rank, tiles, ew, lane)
                 : epilogue_tile<FC2>(ctl, buf, p, m, t, column<FC2>(j), tmem, rank, tiles, ew, lane);
    }
    // the buffers and the outputs must outlive the TMA stores
    if (lane == 0) ptx::bulk_wait_group0();
    __syncwarp();
  } else {
    regs_dec<kRegsControl>();
    ScaleState st;
    for (uint32_t n = 0; ok; ++n) {
      const int i = handed_tile(ctl, n, p.status, true);
      ok = i >= 0;
      if (!ok || i >= total) break;
      ok = i < total1 ? scales_strip<FC1>(ctl, smem, p, strip1(i), tmem, rank, st, warp - 12, lane)
                      : scales_strip<FC2>(ctl, smem, p, strip2(i), tmem, rank, st, warp - 12, lane);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::cluster_sync();  // the peer may still arrive on this CTA's barriers
  if (warp == 1) ptx::tmem_dealloc_pair(tmem, kTmemCols);
}

// ------------------------------------------------------------------ host side
void cluster_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* at, int pairs, cudaStream_t st) {
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = MOE_PDL;
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kDynSmem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
}

// How many pairs can be resident at once on the current device, after setting
// the kernel's shared memory up there (once for each device).
cudaError_t resident_pairs(int* pairs) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*pairs = known[dev].load()) > 0) return cudaSuccess;
  e = cudaFuncSetAttribute(grouped_gemm_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kDynSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  cluster_config(cfg, at, device_sm_count() / 2, 0);
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(pairs, grouped_gemm_fp4_kernel, &cfg);
  if (e == cudaSuccess && *pairs < 1) e = cudaErrorLaunchOutOfResources;
  if (e == cudaSuccess && dev < 64) known[dev].store(*pairs);
  return e;
}

}  // namespace

moe_status_t launch_ffn_fwd_fp4(const moe_layer_desc_t& d, const uint8_t* xq, const uint8_t* xs,
                                const int32_t* off, const Fp4Weights& w, bf16* a, bf16* h,
                                uint8_t* hq, uint8_t* hs, bf16* o, int* status, int* dep,
                                cudaStream_t st, bool counters_zeroed) {
  const long long N = (long long)d.T * d.k;
  if (N == 0) return MOE_OK;
  if (N <= kFp4FewRows * d.E)
    return launch_ffn_rows_fp4(d, xq, xs, off, w, a, h, hq, hs, o, status, dep, st,
                               counters_zeroed);
  Maps m = {};
  if (!make_map(&m.a1, xq, 2, d.H / 2, N, 1, BM, 1) ||
      !make_map(&m.s1, xq, 2, d.H / 2, N, 1, kABoxRows, 1) ||
      !make_map(&m.b1, w.w1q, 2, d.H / 2, 2ll * d.E * d.F, 1, 128, 1) ||
      !make_map(&m.a2, hq, 2, d.F / 2, N, 1, BM, 1) ||
      !make_map(&m.s2, hq, 2, d.F / 2, N, 1, kABoxRows, 1) ||
      !make_map(&m.b2, w.w2q, 2, d.F / 2, (long long)d.E * d.H, 1, 128, 1) ||
      !make_rows_map(&m.o3, o, N, d.H, 32) || (a && !make_rows_map(&m.o1, a, N, 2 * d.F, 32)) ||
      (h && !make_rows_map(&m.o2, h, N, d.F, 32)))
    return MOE_ERR_CUDA;
  KParams p = {d.E, d.H, d.F, N, off, xs, w.w1s, w.w2s, a, h, o, hq, hs,
               status, dep, tile_counter(status)};
  // A's slots hold the longer product's rows where they can, half of all where not
  const int stages = std::max(fp4_groups(d.H), fp4_groups(d.F));
  p.na = stages <= kMaxA ? std::max(stages, kSlots - kMaxB) : kSlots / 2;
  p.nb = kSlots - p.na;
  const long long rt = std::max<long long>(1, N / (2 * BM));  // row tiles, at the least
  int pairs = 0;
  cudaError_t e = resident_pairs(&pairs);
  if (e == cudaSuccess && !counters_zeroed) e = launch_zero_counters(dep, d.E, p.tile, st);
  if (e != cudaSuccess) {
    set_error("grouped_gemm_fp4_kernel set-up: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  const int nt[2] = {ceil_div(d.F, 128), ceil_div(d.H, BN)}, nk[2] = {fp4_groups(d.H), fp4_groups(d.F)};
  for (int g = 0; g < 2; ++g)
    p.strip[g] = nk[g] > p.na ? 1 : ceil_div(nt[g], std::min(nt[g], ceil_div(kStrips[g] * pairs, rt)));
  // one pair for every two SMs, and no more than there can be tiles
  const long long rows = N / (2 * BM) + std::min<long long>(N, d.E);
  pairs = (int)std::min<long long>(pairs, rows * (ceil_div(d.F, 128) + ceil_div(d.H, BN)));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  cluster_config(cfg, at, pairs, st);
  {
    LaunchScope _ls(K_FP4_FFN_FWD, st);
    e = cudaLaunchKernelEx(&cfg, grouped_gemm_fp4_kernel, m, p);
  }
  if (e != cudaSuccess) {
    set_error("grouped_gemm_fp4_kernel launch: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return check_launch("grouped_gemm_fp4_kernel");
}

}  // namespace moe
