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
// One persistent kernel per GEMM, one CTA per SM, warp-specialised:
//   warp 0      TMA producer of the operand ring (A 128 x 128 B | B 256 x 128 B a stage)
//   warp 1      TMEM allocator + single-thread MMA issuer
//   warp 2      scales: packs the scale bytes of four K blocks (the four bytes
//               of a TMEM cell) into shared memory, ahead of the MMA issuer,
//               which copies them into TMEM (tcgen05.cp)
//   warps 4..11 epilogue: TMEM -> registers -> SwiGLU (or its gradient),
//               rounding, block maxima, e4m3 -> global; two warps per TMEM lane
//               quarter, each owning 64 of every 128 columns
//
// Ragged groups as in the bf16 GEMMs: expert e owns rows off[e]..off[e+1]-1; a
// tile's rows past the expert's end are computed on whatever TMA loaded and
// not stored (rows of A do not mix). Columns past a matrix edge likewise. K past
// an edge must add nothing: maps whose K dimension ends with the expert (or the
// gate or up half) zero-fill it.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "fp8.cuh"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

enum Fp8Mode {
  FC1_FWD = 0,   // a, h, hq = SwiGLU(xq @ W1q^T)
  FC2_FWD = 1,   // o = hq @ W2q^T
  FC2_DGRAD = 2, // da, daq = SwiGLU'(dq @ W2q, a)
  FC1_DGRAD = 3  // dx_perm = daq @ W1q
};

constexpr int BM = 128, BN = 256, BK = 128;
constexpr int kABytes = BM * BK, kBBytes = BN * BK;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kStages = 4;
constexpr int kScaleSlots = 4;                // four-K-block groups of scales in flight
constexpr int kScaleBytes = 512 + 2 * 512;    // A rows, then both 128-column halves of B
constexpr size_t kEpiStageBytes = 8 * 2048;
constexpr int kTmemCols = 512;
constexpr int kTmemScales = 480;              // two buffers of 12 columns
constexpr int kThreads = 384;
constexpr int kMaxE = 256;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr size_t kDynSmem =
    (size_t)kStages * kStageBytes + kScaleSlots * kScaleBytes + kEpiStageBytes + 1024;

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
  const bf16* aux;    // FC2 dgrad: the saved pre-activation
  int* status;
};

template <int MODE>
struct Mode {
  static constexpr bool kBMn = MODE == FC2_DGRAD || MODE == FC1_DGRAD;  // N contiguous in B
  __device__ static int kblocks(const KParams& p) {
    const int nh = (p.H + 127) / 128, nf = (p.F + 127) / 128;
    return MODE == FC1_FWD || MODE == FC2_DGRAD ? nh : MODE == FC2_FWD ? nf : 2 * nf;
  }
  __device__ static int ntiles(const KParams& p) {
    return MODE == FC1_FWD ? (p.F + 127) / 128
                           : ((MODE == FC2_DGRAD ? p.F : p.H) + BN - 1) / BN;
  }
};

struct Tile {
  int e, m0, n0, rows, row0;
};

struct SmemCtl {
  uint64_t full[kStages], empty[kStages];
  uint64_t sf_full[kScaleSlots], sf_empty[kScaleSlots];
  uint64_t tmem_full, tmem_empty, drain;
  uint32_t tmem_base;
  int abort;
  int tstart[kMaxE + 1];
  int off[kMaxE + 1];
  uint32_t amax[2][8][32];  // block maxima handed between the two warps of a quarter
};

template <int MODE>
__device__ __forceinline__ Tile tile_at(const KParams& p, const SmemCtl& c, int tile,
                                        int& cursor) {
  while (c.tstart[cursor + 1] <= tile) ++cursor;
  Tile t;
  t.e = cursor;
  t.row0 = c.off[cursor];
  const int cnt = c.off[cursor + 1] - t.row0;
  const int local = tile - c.tstart[cursor];
  const int mt = (cnt + BM - 1) / BM;
  t.m0 = (local % mt) * BM;
  t.n0 = (local / mt) * (MODE == FC1_FWD ? 128 : BN);
  t.rows = min(BM, cnt - t.m0);
  return t;
}

__device__ __forceinline__ void flag_timeout(SmemCtl& c, int* status, int where) {
  c.abort = 1;
  atomicExch(status + ST_TIMEOUT, where);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}

// s(x) = 1 / (1 + e^-x): relative error near 1e-6 over the whole range
__device__ __forceinline__ float sigmoid_f(float x) {
  return __fdividef(1.f, 1.f + __expf(-x));
}

// ---------------------------------------------------------------- tcgen05, block-scaled
// kind::mxf8f6f4 instruction descriptor: e4m3 operands (format 0), UE8M0 scales
// (bit 23), fp32 D; bits 4-5 and 29-30 select the byte of the scale cells.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N, int b_mn) {
  return ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 4) << 24);
}
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
// 32 rows of 16 bytes from shared memory into four TMEM columns, repeated in
// each warp's 32 lanes
__device__ __forceinline__ void tmem_cp_scales(uint32_t dst, uint32_t saddr) {
  // no swizzle: 8-row groups 128 bytes apart
  const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 16) |
                        ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(dst), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// ---------------------------------------------------------------- stores
// A warp's 32 rows x 64 bytes (thread i holds row i as four 16-byte chunks)
// through its 2 KB buffer, so that each store covers 8 rows x 64 contiguous
// bytes. Chunk c of row r sits at c ^ ((r >> 1) & 3): no bank conflicts.
__device__ __forceinline__ void warp_store64(uint4* stage, const uint4 (&v)[4], uint8_t* base,
                                             size_t pitch, int lane, int valid_rows,
                                             bool cols_ok) {
#pragma unroll
  for (int q = 0; q < 4; ++q) stage[lane * 4 + (q ^ ((lane >> 1) & 3))] = v[q];
  __syncwarp();
  if (cols_ok) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i * 8 + (lane >> 2), c = lane & 3;
      if (row < valid_rows)
        *reinterpret_cast<uint4*>(base + (size_t)row * pitch + c * 16) =
            stage[row * 4 + (c ^ ((row >> 1) & 3))];
    }
  }
  __syncwarp();
}
// 32 bf16 columns held as 16 packed words
__device__ __forceinline__ void warp_store_words(uint4* stage, const uint32_t* w, bf16* base,
                                                 size_t ld, int lane, int valid_rows,
                                                 bool cols_ok) {
  uint4 v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  warp_store64(stage, v, reinterpret_cast<uint8_t*>(base), ld * 2, lane, valid_rows, cols_ok);
}
// 64 bf16 columns (32 packed words) rounded to e4m3
__device__ __forceinline__ void warp_store_fp8(uint4* stage, const uint32_t* w, float inv,
                                               uint8_t* base, size_t ld, int lane, int valid_rows,
                                               bool cols_ok) {
  uint4 v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    v[q] = make_uint4(fp8x4_of_bf16(w[8 * q], w[8 * q + 1], inv),
                      fp8x4_of_bf16(w[8 * q + 2], w[8 * q + 3], inv),
                      fp8x4_of_bf16(w[8 * q + 4], w[8 * q + 5], inv),
                      fp8x4_of_bf16(w[8 * q + 6], w[8 * q + 7], inv));
  warp_store64(stage, v, base, ld, lane, valid_rows, cols_ok);
}

// ================================================================ producer
template <int MODE>
__device__ __forceinline__ bool producer_tile(SmemCtl& c, uint8_t* smem, const KParams& p,
                                              const CUtensorMap* tmA, const CUtensorMap* tmB,
                                              const Tile& t, int& stage, uint32_t& phase) {
  const int nk = Mode<MODE>::kblocks(p), nf = (p.F + 127) / 128;
  for (int kt = 0; kt < nk; ++kt) {
    if (!ptx::mbar_wait(&c.empty[stage], phase ^ 1, &c.abort, kWaitLimitNs)) {
      flag_timeout(c, p.status, 1);
      return false;
    }
    uint8_t* sA = smem + stage * kStageBytes;
    uint8_t* sB = sA + kABytes;
    uint64_t* bar = &c.full[stage];
    const int k0 = kt * BK;
    ptx::mbar_arrive_expect_tx(bar, kStageBytes);
    if (MODE == FC1_FWD) {
      ptx::tma_load_2d(sA, tmA, bar, k0, t.row0 + t.m0);
      ptx::tma_load_2d(sB, tmB, bar, k0, t.e * 2 * p.F + t.n0);                // 128 gate rows
      ptx::tma_load_2d(sB + 16384, tmB, bar, k0, t.e * 2 * p.F + p.F + t.n0);  // 128 up rows
    } else if (MODE == FC2_FWD) {
      ptx::tma_load_2d(sA, tmA, bar, k0, t.row0 + t.m0);
      ptx::tma_load_2d(sB, tmB, bar, k0, t.e * p.H + t.n0);
      ptx::tma_load_2d(sB + 16384, tmB, bar, k0, t.e * p.H + t.n0 + 128);
    } else if (MODE == FC2_DGRAD) {
      ptx::tma_load_2d(sA, tmA, bar, k0, t.row0 + t.m0);
      tma_load_3d(sB, tmB, bar, t.n0, k0, t.e);
      tma_load_3d(sB + 16384, tmB, bar, t.n0 + 128, k0, t.e);
    } else {
      const int half = kt >= nf, kb = (kt - half * nf) * BK;
      tma_load_3d(sA, tmA, bar, kb, half, t.row0 + t.m0);
      tma_load_3d(sB, tmB, bar, t.n0, kb, 2 * t.e + half);
      tma_load_3d(sB + 16384, tmB, bar, t.n0 + 128, kb, 2 * t.e + half);
    }
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
  return true;
}

// ================================================================ scales
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
__device__ __forceinline__ bool scales_tile(SmemCtl& c, uint8_t* sf, const KParams& p,
                                            const Tile& t, uint32_t& group, int lane) {
  const int nk = Mode<MODE>::kblocks(p);
  const uint32_t* words = reinterpret_cast<const uint32_t*>(p.sa);
  const long long r0 = (long long)t.row0 + t.m0;
  for (int g = 0; g * 4 < nk; ++g, ++group) {
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
    const int slot = group % kScaleSlots;
    if (!ptx::mbar_wait(&c.sf_empty[slot], ((group / kScaleSlots) & 1) ^ 1, &c.abort,
                        kWaitLimitNs)) {
      if (lane == 0) flag_timeout(c, p.status, 2);
      return false;
    }
    uint4* dst = reinterpret_cast<uint4*>(sf + slot * kScaleBytes);
    dst[lane] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[32 + lane] = make_uint4(wb[0], wb[0], wb[0], wb[0]);
    dst[64 + lane] = make_uint4(wb[1], wb[1], wb[1], wb[1]);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&c.sf_full[slot]);
  }
  return true;
}

// ================================================================ MMA issuer
template <int MODE>
__device__ __forceinline__ bool mma_tile(SmemCtl& c, uint8_t* smem, uint8_t* sf, const KParams& p,
                                         uint32_t tmem, int& stage, uint32_t& phase,
                                         uint32_t& group, uint32_t& acc_phase) {
  constexpr uint32_t idesc = idesc_mxf8(BM, BN, Mode<MODE>::kBMn);
  constexpr uint32_t b_lbo = Mode<MODE>::kBMn ? 16384 : 16;
  constexpr uint32_t b_adv = Mode<MODE>::kBMn ? (4096 >> 4) : (32 >> 4);
  const int nk = Mode<MODE>::kblocks(p);
  if (!ptx::mbar_wait(&c.tmem_empty, acc_phase ^ 1, &c.abort, kWaitLimitNs)) {
    flag_timeout(c, p.status, 3);
    return false;
  }
  ptx::tc_fence_after();
  uint32_t sfa = 0, sfb = 0;
  for (int kt = 0; kt < nk; ++kt) {
    if ((kt & 3) == 0) {
      // the next four K blocks' scales into the other TMEM buffer, once the
      // MMAs that read it two groups ago are done
      const int slot = group % kScaleSlots;
      bool ok = ptx::mbar_wait(&c.sf_full[slot], (group / kScaleSlots) & 1, &c.abort, kWaitLimitNs);
      if (ok && group >= 2)
        ok = ptx::mbar_wait(&c.sf_empty[(group - 2) % kScaleSlots],
                            ((group - 2) / kScaleSlots) & 1, &c.abort, kWaitLimitNs);
      if (!ok) {
        flag_timeout(c, p.status, 4);
        return false;
      }
      ptx::tc_fence_after();
      sfa = tmem + kTmemScales + (group & 1) * 12;
      sfb = sfa + 4;
      const uint32_t s = ptx::smem_u32(sf + slot * kScaleBytes);
      tmem_cp_scales(sfa, s);
      tmem_cp_scales(sfb, s + 512);
      tmem_cp_scales(sfb + 4, s + 1024);
    }
    if (!ptx::mbar_wait(&c.full[stage], phase, &c.abort, kWaitLimitNs)) {
      flag_timeout(c, p.status, 5);
      return false;
    }
    ptx::tc_fence_after();
    const uint32_t a_addr = ptx::smem_u32(smem + stage * kStageBytes);
    const uint64_t adesc = ptx::sdesc_sw128(a_addr, 16, 1024);
    const uint64_t bdesc = ptx::sdesc_sw128(a_addr + kABytes, b_lbo, 1024);
    const uint32_t id = idesc | ((uint32_t)(kt & 3) << 4) | ((uint32_t)(kt & 3) << 29);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      umma_mxf8(tmem, adesc + (uint64_t)(kk * 2), bdesc + (uint64_t)(kk * b_adv), id, sfa, sfb,
                (kt | kk) != 0);
    ptx::umma_commit(&c.empty[stage]);
    if ((kt & 3) == 3 || kt == nk - 1) {
      ptx::umma_commit(&c.sf_empty[group % kScaleSlots]);
      ++group;
    }
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
  ptx::umma_commit(&c.tmem_full);
  acc_phase ^= 1;
  return true;
}

// ================================================================ epilogue
// Larger of this thread's and its partner warp's block maximum (the same row,
// the other 64 columns), as fp32 bits. buf alternates between calls, so that a
// warp never overwrites a value that its partner has yet to read: it passes the
// next call's barrier only after the partner has read this call's.
__device__ __forceinline__ uint32_t pair_max(SmemCtl& c, uint32_t m, int ew, int lane, int buf) {
  c.amax[buf][ew][lane] = m;
  asm volatile("bar.sync %0, 64;" ::"r"(1 + (ew & 3)) : "memory");
  return max(m, c.amax[buf][ew ^ 4][lane]);
}

// Plain fp32 tile -> bf16: this warp's 32 rows x 64 columns of each 128.
__device__ __forceinline__ void store_plain(uint4* stage, uint32_t tbase, int hf, bf16* slab,
                                            int ld, int n0, int lane, int slab_rows) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int cc = (i >> 1) * 4 + 2 * hf + (i & 1);
    uint32_t v[32];
    ptx::tmem_ld_32x32b_x32(tbase + 32 * cc, v);
    ptx::tmem_ld_wait(v);
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
      w[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
    warp_store_words(stage, w, slab + 32 * cc, ld, lane, slab_rows, n0 + 32 * cc < ld);
  }
}

template <int MODE>
__device__ __forceinline__ bool epilogue_tile(SmemCtl& c, uint8_t* stage_base, const KParams& p,
                                              const Tile& t, uint32_t tmem, uint32_t& acc_phase,
                                              int ew, int lane) {
  const int q = ew & 3, hf = ew >> 2;
  uint4* stage = reinterpret_cast<uint4*>(stage_base) + ew * 128;
  if (!ptx::mbar_wait(&c.tmem_full, acc_phase, &c.abort, kWaitLimitNs)) {
    if (lane == 0) flag_timeout(c, p.status, 6);
    return false;
  }
  ptx::tc_fence_after();
  const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
  const size_t row0 = (size_t)t.row0 + t.m0 + q * 32;  // this warp's 32 rows
  const int slab_rows = min(32, t.rows - q * 32);
  if (MODE == FC1_FWD) {
    // columns 0..127 gate, 128..255 up of one 128-wide block of h
    uint32_t hw[32];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int cc = 2 * hf + i, f = t.n0 + 32 * cc;
      const bool ok = f < p.F;
      uint32_t g[32], u[32];
      ptx::tmem_ld_32x32b_x32(tbase + 32 * cc, g);
      ptx::tmem_ld_32x32b_x32(tbase + 128 + 32 * cc, u);
      ptx::tmem_ld_wait(g, u);
      uint32_t gw[16], uw[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        gw[j] = pack_bf16x2(__uint_as_float(g[2 * j]), __uint_as_float(g[2 * j + 1]));
        uw[j] = pack_bf16x2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
        const float g0 = bf16_lo(gw[j]), g1 = bf16_hi(gw[j]);
        const uint32_t h2 = pack_bf16x2(g0 * sigmoid_f(g0) * bf16_lo(uw[j]),
                                        g1 * sigmoid_f(g1) * bf16_hi(uw[j]));
        hw[16 * i + j] = h2;
        if (ok) mx = absmax_bf16x2(mx, h2);  // columns past F are not part of the block
      }
      if (p.out0) {
        bf16* abase = p.out0 + row0 * (size_t)(2 * p.F);
        warp_store_words(stage, gw, abase + f, 2 * p.F, lane, slab_rows, ok);
        warp_store_words(stage, uw, abase + p.F + f, 2 * p.F, lane, slab_rows, ok);
      }
      if (p.out1)
        warp_store_words(stage, hw + 16 * i, p.out1 + row0 * (size_t)p.F + f, p.F, lane, slab_rows,
                         ok);
    }
    const uint32_t b = fp8_scale_byte(pair_max(c, absmax_bits(mx), ew, lane, acc_phase));
    const int f = t.n0 + 64 * hf, fb = t.n0 / 128;
    warp_store_fp8(stage, hw, fp8_inv_scale(b), p.q + row0 * (size_t)p.F + f, p.F, lane, slab_rows,
                   f < p.F);
    if (hf == 0 && lane < slab_rows)
      p.s[((size_t)(fb >> 2) * p.N + row0 + lane) * 4 + (fb & 3)] = (uint8_t)b;
  } else if (MODE == FC2_DGRAD) {
    const int nf = (p.F + 127) / 128;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {  // 128 columns: one block of da_gate, one of da_up
      if (t.n0 + 128 * half >= p.F) break;
      uint32_t gw[32], uw[32];
      uint32_t mg = 0, mu = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int cc = 4 * half + 2 * hf + i, f = t.n0 + 32 * cc;
        const bool ok = f < p.F;
        uint32_t v[32];
        ptx::tmem_ld_32x32b_x32(tbase + 32 * cc, v);
        uint4 gc[4], uc[4];
        const bool rok = ok && lane < slab_rows;
        const uint4* src =
            reinterpret_cast<const uint4*>(p.aux + (row0 + lane) * (size_t)(2 * p.F) + f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          gc[j] = rok ? __ldg(src + j) : make_uint4(0, 0, 0, 0);
          uc[j] = rok ? __ldg(src + p.F / 8 + j) : make_uint4(0, 0, 0, 0);
        }
        ptx::tmem_ld_wait(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t* gp = reinterpret_cast<const uint32_t*>(gc);
          const uint32_t* up = reinterpret_cast<const uint32_t*>(uc);
          const float d0 = __uint_as_float(v[2 * j]), d1 = __uint_as_float(v[2 * j + 1]);
          const float a0 = bf16_lo(gp[j]), a1 = bf16_hi(gp[j]);
          const float s0 = sigmoid_f(a0), s1 = sigmoid_f(a1);
          uw[16 * i + j] = pack_bf16x2(d0 * a0 * s0, d1 * a1 * s1);
          gw[16 * i + j] = pack_bf16x2(d0 * bf16_lo(up[j]) * s0 * (1.f + a0 * (1.f - s0)),
                                       d1 * bf16_hi(up[j]) * s1 * (1.f + a1 * (1.f - s1)));
          if (ok) {
            mu = absmax_bf16x2(mu, uw[16 * i + j]);
            mg = absmax_bf16x2(mg, gw[16 * i + j]);
          }
        }
        if (p.out0) {
          bf16* dbase = p.out0 + row0 * (size_t)(2 * p.F);
          warp_store_words(stage, gw + 16 * i, dbase + f, 2 * p.F, lane, slab_rows, ok);
          warp_store_words(stage, uw + 16 * i, dbase + p.F + f, 2 * p.F, lane, slab_rows, ok);
        }
      }
      const uint32_t bg = fp8_scale_byte(pair_max(c, absmax_bits(mg), ew, lane, 0));
      const uint32_t bu = fp8_scale_byte(pair_max(c, absmax_bits(mu), ew, lane, 1));
      const int f = t.n0 + 128 * half + 64 * hf;
      uint8_t* qbase = p.q + row0 * (size_t)(2 * p.F);
      warp_store_fp8(stage, gw, fp8_inv_scale(bg), qbase + f, 2 * p.F, lane, slab_rows, f < p.F);
      warp_store_fp8(stage, uw, fp8_inv_scale(bu), qbase + p.F + f, 2 * p.F, lane, slab_rows,
                     f < p.F);
      if (lane < slab_rows) {
        const int kb = hf * nf + t.n0 / 128 + half;  // the gate's byte or the up half's
        p.s[((size_t)(kb >> 2) * p.N + row0 + lane) * 4 + (kb & 3)] = (uint8_t)(hf ? bu : bg);
      }
    }
  } else {
    store_plain(stage, tbase, hf, p.out0 + row0 * (size_t)p.H + t.n0, p.H, t.n0, lane, slab_rows);
  }
  ptx::tc_fence_before();
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(&c.tmem_empty);
  acc_phase ^= 1;
  return true;
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA,
                            const __grid_constant__ CUtensorMap tmB, const KParams p) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ SmemCtl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sf = smem + kStages * kStageBytes;
  uint8_t* stage_base = sf + kScaleSlots * kScaleBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&ctl.full[s], 1);
      ptx::mbar_init(&ctl.empty[s], 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      ptx::mbar_init(&ctl.sf_full[s], 1);
      ptx::mbar_init(&ctl.sf_empty[s], 1);
    }
    ptx::mbar_init(&ctl.tmem_full, 1);
    ptx::mbar_init(&ctl.tmem_empty, 8);
    ptx::mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&ctl.tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    ptx::tma_prefetch_desc(&tmA);
    ptx::tma_prefetch_desc(&tmB);
  }
  pdl_wait();
  // offsets outside 0..N would send stores out of the buffers
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x)
    ctl.off[e] = (int)min(max((long long)p.off[e], 0ll), p.N);
  __syncthreads();
  if (warp == 0) {  // tiles per expert -> exclusive prefix
    int carry = 0;
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      int n = 0;
      if (e < p.E) {
        const int cnt = ctl.off[e + 1] - ctl.off[e];
        n = cnt > 0 ? (cnt + BM - 1) / BM * Mode<MODE>::ntiles(p) : 0;
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (e < p.E) ctl.tstart[e] = carry + incl - n;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) ctl.tstart[p.E] = carry;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  const int total = ctl.tstart[p.E];
  int cursor = 0;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int tile = blockIdx.x; tile < total; tile += gridDim.x)
        if (!producer_tile<MODE>(ctl, smem, p, &tmA, &tmB, tile_at<MODE>(p, ctl, tile, cursor),
                                 stage, phase))
          break;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, group = 0, acc_phase = 0;
      for (int tile = blockIdx.x; tile < total; tile += gridDim.x)
        if (!mma_tile<MODE>(ctl, smem, sf, p, tmem, stage, phase, group, acc_phase)) break;
      // no MMA may still run when TMEM is released
      ptx::umma_commit(&ctl.drain);
      if (!ptx::mbar_wait(&ctl.drain, 0, &ctl.abort, kWaitLimitNs)) {
        int dummy = 0;
        ptx::mbar_wait(&ctl.drain, 0, &dummy, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    uint32_t group = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x)
      if (!scales_tile<MODE>(ctl, sf, p, tile_at<MODE>(p, ctl, tile, cursor), group, lane)) break;
  } else if (warp >= 4) {
    uint32_t acc_phase = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x)
      if (!epilogue_tile<MODE>(ctl, stage_base, p, tile_at<MODE>(p, ctl, tile, cursor), tmem,
                               acc_phase, warp - 4, lane))
        break;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
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
bool make_map(CUtensorMap* m, const void* base, int dims, long long d0, long long d1, long long d2,
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
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, const_cast<void*>(base), dim, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for a %lld x %lld x %lld map", (int)r, d2, d1,
              d0);
    return false;
  }
  return true;
}

template <int MODE>
moe_status_t launch_mode(const moe_layer_desc_t& d, const CUtensorMap& a, const CUtensorMap& b,
                         const KParams& p, cudaStream_t st) {
  // once for each device (the attribute belongs to the device's copy of the kernel)
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t attr = cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (attr == cudaSuccess && !(ready.load() & bit)) {
    attr = cudaFuncSetAttribute(grouped_gemm_fp8_kernel<MODE>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDynSmem);
    if (attr == cudaSuccess) ready.fetch_or(bit);
  }
  if (attr != cudaSuccess) {
    set_error("kernel attribute setup failed: %s", cudaGetErrorString(attr));
    return MOE_ERR_CUDA;
  }
  const int nt = MODE == FC1_FWD ? ceil_div(d.F, 128)
                                 : ceil_div(MODE == FC2_DGRAD ? d.F : d.H, BN);
  const long long tiles = (p.N / BM + (p.N < d.E ? p.N : d.E)) * nt;  // at most
  const int grid = (int)std::min<long long>(device_sm_count(), tiles);
  cudaError_t e;
  {
    LaunchScope _ls(K_FP8_FC1_FWD + MODE, st);
    e = launch_k(grouped_gemm_fp8_kernel<MODE>, grid, kThreads, kDynSmem, st, a, b, p);
  }
  if (e != cudaSuccess) {
    set_error("grouped_gemm_fp8_kernel launch: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return check_launch("grouped_gemm_fp8_kernel");
}

KParams params(const moe_layer_desc_t& d, const int32_t* off, int* status) {
  KParams p = {};
  p.E = d.E;
  p.H = d.H;
  p.F = d.F;
  p.N = (long long)d.T * d.k;
  p.off = off;
  p.status = status;
  return p;
}

}  // namespace

moe_status_t launch_ffn_fwd_fp8(const moe_layer_desc_t& d, const uint8_t* xq, const uint8_t* xs,
                                const int32_t* off, const Fp8Weights& w, bf16* a, bf16* h,
                                uint8_t* hq, uint8_t* hs, bf16* o, int* status, int* dep,
                                cudaStream_t st, bool counters_zeroed) {
  const long long N = (long long)d.T * d.k;
  if (N == 0) return MOE_OK;
  CUtensorMap a1, b1, a2, b2;
  if (!make_map(&a1, xq, 2, d.H, N, 1, BM, 1) ||
      !make_map(&b1, w.w1q, 2, d.H, 2ll * d.E * d.F, 1, 128, 1) ||
      !make_map(&a2, hq, 2, d.F, N, 1, BM, 1) ||
      !make_map(&b2, w.w2q, 2, d.F, (long long)d.E * d.H, 1, 128, 1))
    return MOE_ERR_CUDA;
  KParams p1 = params(d, off, status), p2 = p1;
  p1.sa = xs;
  p1.sb = w.w1s;
  p1.out0 = a;
  p1.out1 = h;
  p1.q = hq;
  p1.s = hs;
  p2.sa = hs;
  p2.sb = w.w2s;
  p2.out0 = o;
  const moe_status_t s = launch_mode<FC1_FWD>(d, a1, b1, p1, st);
  return s != MOE_OK ? s : launch_mode<FC2_FWD>(d, a2, b2, p2, st);
}

moe_status_t launch_ffn_dgrad_fp8(const moe_layer_desc_t& d, const uint8_t* dq, const uint8_t* ds,
                                  const bf16* a, const int32_t* off, const Fp8Weights& w, bf16* da,
                                  uint8_t* daq, uint8_t* das, bf16* dx_perm, int* status, int* dep,
                                  cudaStream_t st, bool counters_zeroed) {
  const long long N = (long long)d.T * d.k;
  if (N == 0) return MOE_OK;
  CUtensorMap a1, b1, a2, b2;
  if (!make_map(&a1, dq, 2, d.H, N, 1, BM, 1) ||
      !make_map(&b1, w.w2q, 3, d.F, d.H, d.E, 128, 1) ||
      !make_map(&a2, daq, 3, d.F, 2, N, 1, BM) ||
      !make_map(&b2, w.w1q, 3, d.H, d.F, 2ll * d.E, 128, 1))
    return MOE_ERR_CUDA;
  KParams p1 = params(d, off, status), p2 = p1;
  p1.sa = ds;
  p1.sb = w.w2s;
  p1.out0 = da;
  p1.aux = a;
  p1.q = daq;
  p1.s = das;
  p2.sa = das;
  p2.sb = w.w1s;
  p2.out0 = dx_perm;
  const moe_status_t s = launch_mode<FC2_DGRAD>(d, a1, b1, p1, st);
  return s != MOE_OK ? s : launch_mode<FC1_DGRAD>(d, a2, b2, p2, st);
}

}  // namespace moe
