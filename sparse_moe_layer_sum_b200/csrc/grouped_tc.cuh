// Grouped products on the tcgen05 tensor cores (bf16 operands, fp32 sums).
//
// Two persistent, warp-specialised kernels fed by TMA.  Warp 0 streams
// operand tiles into a ring of shared-memory stages, one thread of warp 1
// issues the MMAs into tensor memory, and the other warps finish the tiles.
//
// rows_gemm -- results with one row per input row (LIN, DX, UP, BWD).  The
//   weights are the MMA's A operand (128 features per SM and MMA) and the
//   group's rows its B operand, because N is a run-time field of the
//   instruction: a tile spends tensor work only on the rows its group has,
//   rounded up to 16.  LIN and UP contract over the weights' contiguous
//   index (K-major tiles); DX and BWD over the other one, which the MMA
//   reads from MN-major tiles, so no transposed copy of a weight exists.
// dw_gemm -- weight gradients.  The contraction runs over the group's rows,
//   so both operands are MN-major.  A group ends anywhere inside a tile: the
//   rows behind it are zeroed in shared memory up to the next multiple of 16
//   (both operands: the next group may hold infinities), and the MMAs beyond
//   are not issued.
//
// Operands that TMA cannot read or the MMA cannot multiply are staged first
// (stage_rows): bf16 rows off the 16-byte pitch are copied to padded rows, and
// fp32 operands are split into three bf16 terms, x = x0 + x1 + x2 with 8 bits
// of the significand each.  Of the nine products of two split operands the six
// down to 2^-16 are multiplied, as six passes over the contraction into the same
// sums; what is left out is within 2^-25 of a product.  The passes go from the
// smallest products to the largest, but a tile that is not cut into parts may
// begin further on in that round (see the producer).  fp32 products run at a sixth of the bf16 rate that way, still
// several times the CUDA cores' rate.
#pragma once

#include <cuda.h>

#include "ckpt.cuh"
#include "grouped.cuh"
#include "sm100.cuh"

namespace moe {
namespace tcg {

using namespace grouped;
using namespace sm100;

constexpr int BK = 64;               // contraction depth of a stage
constexpr int BM = 128;              // features of one MMA tile and SM
constexpr int BOX = 64 * BK * 2;     // a 64 x 64 box: 8 KB
constexpr int TILE = BM * BK * 2;    // an A tile: 16 KB
constexpr int64_t WAIT_NS = 1000000000LL;

// ------------------------------------------------------------- PTX wrappers

// 3-D tiled load; completion is counted on an mbarrier given by its
// shared::cluster address (CG 2: of either CTA of the pair).
template <int CG>
__device__ __forceinline__ void load_3d(const CUtensorMap *m, void *dst, uint32_t bar, int x, int y,
                                        int z, uint64_t pol) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(pol)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(pol)
        : "memory");
}

template <int CG>
__device__ __forceinline__ void load_2d(const CUtensorMap *m, void *dst, uint32_t bar, int x, int y,
                                        uint64_t pol) {
  if (CG == 2)
    tma_load_2d_pair(m, dst, bar, x, y, pol);
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar), "l"(pol)
        : "memory");
}

__device__ __forceinline__ void store_3d(const CUtensorMap *m, const void *src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}
// The same, added to what is there (fp32, one rounding; the memory system
// flushes subnormal sums to zero).
__device__ __forceinline__ void reduce_3d(const CUtensorMap *m, const void *src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Arrive with cluster-scope release on a barrier of either CTA of the pair.
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// MN-major operand tile as TMA SWIZZLE_128B boxes of 64 (contiguous) x BK
// write it: 8-row groups of the contraction index 1024 bytes apart (stride
// offset), the next 64 contiguous values one box further (leading offset).
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((uint32_t)BOX >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t A_MN = 1u << 15, B_MN = 1u << 16;  // instruction descriptor: MN-major operands

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (CG == 2)
    mma_bf16_pair(d, a, b, idesc, acc);
  else
    mma_bf16(d, a, b, idesc, acc);
}
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar) {  // CG 2: on both CTAs' barriers
  if (CG == 2)
    mma_commit_pair_mc(bar, 0x3);
  else
    mma_commit(bar);
}

// Waits for copies or MMAs in flight before the block leaves, with a limit
// but regardless of the abort flag.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if ((int64_t)(globaltimer_ns() - t0) > WAIT_NS) break;
}
__device__ __forceinline__ void pause_ns(int64_t ns) {
  const uint64_t t0 = globaltimer_ns();
  while ((int64_t)(globaltimer_ns() - t0) < ns) {
  }
}

// Register split of the blocks with eight epilogue warps: the first four warps
// (producer, MMA issuer, two idle) give theirs to the epilogue, which keeps
// 128 sums per thread.  4 * 72 + 8 * 216 = 12 * 168, the count at launch.
constexpr int REG_LAUNCH = 168, REG_LOW = 72, REG_HIGH = 216;
static_assert(4 * REG_LOW + 8 * REG_HIGH == 12 * REG_LAUNCH, "register split");
__device__ __forceinline__ void regs_low() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOW));
}
__device__ __forceinline__ void regs_high() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_HIGH));
}

// A whole warp waits: lane 0 polls and tells the others, so that the lanes
// cannot disagree about a wait that runs out.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort,
                                          int32_t *status) {
  int ok = 1;
  if (threadIdx.x % 32 == 0) ok = wait_bounded(bar, parity, abort, WAIT_NS, status);
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {  // bf16x2, rounded to nearest
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}

struct Ring {  // position in a ring of stages
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ uint8_t *align_smem(uint8_t *raw) {
  return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                     ~static_cast<uintptr_t>(1023));
}

// -------------------------------------------------------------------- staging

constexpr int SPLIT_TERMS = 3, SPLIT_PASSES = 6;

// Terms of the two operands that pass q multiplies, from the smallest products
// to the largest.
__device__ __forceinline__ int term_a(int q) { return (0x118 >> (2 * q)) & 3; }  // 0 2 1 0 1 0
__device__ __forceinline__ int term_b(int q) { return (0x052 >> (2 * q)) & 3; }  // 2 0 1 1 0 0

// src [rows, k] into TERMS planes [rows, kp] of bf16, kp = k rounded up to 8,
// zeros behind k.  One term is a copy (bf16 src).  A value that is not finite
// stays in the first term alone.  A finite one above bf16's largest, which
// would round to infinity, takes that largest as its first term and leaves the
// rest to the others.  Bits below 2^-133, bf16's smallest step, are lost.
constexpr float BF16_MAX = 0x1.fep127f;
template <typename TI, int TERMS>
__global__ void __launch_bounds__(256) stage_rows(const TI *__restrict__ src, int64_t rows, int k,
                                                  int kp, bf16 *__restrict__ dst) {
  const int64_t per = kp / 8, total = rows * per, plane = rows * kp;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = ckpt::item_row(i, (int)per);
    const int c = (int)(i - r * per) * 8;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < k ? to_f(src[r * k + c + j]) : 0.0f;
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      uint32_t w[4];
      float q[8];  // what is rounded
#pragma unroll
      for (int j = 0; j < 8; ++j)
        q[j] = TERMS > 1 && t == 0 && isfinite(v[j]) ? fminf(fmaxf(v[j], -BF16_MAX), BF16_MAX) : v[j];
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(q[j], q[j + 1]);
        w[j / 2] = *reinterpret_cast<const uint32_t *>(&h);
        if (t + 1 < TERMS) {
          const float2 f = __bfloat1622float2(h);
          v[j] = isfinite(f.x) ? v[j] - f.x : 0.0f;  // exact
          v[j + 1] = isfinite(f.y) ? v[j + 1] - f.y : 0.0f;
        }
      }
      *reinterpret_cast<uint4 *>(dst + t * plane + r * kp + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ----------------------------------------------------------------- rows_gemm

enum Op { LIN, DX, UP, BWD };

struct RowParams {
  const int32_t *offsets;
  int G, F;          // F: features (columns of the result)
  int kb0, kb;       // k-blocks of one pass, of all passes of all sources
  int passes;        // 1, or SPLIT_PASSES for split operands
  int splits;        // LIN, DX: parts of the contraction, each with its own out
  int vec;           // UP, BWD: rows of the results in whole vectors of 4
  int64_t rows;
  void *out;         // LIN, DX: [rows, F]; UP: h
  int32_t *status;
  ckpt::Saved saved;  // UP: written; BWD: read
  const float *gate;  // BWD, may be NULL
  void *da, *du, *hg;
  float *part;        // BWD: [ceil(F / 32), rows] terms of dgate
};

// Depth after which a partial sum leaves tensor memory and is added to the
// others in fp32 registers.  The tensor cores cut a sum off at 2^-24 of its
// size with every 16-deep MMA, always towards zero: 8e-6 of the result after
// 7168 values, 5e-7 after 512.  fp32 results, and 8-bit codes next to a rounding
// border, show it; results that are rounded to bf16 do not until the sum is
// long: LONG_SUM values of one sign lose some 2^-12, a sixteenth of bf16's own
// half step, and longer sums leave tensor memory too.
constexpr int SEG = 512 / BK;
constexpr int LONG_SUM = 1 << 16;

// k-blocks of the i-th segment of a tile of nkb.  BWD ends a tile with
// arithmetic that takes the MMAs of several segments, and the MMAs may run two
// segments ahead of it: in a long contraction its first two are twice as long
// (6% less time over 32 groups, 16384 rows; error 6e-7 instead of 5e-7).
// UP's codes change with the sums' last bits near a border. Over a short
// contraction, where plain fp32 sums are better than that, its segments are
// shorter: of 1e9 codes of a 256-deep contraction 3200 differ from exact sums'
// codes with 64 values a segment, 4400 with 128, 7000 with 256 and 4000 with
// plain fp32 sums; 512 deep 5000 with 128, 8300 with 256 and 5900 with plain
// sums. It costs time only where the read-out shows, in many rows (16 groups,
// 16000 rows, to 1024: from 512 102 us with 128, 89 with 256; from 256 92 with
// 64, 79 with 256; 8 groups, 2000 rows, 256 -> 256 12.9 and 12.5).
template <int OP>
__device__ __forceinline__ int segment(int i, int nkb) {
  if (OP == UP && nkb <= 32) return nkb <= 4 ? SEG / 8 : nkb <= 8 ? SEG / 4 : SEG / 2;
  return OP == BWD && i < 2 && nkb >= 64 ? 2 * SEG : SEG;
}

// CG: SMs per tile.  AT: A tiles per SM (UP: one of w1 and the same rows of
// w3; LIN, DX: two blocks of features, which halves the row bytes each weight
// byte is paired with).  BN: rows of a tile.  SEGS: sums in segments; the
// registers of the epilogue hold 128 x 256 of them per SM.
template <int OP, int CG, int AT, int BN, int STAGES, bool SEGS>
struct RowCfg {
  static constexpr bool KMAJOR = OP == LIN || OP == UP;
  static constexpr int EPI = BN >= 128 ? 8 : 4;  // epilogue warps
  static constexpr int NT = 32 * (4 + EPI);      // warps 2 and 3 idle
  static constexpr int BROWS = BN / CG;  // rows of the B tile in one SM
  static constexpr int BOXN = BROWS < 32 ? BROWS : 32;
  static constexpr int A_ALL = AT * TILE;
  static constexpr int STAGE = A_ALL + BROWS * BK * 2;
  static constexpr int FEAT = (OP == UP ? BM : AT * BM) * CG;
  static constexpr int ACC = AT * BN;
  static constexpr int NBUF = 2 * ACC <= 512 ? 2 : 1;
  static constexpr int COLS = NBUF * ACC;
  static constexpr uint32_t TMEM = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr int XBUF = STAGES * STAGE;  // UP, BWD: 2 KB per epilogue warp
  static constexpr int BAR = XBUF + (OP == UP || OP == BWD ? EPI * 2048 : 0);
  static constexpr int NBARS = 2 * STAGES + 5;
  static constexpr int MISC = BAR + NBARS * 8;
  static constexpr int TAB = (MISC + 16 + 4 * STAGES + 15) / 16 * 16;
  static size_t smem(int G) { return 1024 + TAB + Table::bytes(G); }
  static_assert(BROWS % BOXN == 0 && BOXN % 8 == 0, "row boxes");
  static_assert(NBUF * ACC <= 512, "tensor memory columns");
  static constexpr int STEP = 32 * (EPI / 4);   // between a warp's 32-row chunks
  static constexpr int NCH = BN / STEP;         // chunks of a warp and A tile
  static_assert(SEGS || NCH % 2 == 0, "chunks are read in pairs");
  static_assert(OP != UP || AT == 2, "UP pairs w1 and w3");
  static_assert(OP != BWD || AT == 1, "BWD finishes one A tile");
  static_assert((OP != UP && OP != BWD) || SEGS, "UP and BWD finish from registers");
  static_assert(!SEGS || (NBUF == 2 && AT * NCH <= 4), "sums in registers");
};

// The result of one accumulator chunk: lane l holds feature fw + l of the 32
// rows from row0 on, the first nv of which belong to the tile.

template <typename TO>
__device__ __forceinline__ void finish_rows(const RowParams &p, int part, const float (&v)[32], int fw,
                                            int row0, int nv) {
  const int f = fw + threadIdx.x % 32;
  if (f >= p.F) return;
  TO *o = static_cast<TO *>(p.out) + ((size_t)part * p.rows + row0) * p.F + f;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (j < nv) *o = from_f<TO>(v[j]);
    o += p.F;
  }
}

// The same from bf16 pairs: row 2 e in the low half of w[e].
__device__ __forceinline__ void finish_packed(const RowParams &p, const uint32_t (&w)[16], int fw,
                                              int row0, int nv) {
  const int f = fw + threadIdx.x % 32;
  if (f >= p.F) return;
  uint16_t *o = static_cast<uint16_t *>(p.out) + (size_t)row0 * p.F + f;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (j < nv) *o = (uint16_t)(j % 2 ? w[j / 2] >> 16 : w[j / 2] & 0xffffu);
    o += p.F;
  }
}

// UP and BWD finish a few rows of a chunk at a time from shared memory, where
// a lane takes 4 consecutive features of one row and a warp 4 rows: whole
// words of codes, 8-byte vectors of results, and one copy of the code in a
// rolled loop (straight-line code for 128 sums per lane stalled on
// instruction fetches).  x: [rows][32 features] of this warp.

template <typename T>
__device__ __forceinline__ void put4(void *base, size_t at, const float (&v)[4], int left, bool vec);
template <>
__device__ __forceinline__ void put4<bf16>(void *base, size_t at, const float (&v)[4], int left, bool vec) {
  bf16 *o = static_cast<bf16 *>(base) + at;
  if (vec) {
    *reinterpret_cast<uint2 *>(o) = make_uint2(pack(v[0], v[1]), pack(v[2], v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) o[i] = __float2bfloat16_rn(v[i]);
  }
}
template <>
__device__ __forceinline__ void put4<float>(void *base, size_t at, const float (&v)[4], int left, bool vec) {
  float *o = static_cast<float *>(base) + at;
  if (vec) {
    *reinterpret_cast<float4 *>(o) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) o[i] = v[i];
  }
}
__device__ __forceinline__ void put4_codes(uint8_t *o, const float (&v)[4], float inv, int left, bool vec) {
  const uint32_t w = (uint32_t)f32x2_to_e4m3x2(ckpt::scaled(v[0], inv), ckpt::scaled(v[1], inv)) |
                     (uint32_t)f32x2_to_e4m3x2(ckpt::scaled(v[2], inv), ckpt::scaled(v[3], inv)) << 16;
  if (vec) {
    *reinterpret_cast<uint32_t *>(o) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) o[i] = (uint8_t)(w >> (8 * i));
  }
}
__device__ __forceinline__ uint32_t get4_codes(const uint8_t *q, int left, bool vec) {
  if (vec) return __ldg(reinterpret_cast<const uint32_t *>(q));
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) w |= (uint32_t)__ldg(q + i) << (8 * i);
  return w;
}

// 8 rows of a and u.  The 32 features are one scale block, so its largest
// magnitude is a reduction over the 8 lanes of a row.
template <typename TO>
__device__ __forceinline__ void finish_up(const RowParams &p, const float *x, int fw, int row0,
                                          int nv) {
  const int lane = threadIdx.x % 32, f = fw + lane % 8 * 4;
  const int nb = (p.F + ckpt::BLOCK - 1) / ckpt::BLOCK;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int r = s * 4 + lane / 8;
    const float4 a4 = *reinterpret_cast<const float4 *>(x + r * 32 + lane % 8 * 4);
    const float4 u4 = *reinterpret_cast<const float4 *>(x + 256 + r * 32 + lane % 8 * 4);
    const float a[4] = {a4.x, a4.y, a4.z, a4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
    uint32_t ma = 0, mu = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ma = max(ma, ckpt::finite_bits(a[i]));
      mu = max(mu, ckpt::finite_bits(u[i]));
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      ma = max(ma, __shfl_xor_sync(0xffffffffu, ma, o));
      mu = max(mu, __shfl_xor_sync(0xffffffffu, mu, o));
    }
    if (r >= nv || f >= p.F) continue;
    const int ea = ckpt::scale_byte(ma), eu = ckpt::scale_byte(mu);
    const float ia = ckpt::inv_scale_of(ea), iu = ckpt::inv_scale_of(eu);
    float h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = a[i] * ckpt::sigmoid<TO>(a[i]) * u[i];
    const size_t at = (size_t)(row0 + r) * p.F + f;
    put4<TO>(p.out, at, h, p.F - f, p.vec);
    put4_codes(p.saved.ca + at, a, ia, p.F - f, p.vec);
    put4_codes(p.saved.cu + at, u, iu, p.F - f, p.vec);
    if (lane % 8 == 0) {
      const size_t sat = (size_t)(row0 + r) * nb + fw / ckpt::BLOCK;
      p.saved.ea[sat] = (uint8_t)ea;
      p.saved.eu[sat] = (uint8_t)eu;
    }
  }
}

// 16 rows of dh: what they need from memory, loaded ahead of the sums.
struct BwdRows {
  uint32_t ca[4], cu[4];
  int e[4];
  float g[4];
  template <bool VEC>
  __device__ __forceinline__ void load_as(const RowParams &p, int fw, int row0, int nv) {
    const int lane = threadIdx.x % 32, f = fw + lane % 8 * 4;
    const int nb = (p.F + ckpt::BLOCK - 1) / ckpt::BLOCK;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int r = s * 4 + lane / 8;
      ca[s] = cu[s] = 0u;
      e[s] = 0;
      g[s] = 1.0f;
      if (r < nv && f < p.F) {
        const size_t at = (size_t)(row0 + r) * p.F + f, sat = (size_t)(row0 + r) * nb + fw / ckpt::BLOCK;
        ca[s] = get4_codes(p.saved.ca + at, p.F - f, VEC);
        cu[s] = get4_codes(p.saved.cu + at, p.F - f, VEC);
        e[s] = __ldg(p.saved.ea + sat) | __ldg(p.saved.eu + sat) << 8;
        if (p.gate) g[s] = __ldg(p.gate + row0 + r);
      }
    }
  }
  // (one branch around all loads: a branch at each kept them from being in
  // flight together and cost 7% of the call)
  __device__ __forceinline__ void load(const RowParams &p, int fw, int row0, int nv) {
    if (p.vec)
      load_as<true>(p, fw, row0, nv);
    else
      load_as<false>(p, fw, row0, nv);
  }
};

template <typename TO>
__device__ __forceinline__ void finish_bwd(const RowParams &p, const BwdRows &in, const float *x, int fw,
                                           int row0, int nv) {
  const int lane = threadIdx.x % 32, f = fw + lane % 8 * 4;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int r = s * 4 + lane / 8;
    const float4 d4 = *reinterpret_cast<const float4 *>(x + r * 32 + lane % 8 * 4);
    const float dh[4] = {d4.x, d4.y, d4.z, d4.w};
    const float sa = ckpt::scale_of(in.e[s] & 0xff), su = ckpt::scale_of(in.e[s] >> 8);
    float da[4], du[4], hg[4], t[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float2 a = ckpt::decode2((uint16_t)(in.ca[s] >> (8 * i))), u = ckpt::decode2((uint16_t)(in.cu[s] >> (8 * i)));
      t[i] = ckpt::swiglu_grad<TO>(a.x * sa, u.x * su, dh[i], in.g[s], da[i], du[i], hg[i]);
      t[i + 1] = ckpt::swiglu_grad<TO>(a.y * sa, u.y * su, dh[i + 1], in.g[s], da[i + 1], du[i + 1], hg[i + 1]);
    }
    if (!p.vec) {  // features behind the last: not in the sum even where dy is not finite
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (f + i >= p.F) t[i] = 0.0f;
    }
    const bool on = r < nv && f < p.F;
    float term = on ? (t[0] + t[1]) + (t[2] + t[3]) : 0.0f;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
    if (!on) continue;
    const size_t at = (size_t)(row0 + r) * p.F + f;
    if (p.vec) {
      put4<TO>(p.da, at, da, 4, true);
      put4<TO>(p.du, at, du, 4, true);
      put4<TO>(p.hg, at, hg, 4, true);
    } else {
      put4<TO>(p.da, at, da, p.F - f, false);
      put4<TO>(p.du, at, du, p.F - f, false);
      put4<TO>(p.hg, at, hg, p.F - f, false);
    }
    if (lane % 8 == 0) p.part[(size_t)(fw / ckpt::BLOCK) * p.rows + row0 + r] = term;
  }
}

__device__ __forceinline__ void prefetch_l2(const void *q) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
}

template <int OP, int CG, int AT, int BN, int STAGES, bool SEGS, typename TO>
__global__ void __launch_bounds__(RowCfg<OP, CG, AT, BN, STAGES, SEGS>::NT, 1)
    rows_gemm(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
              const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
              const RowParams p) {
  using C = RowCfg<OP, CG, AT, BN, STAGES, SEGS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = align_smem(smem_raw);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::BAR), *empty = full + STAGES;
  uint64_t *accf = empty + STAGES, *acce = accf + 2, *drained = acce + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::MISC + 4);
  volatile int *pending = reinterpret_cast<volatile int *>(sm + C::MISC + 16);
  const Table tab(sm + C::TAB, p.G, BN);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  const int unit = CG == 2 ? (int)cluster_id_x() : (int)blockIdx.x;
  const int nunits = CG == 2 ? (int)cluster_count_x() : (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
      pending[s] = -1;
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf + b, 1);
      mbar_init(acce + b, C::EPI * CG);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA0);
    tma_prefetch_desc(&tmB0);
  }
  if (warp == 1) {
    if (CG == 2) {
      tmem_alloc_pair(tmem_slot, C::TMEM);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, C::TMEM);
      tmem_relinquish();
    }
  }
  build_table(tab, p.offsets, p.G, p.rows, (p.F + C::FEAT - 1) / C::FEAT, p.status);
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // the pair's barriers exist before any remote arrive
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // with few tiles each is computed in parts of the contraction, which other
  // SMs take (sum_splits adds them up)
  const int splits = (OP == LIN || OP == DX) && SEGS ? p.splits : 1;
  const int total = tab.start[p.G] * splits, per = (p.kb + splits - 1) / splits;
  auto whole = [&](int tile) { return splits == 1 ? tile : tile / splits; };
  auto part_of = [&](int tile) { return splits == 1 ? 0 : tile % splits; };
  auto blocks = [&](int tile) { return min(per, p.kb - part_of(tile) * per); };  // k-blocks of a part

  if (warp < 4) {
    if (C::EPI == 8) regs_low();
    if (warp == 0) {
      if (lane == 0) {
        // ------------------------------------------------------ TMA producer
        // a weight tile that several row tiles of its group read is kept in L2,
        // one that is read once leaves first; the rows are read by every
        // feature tile
        const uint64_t keep = policy_evict_normal(), once = policy_evict_first();
        const uint64_t pol_b = policy_evict_last();
        Ring r;
        bool ok = true;
        for (int tile = unit; ok && tile < total; tile += nunits) {
          const Tile t = find_tile(tab, whole(tile), p.G);
          const int nkb = blocks(tile);
          const uint64_t pol_a = t.ntt > 1 ? keep : once;
          const int brows = ((t.nvalid + 15) & ~15) / CG;  // this SM's share
          const int b0 = t.row0 + (int)rank * brows;
          const int f0 = t.ft * C::FEAT + (int)rank * BM;
          const int nbox = (brows + C::BOXN - 1) / C::BOXN;
          const uint32_t bytes = (uint32_t)(C::A_ALL + nbox * C::BOXN * BK * 2);
          // tiles that run together start at different k-blocks, which spreads
          // their reads of shared operands over L2
          const int k0 = splits == 1 ? (t.ft * 7 + t.tt * 5) % p.kb : part_of(tile) * per;
          int q = k0 / p.kb0, blk = k0 - q * p.kb0;  // pass (of all sources) and block of it
          for (int i = 0; i < nkb; ++i) {
            if (!wait_bounded(empty + r.stage, r.phase ^ 1u, abort_flag, WAIT_NS, p.status)) {
              ok = false;
              break;
            }
            // the leader's barrier counts the bytes of both SMs
            if (leader) mbar_arrive_expect_tx(full + r.stage, bytes * CG);
            pending[r.stage] = (int)r.phase;
            uint8_t *a = sm + r.stage * C::STAGE, *b = a + C::A_ALL;
            const uint32_t bar = CG == 2 ? mapa_shared(smem_u32(full + r.stage), 0) : smem_u32(full + r.stage);
            const bool second = q >= p.passes;
            const int kk = blk * BK;
            const int term = p.passes == 1 ? SPLIT_PASSES - 1 : second ? q - p.passes : q;
            const int za = term_a(term) * p.G + t.g;                    // plane of the weights
            const int yb = term_b(term) * (int)p.rows + b0;             // row of the row planes
            if (++blk == p.kb0) {
              blk = 0;
              if (++q * p.kb0 == p.kb) q = 0;
            }
            const CUtensorMap *ma = second ? &tmA1 : &tmA0, *mb = second ? &tmB1 : &tmB0;
#pragma unroll
            for (int i2 = 0; i2 < AT; ++i2) {
              const int f = f0 + (OP == UP ? 0 : i2 * BM * CG);
              if (C::KMAJOR) {
                load_3d<CG>(OP == UP && i2 == 1 ? &tmA1 : ma, a + i2 * TILE, bar, kk, f, za, pol_a);
              } else {
                load_3d<CG>(ma, a + i2 * TILE, bar, f, kk, za, pol_a);
                load_3d<CG>(ma, a + i2 * TILE + BOX, bar, f + 64, kk, za, pol_a);
              }
            }
            for (int j = 0; j < nbox; ++j)
              load_2d<CG>(mb, b + j * C::BOXN * BK * 2, bar, kk, yb + j * C::BOXN, pol_b);
            r.next(STAGES);
          }
        }
      }
    } else if (warp == 1) {
      if (lane == 0 && leader) {
        // -------------------------------------------------------- MMA issuer
        Ring r, acc;
        bool ok = true;
        for (int tile = unit; ok && tile < total; tile += nunits) {
          const Tile t = find_tile(tab, whole(tile), p.G);
          const int nkb = blocks(tile);
          const uint32_t idesc =
              idesc_bf16_f32(BM * CG, (t.nvalid + 15) & ~15) | (C::KMAJOR ? 0u : A_MN);
          uint32_t d = 0;
          int seg = 0, cut = 0;  // segments begun, the k-block that begins the next
          for (int kb = 0; kb < nkb; ++kb) {
            const bool first = SEGS ? kb == cut : kb == 0;
            if (first) {
              if (SEGS) cut += segment<OP>(seg++, nkb);
              if (kb > 0) {
                commit<CG>(accf + acc.stage);
                acc.next(C::NBUF);
              }
              if (!(ok = wait_bounded(acce + acc.stage, acc.phase ^ 1u, abort_flag, WAIT_NS, p.status))) break;
              d = tmem + (uint32_t)(acc.stage * C::ACC);
            }
            if (!(ok = wait_bounded(full + r.stage, r.phase, abort_flag, WAIT_NS, p.status))) break;
            pending[r.stage] = -1;
            tc_fence_after();
            const uint32_t a = smem_u32(sm + r.stage * C::STAGE), b = a + C::A_ALL;
            // MMAs that share their rows back to back: the other order, all of
            // one A tile first, was 5% slower
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
              const uint64_t bd = sdesc_sw128(b + kk * 32);
#pragma unroll
              for (int i = 0; i < AT; ++i) {
                const uint64_t ad = C::KMAJOR ? sdesc_sw128(a + i * TILE + kk * 32)
                                              : desc_mn(a + i * TILE + kk * 2048);
                mma<CG>(d + i * BN, ad, bd, idesc, first && kk == 0 ? 0u : 1u);
              }
            }
            commit<CG>(empty + r.stage);
            r.next(STAGES);
          }
          if (!ok) break;
          commit<CG>(accf + acc.stage);
          acc.next(C::NBUF);
        }
        if (!ok) {  // no MMA may still write tensor memory when it is freed
          if (CG == 2)
            mma_commit_pair(drained);
          else
            mma_commit(drained);
          drain(drained, 0);
        }
      }
    }
  } else {
    if (C::EPI == 8) regs_high();
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;            // TMEM lane quarter of this warp
    const int half = (warp - 4) >> 2;  // alternate 32-row chunks with 8 warps
    constexpr int STEP = C::STEP, NCH = C::NCH;
    Ring acc;
    uint32_t tb = 0;
    auto acquire = [&]() {
      if (!wait_warp(accf + acc.stage, acc.phase, abort_flag, p.status)) return false;
      tc_fence_after();
      tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc.stage * C::ACC);
      return true;
    };
    auto release = [&]() {  // hands the accumulator back to the MMA
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          mbar_arrive_cluster(mapa_shared(smem_u32(acce + acc.stage), 0));
        else
          mbar_arrive(acce + acc.stage);
      }
      acc.next(C::NBUF);
    };
    for (int tile = unit; tile < total; tile += nunits) {
      const Tile t = find_tile(tab, whole(tile), p.G);
        const int nkb = blocks(tile);
      const int fw = t.ft * C::FEAT + (int)rank * BM + q * 32;  // the warp's first feature
      if (SEGS) {
        // sum[a * NCH + ch]: chunk ch of A tile a
        float sum[AT * NCH][32];
#pragma unroll
        for (int i = 0; i < AT * NCH; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[i][j] = 0.0f;
        // UP, BWD: HR rows are finished at a time; row of the tile that part h
        // of this warp begins with
        constexpr int HR = OP == UP ? 8 : 16, PARTS = 32 / HR;
        auto part_row = [&](int h) { return half * 32 + h / PARTS * STEP + h % PARTS * HR; };
        BwdRows ahead;  // BWD: what the next part reads, in flight
        bool ok = true;
        for (int kb = 0, seg = 0; kb < nkb; kb += segment<OP>(seg++, nkb)) {
          if (OP == BWD && kb + segment<OP>(seg, nkb) >= nkb) ahead.load(p, fw, t.row0 + part_row(0), t.nvalid - part_row(0));
          if (!(ok = acquire())) break;
          if (OP == BWD && kb == 0 && fw < p.F) {
            // the codes are needed after the last segment: into L2 by then
            for (int c = half * 32 + lane; c < t.nvalid; c += STEP) {
              const size_t at = (size_t)(t.row0 + c) * p.F + fw;
              prefetch_l2(p.saved.ca + at);
              prefetch_l2(p.saved.cu + at);
            }
          }
#pragma unroll
          for (int i = 0; i < AT * NCH; ++i) {
            const int c0 = half * 32 + i % NCH * STEP;
            if (c0 >= t.nvalid) continue;
            uint32_t v[32];
            tmem_ld_32x32b_x32(tb + (uint32_t)(i / NCH * BN + c0), v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[i][j] += __uint_as_float(v[j]);
          }
          release();
        }
        if (!ok) break;
        if constexpr (OP == UP || OP == BWD) {
          // the registers of part h go through x
          float *x = reinterpret_cast<float *>(sm + C::XBUF) + (warp - 4) * 512;
#pragma unroll 1
          for (int h = 0; h < NCH * PARTS; ++h) {
            const int c0 = part_row(h);
            if (c0 >= t.nvalid) break;
            const BwdRows in = ahead;
            if (OP == BWD && h + 1 < NCH * PARTS)
              ahead.load(p, fw, t.row0 + part_row(h + 1), t.nvalid - part_row(h + 1));
            __syncwarp();  // x has been read
#pragma unroll
            for (int k = 0; k < NCH * PARTS; ++k)
              if (k == h) {
#pragma unroll
                for (int r = 0; r < HR; ++r) {
                  x[r * 32 + lane] = sum[k / PARTS][k % PARTS * HR + r];
                  if (OP == UP) x[256 + r * 32 + lane] = sum[(AT - 1) * NCH + k / PARTS][k % PARTS * HR + r];
                }
              }
            __syncwarp();
            if (OP == UP)
              finish_up<TO>(p, x, fw, t.row0 + c0, t.nvalid - c0);
            else
              finish_bwd<TO>(p, in, x, fw, t.row0 + c0, t.nvalid - c0);
          }
        } else {
#pragma unroll
          for (int i = 0; i < AT * NCH; ++i) {
            const int c0 = half * 32 + i % NCH * STEP;
            if (c0 < t.nvalid)
              finish_rows<TO>(p, part_of(tile), sum[i], fw + i / NCH * BM * CG, t.row0 + c0, t.nvalid - c0);
          }
        }
      } else {
        // all sums are read out as packed bf16 and the accumulator is handed
        // back before any of them is stored, so the stores overlap the next
        // tile's MMAs
        uint32_t w[AT * NCH][16];
        if (!acquire()) break;
#pragma unroll
        for (int a = 0; a < AT; ++a)
#pragma unroll
          for (int ch = 0; ch < NCH; ch += 2) {
            const int c0 = half * 32 + ch * STEP;
            if (c0 >= t.nvalid) continue;
            uint32_t v0[32], v1[32];
            tmem_ld_32x32b_x32(tb + (uint32_t)(a * BN + c0), v0);
            tmem_ld_32x32b_x32(tb + (uint32_t)(a * BN + c0 + STEP), v1);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              w[a * NCH + ch][e] = pack(__uint_as_float(v0[2 * e]), __uint_as_float(v0[2 * e + 1]));
              w[a * NCH + ch + 1][e] = pack(__uint_as_float(v1[2 * e]), __uint_as_float(v1[2 * e + 1]));
            }
          }
        release();
#pragma unroll
        for (int i = 0; i < AT * NCH; ++i) {
          const int c0 = half * 32 + i % NCH * STEP;
          if (c0 < t.nvalid)
            finish_packed(p, w[i], fw + i / NCH * BM * CG, t.row0 + c0, t.nvalid - c0);
        }
      }
    }
  }

  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) {
    // a stalled pipeline stopped early: let copies already issued land (the
    // leader's barriers count both SMs' copies; the other SM allows its own
    // some time)
    if (leader) {
      for (int s = 0; s < STAGES; ++s)
        if (pending[s] >= 0) drain(full + s, (uint32_t)pending[s]);
    } else {
      pause_ns(200000);
    }
  }
  __syncthreads();
  if (CG == 2) cluster_sync();  // neither SM leaves while the other may touch its memory
  if (warp == 1) {
    tc_fence_after();
    if (CG == 2)
      tmem_dealloc_pair(tmem, C::TMEM);
    else
      tmem_dealloc(tmem, C::TMEM);
  }
}

// out = the sum of the splits' planes, in order, over the rows of the groups
// (offsets NULL: all rows).
template <typename TO>
__global__ void __launch_bounds__(256) sum_splits(const float *__restrict__ part, int splits,
                                                  const int32_t *offsets, int G, int64_t rows,
                                                  int64_t cols, TO *__restrict__ out, int accumulate) {
  int64_t lo = 0, hi = rows;
  if (offsets) ckpt::live_rows(offsets, G, rows, lo, hi);
  const int64_t plane = rows * cols, step = (int64_t)gridDim.x * 256;
  for (int64_t i = lo * cols + (int64_t)blockIdx.x * 256 + threadIdx.x; i < hi * cols; i += step) {
    float s = part[i];
    for (int k = 1; k < splits; ++k) s += part[k * plane + i];
    out[i] = from_f<TO>(accumulate ? to_f(out[i]) + s : s);
  }
}

// dgate[row] = the sum of its terms over the feature blocks, in order.
__global__ void __launch_bounds__(256) sum_parts(const float *__restrict__ part,
                                                 const int32_t *offsets, int G, int64_t rows,
                                                 int nb, float *__restrict__ dgate) {
  int64_t lo, hi;
  ckpt::live_rows(offsets, G, rows, lo, hi);
  const int64_t row = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (row < lo || row >= hi) return;
  float s = 0.0f;
  for (int b = 0; b < nb; ++b) s += part[(size_t)b * rows + row];
  dgate[row] = s;
}

// ------------------------------------------------------------------- dw_gemm

struct DwParams {
  const int32_t *offsets;
  int G, n, k;
  int64_t rows;
  void *dw;
  int accumulate;
  int passes;     // 1, or SPLIT_PASSES for split operands
  int splits;     // parts of each group's rows, each with its own dw
  int above, upto;  // the groups of more than `above` rows and at most `upto`
  int tma_store;  // rows of dw are multiples of 16 bytes, dw is 16-byte aligned
  int32_t *status;
};

// A tile of AT * 256 features of dy (AT blocks of 128 per SM of the pair) by
// 256 columns of x.
// SEGS: sums in segments.
template <typename TO, int AT, bool SEGS>
struct DwCfg {
  static constexpr int EPI = 8, NT = 32 * (4 + EPI);
  static constexpr int FEAT = AT * 256;
  static constexpr int STAGE = AT * TILE + 128 * BK * 2;  // per SM: AT * 128 + 128 columns
  static constexpr int STAGES = AT == 2 ? 4 : 6;          // 192 KB in flight
  static constexpr int NBUF = 2 / AT;                     // accumulators of AT * 256 columns
  static constexpr int CHUNK = 128 / (int)sizeof(TO);     // columns of a 128-byte staging row
  static constexpr int STG = STAGES * STAGE;              // a 32 x 128-byte buffer per warp
  static constexpr int BAR = STG + EPI * 4096;
  static constexpr int NBARS = 3 * STAGES + 5;
  static constexpr int MISC = BAR + NBARS * 8;
  static constexpr int BYTES = 1024 + MISC + 16 + 4 * STAGES;
  static_assert(!SEGS || AT == 1, "sums in registers");
  static_assert(BYTES <= 232448, "shared memory");
};

template <typename TO, int AT, bool SEGS>
__global__ void __launch_bounds__(DwCfg<TO, AT, SEGS>::NT, 1)
    dw_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
            const __grid_constant__ CUtensorMap tmC, const DwParams p) {
  using C = DwCfg<TO, AT, SEGS>;
  constexpr int STAGES = C::STAGES;
  bool idle = false;
  if (p.above >= 0) {  // nothing to do where no group is so long
    bool any = false;
    for (int g = threadIdx.x; g < p.G; g += C::NT) {
      int lo, n;
      group_bounds(p.offsets, g, p.rows, lo, n, nullptr);
      any |= n > p.above;
    }
    idle = !__syncthreads_or(any);
  }
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = align_smem(smem_raw);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::BAR), *empty = full + STAGES;
  uint64_t *tail = empty + STAGES, *accf = tail + STAGES, *acce = accf + 2, *drained = acce + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::MISC + 4);
  // per stage: -1, or the phase its copies complete, + 2 when they count on `tail`
  volatile int *pending = reinterpret_cast<volatile int *>(sm + C::MISC + 16);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int unit = (int)cluster_id_x(), nunits = (int)cluster_count_x();

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 2);
      mbar_init(empty + s, 2);  // the MMAs, and the warp of the tail rows
      mbar_init(tail + s, 1);
      pending[s] = -1;
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf + b, 1);
      mbar_init(acce + b, C::EPI * 2);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int ntiles = (p.n + C::FEAT - 1) / C::FEAT, ktiles = (p.k + 255) / 256;
  const int64_t total = idle ? 0 : (int64_t)p.G * p.splits * ntiles * ktiles;

  struct Job {
    int g, n0, k0, lo, kc;  // g: plane of dw, of split s and group g' s * G + g'
    int kb0, kb, tail;  // k-blocks of one pass and of all; rows of a pass's last one
    int nmma;           // columns of the MMA
    bool other;         // not a group of this launch (kb 0)
    // rows of k-block b of a pass, and whether it ends inside a 16-row step
    __device__ __forceinline__ int depth(int b) const { return b == kb0 - 1 ? tail : BK; }
    __device__ __forceinline__ bool fix(int b) const { return depth(b) % 16 != 0; }
  };
  auto job = [&](int64_t tile) {
    Job j;
    j.g = (int)(tile / (ntiles * ktiles));
    const int local = (int)(tile - (int64_t)j.g * ntiles * ktiles);
    j.n0 = local / ktiles * C::FEAT;
    j.k0 = local % ktiles * 256;
    const int split = p.splits == 1 ? 0 : j.g / p.G;
    group_bounds(p.offsets, j.g - split * p.G, p.rows, j.lo, j.kc, threadIdx.x == 0 ? p.status : nullptr);
    j.other = j.kc <= p.above || j.kc > p.upto;
    if (j.other) j.kc = 0;
    if (p.splits > 1) {  // whole k-blocks of the group's rows
      const int part = ((j.kc + p.splits - 1) / p.splits + BK - 1) / BK * BK;
      const int skip = min(j.kc, split * part);
      j.lo += skip;
      j.kc = min(part, j.kc - skip);
    }
    j.kb0 = (j.kc + BK - 1) / BK;
    j.kb = j.kb0 * p.passes;
    j.tail = j.kc - (j.kb0 - 1) * BK;
    j.nmma = min(256, (p.k - j.k0 + 31) / 32 * 32);
    return j;
  };

  if (warp < 4) {
    regs_low();
    if (warp == 0) {
      if (lane == 0) {
        // ------------------------------------------------------ TMA producer
        const uint64_t pol = policy_evict_normal();
        Ring r;
        bool ok = true;
        for (int64_t tile = unit; ok && tile < total; tile += nunits) {
          const Job j = job(tile);
          const int hb = j.nmma / 2, nbox = (hb + 63) / 64;
          const int n0 = j.n0 + (int)rank * BM, k0 = j.k0 + (int)rank * hb;
          const uint32_t bytes = (uint32_t)(AT * TILE + nbox * BOX);
          int q = 0, blk = 0;  // pass and block of it
          for (int i = 0; i < j.kb; ++i) {
            if (!wait_bounded(empty + r.stage, r.phase ^ 1u, abort_flag, WAIT_NS, p.status)) {
              ok = false;
              break;
            }
            // a last block that ends inside a 16-row step is completed on each
            // SM's own `tail` barrier and handed on when its rows are zeroed
            const bool fix = j.fix(blk);
            uint32_t bar;
            if (fix) {
              mbar_arrive_expect_tx(tail + r.stage, bytes);
              bar = mapa_shared(smem_u32(tail + r.stage), rank);
            } else {
              mbar_arrive(tail + r.stage);
              if (leader) {
                mbar_arrive_expect_tx(full + r.stage, bytes * 2);
                mbar_arrive(full + r.stage);
              }
              bar = mapa_shared(smem_u32(full + r.stage), 0);
            }
            pending[r.stage] = (int)r.phase + (fix ? 2 : 0);
            uint8_t *a = sm + r.stage * C::STAGE, *b = a + AT * TILE;
            const int term = p.passes == 1 ? SPLIT_PASSES - 1 : q;
            const int row = j.lo + blk * BK;
            const int ya = term_a(term) * (int)p.rows + row, yb = term_b(term) * (int)p.rows + row;
            if (++blk == j.kb0) {
              blk = 0;
              ++q;
            }
#pragma unroll
            for (int c = 0; c < 2 * AT; ++c)
              load_2d<2>(&tmA, a + c * BOX, bar, n0 + c / 2 * 256 + c % 2 * 64, ya, pol);
            for (int c = 0; c < nbox; ++c) load_2d<2>(&tmB, b + c * BOX, bar, k0 + c * 64, yb, pol);
            r.next(STAGES);
          }
        }
      }
    } else if (warp == 1) {
      if (lane == 0 && leader) {
        // -------------------------------------------------------- MMA issuer
        Ring r, acc;
        bool ok = true;
        for (int64_t tile = unit; ok && tile < total; tile += nunits) {
          const Job j = job(tile);
          if (j.kb == 0) continue;
          const uint32_t idesc = idesc_bf16_f32(256, j.nmma) | A_MN | B_MN;
          uint32_t d = 0;
          for (int i = 0, blk = 0; i < j.kb; ++i, blk = blk + 1 == j.kb0 ? 0 : blk + 1) {
            const bool first = i == 0 || (SEGS && i % SEG == 0);
            if (first) {
              if (i > 0) {
                commit<2>(accf + acc.stage);
                acc.next(C::NBUF);
              }
              if (!(ok = wait_bounded(acce + acc.stage, acc.phase ^ 1u, abort_flag, WAIT_NS, p.status))) break;
              d = tmem + (uint32_t)(acc.stage * AT * 256);
            }
            if (!(ok = wait_bounded(full + r.stage, r.phase, abort_flag, WAIT_NS, p.status))) break;
            pending[r.stage] = -1;
            tc_fence_after();
            const uint32_t a = smem_u32(sm + r.stage * C::STAGE), b = a + AT * TILE;
            const int steps = (j.depth(blk) + 15) / 16;
            for (int s = 0; s < steps; ++s)
#pragma unroll
              for (int c = 0; c < AT; ++c)
                mma<2>(d + c * 256, desc_mn(a + c * TILE + s * 2048), desc_mn(b + s * 2048), idesc,
                       first && s == 0 ? 0u : 1u);
            commit<2>(empty + r.stage);
            r.next(STAGES);
          }
          if (!ok) break;
          commit<2>(accf + acc.stage);
          acc.next(C::NBUF);
        }
        if (!ok) {
          mma_commit_pair(drained);
          drain(drained, 0);
        }
      }
    } else if (warp == 2) {
      // ------------------------------------------- tail rows, ahead of the MMAs
      // (done by the issuing warp itself, this held up every tile of a short
      // group: 455 -> 385 us for 32 groups of about 128 rows)
      // The warp passes every block and counts on `empty` as the MMAs do: were
      // it a ring behind the producer, `tail` would have gone through two
      // phases, which their one parity bit does not tell from none.
      Ring r;
      for (int64_t tile = unit; tile < total; tile += nunits) {
        const Job j = job(tile);
        for (int i = 0, blk = 0; i < j.kb; ++i, blk = blk + 1 == j.kb0 ? 0 : blk + 1) {
          if (!wait_warp(tail + r.stage, r.phase, abort_flag, p.status)) {
            tile = total;
            break;
          }
          if (j.fix(blk)) {
            // rows tail .. next multiple of 16 of every 64-column box: 128
            // bytes each, whole rows, so the swizzle does not matter
            uint8_t *st = sm + r.stage * C::STAGE + j.tail * 128;
            const int bytes = (16 - j.tail % 16) * 128, nbox = 2 * AT + (j.nmma / 2 + 63) / 64;
            for (int bx = 0; bx < nbox; ++bx)
              for (int at = lane * 16; at < bytes; at += 512)
                *reinterpret_cast<uint4 *>(st + bx * BOX + at) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              pending[r.stage] = -1;
              arrive_cluster(mapa_shared(smem_u32(full + r.stage), 0));
            }
          }
          if (lane == 0) mbar_arrive(empty + r.stage);
          r.next(STAGES);
        }
      }
    }
  } else {
    regs_high();
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - 4) >> 2;
    constexpr int CH = C::CHUNK, NCH = 128 / CH;  // this warp's 128 columns in chunks
    uint8_t *stg = sm + C::STG + (warp - 4) * 4096;
    // fp32 sums are added to dw by the copy itself (an element has one tile)
    const bool reduce = sizeof(TO) == 4 && p.accumulate && p.tma_store;
    Ring acc;
    uint32_t tb = 0;
    auto acquire = [&]() {
      if (!wait_warp(accf + acc.stage, acc.phase, abort_flag, p.status)) return false;
      tc_fence_after();
      tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc.stage * AT * 256 + half * 128);
      return true;
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(acce + acc.stage), 0));
      acc.next(C::NBUF);
    };
    for (int64_t tile = unit; tile < total; tile += nunits) {
      const Job j = job(tile);
      if (j.other || (j.kb == 0 && p.accumulate)) continue;
      // lane l stores columns k0 .. k0 + CH - 1 of feature n0 + l; `word(i)`
      // is the i-th 4-byte word of its row of the staging buffer
      auto store = [&](int n0, int k0, auto word) {
        if (lane == 0) store_wait_read<0>();  // the last store has left the buffer
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4 *>(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) =
              make_uint4(word(4 * i), word(4 * i + 1), word(4 * i + 2), word(4 * i + 3));
        if (p.tma_store) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (reduce)
              reduce_3d(&tmC, stg, k0, n0, j.g);
            else
              store_3d(&tmC, stg, k0, n0, j.g);
            store_commit();
          }
          return;
        }
        // rows off the 16-byte pitch: a row of the buffer at a time
        __syncwarp();
        const int nr = min(32, p.n - n0), nc = min(CH, p.k - k0);
        TO *o = static_cast<TO *>(p.dw) + ((size_t)j.g * p.n + n0) * p.k + k0;
        for (int r = 0; r < nr; ++r, o += p.k)
          for (int c = lane; c < nc; c += 32) {
            constexpr int V = 16 / sizeof(TO);  // values of a 16-byte unit
            o[c] = *reinterpret_cast<const TO *>(stg + r * 128 + (((c / V) ^ (r & 7)) << 4) + c % V * sizeof(TO));
          }
        __syncwarp();
      };
      auto emit = [&](float (&v)[CH], int c) {
        const int n0 = j.n0 + (int)rank * BM + q * 32, k0 = j.k0 + half * 128 + c * CH;
        if (k0 >= p.k || n0 >= p.n) return;
        if (p.accumulate && !reduce) {
          if (sizeof(TO) == 2 && p.tma_store) {
            // old values: whole rows of the chunk (8 lanes of 16 bytes each)
            // into the staging buffer, from there each lane's own row
            const TO *o = static_cast<const TO *>(p.dw) + ((size_t)j.g * p.n + n0) * p.k + k0;
            uint4 old[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = i * 4 + lane / 8, u = lane % 8 * 8;
              old[i] = make_uint4(0, 0, 0, 0);
              if (n0 + r < p.n && k0 + u < p.k) old[i] = *reinterpret_cast<const uint4 *>(o + (size_t)r * p.k + u);
            }
            if (lane == 0) store_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = i * 4 + lane / 8;
              *reinterpret_cast<uint4 *>(stg + r * 128 + (((lane % 8) ^ (r & 7)) << 4)) = old[i];
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 w = *reinterpret_cast<const uint4 *>(stg + lane * 128 + ((i ^ (lane & 7)) << 4));
              const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[(8 * i + 2 * e) % CH] += __uint_as_float(x[e] << 16);
                v[(8 * i + 2 * e + 1) % CH] += __uint_as_float(x[e] & 0xffff0000u);
              }
            }
          } else if (n0 + lane < p.n) {
            const TO *o = static_cast<const TO *>(p.dw) + ((size_t)j.g * p.n + n0 + lane) * p.k + k0;
#pragma unroll
            for (int i = 0; i < CH; ++i)
              if (k0 + i < p.k) v[i] += to_f(o[i]);
          }
        }
        store(n0, k0, [&](int i) {
          if (sizeof(TO) == 4) return __float_as_uint(v[i % CH]);
          return pack(v[2 * i % CH], v[(2 * i + 1) % CH]);
        });
      };
      if constexpr (AT == 2) {
        // the accumulators are read out as packed bf16 (128 registers) and
        // handed back before any of it is stored
        uint32_t w[2][64];
        if (j.kb > 0) {
          if (!acquire()) break;
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
              uint32_t v0[32], v1[32];
              tmem_ld_32x32b_x32(tb + (uint32_t)(a * 256 + c * 32), v0);
              tmem_ld_32x32b_x32(tb + (uint32_t)(a * 256 + c * 32 + 32), v1);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                w[a][c * 16 + e] = pack(__uint_as_float(v0[2 * e]), __uint_as_float(v0[2 * e + 1]));
                w[a][c * 16 + 16 + e] = pack(__uint_as_float(v1[2 * e]), __uint_as_float(v1[2 * e + 1]));
              }
            }
          release();
        } else {
#pragma unroll
          for (int i = 0; i < 64; ++i) w[0][i] = w[1][i] = 0u;
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int c = 0; c < NCH; ++c) {
            const int n0 = j.n0 + a * 256 + (int)rank * BM + q * 32, k0 = j.k0 + half * 128 + c * CH;
            if (n0 < p.n && k0 < p.k) store(n0, k0, [&](int i) { return w[a][c * 32 + i]; });
          }
        continue;
      }
      if (SEGS || j.kb == 0) {
        float sum[NCH][CH];
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
          for (int i = 0; i < CH; ++i) sum[c][i] = 0.0f;
        bool ok = true;
        for (int i = 0; i < j.kb; i += SEG) {
          if (!(ok = acquire())) break;
#pragma unroll
          for (int c = 0; c < NCH * CH / 32; ++c) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tb + (uint32_t)(c * 32), v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) sum[c * 32 / CH][c * 32 % CH + e] += __uint_as_float(v[e]);
          }
          release();
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < NCH; ++c) emit(sum[c], c);
      } else {
        if (!acquire()) break;
        const uint32_t t0 = tb;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          float o[CH];
#pragma unroll
          for (int h = 0; h < CH / 32; ++h) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(t0 + (uint32_t)(c * CH + h * 32), v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[h * 32 + e] = __uint_as_float(v[e]);
          }
          if (c == NCH - 1) release();
          emit(o, c);
        }
      }
    }
    if (lane == 0) store_wait_all();
  }

  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) {
    for (int s = 0; s < STAGES; ++s)
      if (pending[s] >= 2) drain(tail + s, (uint32_t)(pending[s] - 2));
    if (leader) {
      for (int s = 0; s < STAGES; ++s)
        if (pending[s] == 0 || pending[s] == 1) drain(full + s, (uint32_t)pending[s]);
    } else {
      pause_ns(200000);
    }
  }
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace tcg
}  // namespace moe
