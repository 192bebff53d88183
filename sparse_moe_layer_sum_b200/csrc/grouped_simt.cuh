// Grouped products on the CUDA cores (fp32 multiply-adds): fp32 operands, and
// bf16 ones whose rows or addresses are not multiples of 16 bytes.
//
// One persistent kernel for the three directions, written as C = A B over a
// contraction index c:
//   LIN  C = y  [rows, n]: A[r][c] = x[r,c],  B[c][j] = w[g,j,c]
//   DX   C = dx [rows, k]: A[r][c] = dy[r,c], B[c][j] = w[g,c,j] (two sources)
//   DW   C = dw [n, k]:    A[r][c] = dy[c,r], B[c][j] = x[c,j], c over the
//        group's rows
// 256 threads compute a T x T tile of C from slices of the operands in two
// alternating shared-memory buffers; the next slice is loaded into registers
// while the current one is multiplied.  Products are added in pairs
// (fma.rn.f32x2, two IEEE fp32 multiply-adds per instruction).
//
// Bound by the multiply-add rate where there are enough tiles (T 128 and 64) of
// rows that fill them (with a row or two a group most multiply-adds are for rows
// that do not exist), by the latency of a slice where there are few: T 32 takes slices four times
// as deep, which four groups of 64 threads multiply at the same time, and adds
// the four partial tiles in a fixed order at the end.
#pragma once

#include "grouped.cuh"

namespace moe {
namespace simt {

using namespace grouped;

enum Dir { LIN, DX, DW };

struct Args {
  const void *a0, *b0, *a1, *b1;  // two sources (DX); a1 == NULL: one
  void *c;
  const int32_t *offsets;
  int G, n, k;
  int64_t rows;
  int accumulate;  // DW
  int splits;      // parts of the contraction, each with its own plane of c
  int32_t *status;
};

constexpr int THREADS = 256;

template <int T>
struct Cfg {
  static constexpr int TT = T == 128 ? 8 : 4;              // values per thread and dimension
  static constexpr int GROUPS = T == 32 ? 4 : 1;           // of threads, over a slice's depth
  static constexpr int BLOCKS = T == 128 ? 2 : 4;          // per SM
  static constexpr int BK = 2048 / T;                      // depth of a slice
  static constexpr int LD = T * BK / THREADS;              // operand values a thread loads: 8
  static constexpr int PITCH = T + 4;
  static constexpr int BUF = 2 * BK * PITCH;               // floats of one A and B slice
  static size_t smem(int G) { return sizeof(float) * 2 * BUF + Table::bytes(G); }
  static_assert(GROUPS * (T / TT) * (T / TT) == THREADS, "threads");
};

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ void fma2(uint64_t &d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

template <typename TI, typename TO, int DIR, int T>
__global__ void __launch_bounds__(THREADS, Cfg<T>::BLOCKS) product(Args p) {
  using C = Cfg<T>;
  constexpr int TT = C::TT, BK = C::BK, LD = C::LD, PITCH = C::PITCH, NT = T / TT;
  extern __shared__ __align__(16) float smem[];
  Table tab(smem + 2 * C::BUF, p.G, T);
  const int cols = DIR == LIN ? p.n : p.k;  // columns of C
  const int ftiles = (cols + T - 1) / T, rtiles = (p.n + T - 1) / T;
  build_table(tab, p.offsets, p.G, p.rows, ftiles, p.status);
  const int64_t whole = DIR == DW ? (int64_t)p.G * rtiles * ftiles : tab.start[p.G];
  const int splits = T == 32 ? p.splits : 1;
  const int64_t tiles = whole * splits;
  const int tid = threadIdx.x, grp = tid / (NT * NT), tx = tid % NT, ty = tid / NT % NT;
  // a thread's values: TT = 8 takes two runs of four, half a tile apart
  auto at = [&](int t, int i) { return i / 4 * (T / 2) + t * 4 + i % 4; };

  for (int64_t at_tile = blockIdx.x; at_tile < tiles; at_tile += gridDim.x) {
    const int part = splits == 1 ? 0 : (int)(at_tile % splits);
    const int64_t tile = splits == 1 ? at_tile : at_tile / splits;
    // C's rows r0 .. r0 + nr - 1 and columns from c0; the contraction runs
    // over [k0, k0 + kc)
    int g, nr, c0, kc;
    int64_t r0, k0 = 0;
    if (DIR == DW) {
      g = (int)(tile / (rtiles * ftiles));
      const int local = (int)(tile % (rtiles * ftiles));
      r0 = (local / ftiles) * T;
      nr = min(T, p.n - (int)r0);
      c0 = (local % ftiles) * T;
      k0 = tab.lo[g];
      kc = tab.rows(g);
      if (kc == 0 && p.accumulate) continue;
    } else {
      const Tile t = find_tile(tab, (int)tile, p.G);
      g = t.g;
      r0 = t.row0;
      nr = t.nvalid;
      c0 = t.ft * T;
      kc = DIR == LIN ? p.k : p.n;
    }
    const size_t wbase = (size_t)g * p.n * p.k;
    const int slices = (kc + BK - 1) / BK, nsrc = DIR == DX && p.a1 ? 2 : 1;
    uint64_t acc[TT][TT / 2];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < TT / 2; ++j) acc[i][j] = 0;

    // Operands whose contraction index is contiguous run over it across
    // threads, the others over their rows; a thread's LD values of a slice lie
    // a fixed step apart, and only the bounds of the last slice vary.
    constexpr bool AC = DIR != DW, BC = DIR == LIN;
    constexpr int STEP = THREADS / BK, CSTEP = THREADS / T;
    const int ac = AC ? tid % BK : tid / T, ar = AC ? tid / BK : tid % T;
    const int bc = BC ? tid % BK : tid / T, bj = BC ? tid / BK : tid % T;
    const size_t lda = AC ? (size_t)kc : (size_t)p.n;  // between rows of A in memory
    const size_t a_at = AC ? (size_t)(r0 + ar) * lda + ac : (size_t)(k0 + ac) * lda + r0 + ar;
    const size_t b_at = BC ? wbase + (size_t)(c0 + bj) * p.k + bc
                           : (DIR == DX ? wbase + (size_t)bc * p.k : (size_t)(k0 + bc) * p.k) + c0 + bj;
    const size_t a_step = (AC ? STEP : CSTEP) * lda, b_step = (size_t)(BC ? STEP : CSTEP) * p.k;
    const size_t a_slice = AC ? (size_t)BK : BK * lda, b_slice = BC ? (size_t)BK : (size_t)BK * p.k;
    const int a_rows = nr - ar, b_cols = cols - c0 - bj;  // left from this thread's first
    float ra[LD], rb[LD];
    auto load = [&](int sl) {
      const bool second = DIR == DX && sl >= slices;
      const int i0 = second ? sl - slices : sl;
      const TI *A = static_cast<const TI *>(second ? p.a1 : p.a0) + a_at + i0 * a_slice;
      const TI *Bm = static_cast<const TI *>(second ? p.b1 : p.b0) + b_at + i0 * b_slice;
      const int left = kc - i0 * BK;  // of the contraction
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const bool on = AC ? ac < left && i * STEP < a_rows : ac + i * CSTEP < left && a_rows > 0;
        ra[i] = on ? to_f(*A) : 0.0f;
        A += a_step;
      }
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const bool on = BC ? bc < left && i * STEP < b_cols : bc + i * CSTEP < left && b_cols > 0;
        rb[i] = on ? to_f(*Bm) : 0.0f;
        Bm += b_step;
      }
    };
    const int per = splits == 1 ? slices * nsrc : (slices * nsrc + splits - 1) / splits, begin = part * per;
    const int total = min(slices * nsrc, begin + per);
    if (begin < total) load(begin);
    for (int sl = begin; sl < total; ++sl) {
      float *As = smem + sl % 2 * C::BUF, *Bs = As + BK * PITCH;
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        As[(AC ? ac : ac + i * CSTEP) * PITCH + (AC ? ar + i * STEP : ar)] = ra[i];
        Bs[(BC ? bc : bc + i * CSTEP) * PITCH + (BC ? bj + i * STEP : bj)] = rb[i];
      }
      __syncthreads();  // (the other buffer's readers are past it too)
      if (sl + 1 < total) load(sl + 1);
      constexpr int DEPTH = BK / C::GROUPS;
#pragma unroll 8
      for (int c = grp * DEPTH; c < (grp + 1) * DEPTH; ++c) {
        float fa[TT];
        uint64_t fb[TT / 2];
#pragma unroll
        for (int i = 0; i < TT; i += 4) {
          *reinterpret_cast<float4 *>(fa + i) = *reinterpret_cast<const float4 *>(As + c * PITCH + at(ty, i));
          const float4 b = *reinterpret_cast<const float4 *>(Bs + c * PITCH + at(tx, i));
          fb[i / 2] = pair(b.x, b.y);
          fb[i / 2 + 1] = pair(b.z, b.w);
        }
#pragma unroll
        for (int i = 0; i < TT; ++i) {
          const uint64_t a2 = pair(fa[i], fa[i]);
#pragma unroll
          for (int j = 0; j < TT / 2; ++j) fma2(acc[i][j], a2, fb[j]);
        }
      }
    }
    float sum[TT][TT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < TT / 2; ++j) unpair(acc[i][j], sum[i][2 * j], sum[i][2 * j + 1]);
    __syncthreads();  // the buffers are free: the next tile's, or the partial tiles'
    if (C::GROUPS > 1) {
      float *mine = smem + (tid % (NT * NT)) * TT * TT;  // of this thread's values
      for (int q = 1; q < C::GROUPS; ++q) {
        if (grp == q) {
#pragma unroll
          for (int i = 0; i < TT * TT; ++i) mine[i] = sum[i / TT][i % TT];
        }
        __syncthreads();
        if (grp == 0) {
#pragma unroll
          for (int i = 0; i < TT * TT; ++i) sum[i / TT][i % TT] += mine[i];
        }
        __syncthreads();
      }
      if (grp != 0) continue;
    }
    TO *Cp = static_cast<TO *>(p.c) + (DIR == DW ? wbase : 0);
    if (T == 32) Cp += part * (DIR == DW ? (int64_t)p.G * p.n * p.k : p.rows * cols);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int r = at(ty, i);
      if (r >= nr) continue;
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const int cc = c0 + at(tx, j);
        if (cc >= cols) continue;
        TO *d = Cp + (size_t)(r0 + r) * cols + cc;
        *d = from_f<TO>(DIR == DW && p.accumulate ? to_f(*d) + sum[i][j] : sum[i][j]);
      }
    }
  }
}

}  // namespace simt
}  // namespace moe
