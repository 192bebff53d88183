// Grouped products on the CUDA cores (fp32 multiply-adds): fp32 operands, and
// bf16 ones whose rows or addresses are not multiples of 16 bytes.
//
// One persistent kernel for the three directions, written as C = A B over a
// contraction index c:
//   LIN  C = y  [rows, n]: A[r][c] = x[r,c],  B[c][j] = w[g,j,c]
//   DX   C = dx [rows, k]: A[r][c] = dy[r,c], B[c][j] = w[g,c,j] (two sources)
//   DW   C = dw [n, k]:    A[r][c] = dy[c,r], B[c][j] = x[c,j], c over the
//        group's rows
// A block computes a B x B tile of C with (B / 16)^2 values per thread from
// BK-deep slices in shared memory; the next slice is loaded into registers
// while the current one is multiplied.
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
  int32_t *status;
};

constexpr int BK = 16, THREADS = 256;

template <int B>
size_t smem_bytes(int G) {
  return sizeof(float) * 2 * BK * (B + 4) + Table::bytes(G);
}

template <typename TI, typename TO, int DIR, int B>
__global__ void __launch_bounds__(THREADS) product(Args p) {
  constexpr int TM = B / 16;                // values per thread and dimension
  constexpr int LD = B * BK / THREADS;      // slice elements a thread loads
  extern __shared__ float smem[];
  float(*As)[B + 4] = reinterpret_cast<float(*)[B + 4]>(smem);
  float(*Bs)[B + 4] = reinterpret_cast<float(*)[B + 4]>(smem + BK * (B + 4));
  Table tab(smem + 2 * BK * (B + 4), p.G, B);
  const int cols = DIR == LIN ? p.n : p.k;  // columns of C
  const int ftiles = (cols + B - 1) / B, rtiles = (p.n + B - 1) / B;
  build_table(tab, p.offsets, p.G, p.rows, ftiles, p.status);
  const int total = DIR == DW ? 0 : tab.start[p.G];
  const int64_t tiles = DIR == DW ? (int64_t)p.G * rtiles * ftiles : total;
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;

  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    // C's rows r0 .. r0 + nr - 1 and columns from c0; the contraction runs
    // over [k0, k0 + kc)
    int g, nr, c0, kc;
    int64_t r0, k0 = 0;
    if (DIR == DW) {
      g = (int)(tile / (rtiles * ftiles));
      const int local = (int)(tile % (rtiles * ftiles));
      r0 = (local / ftiles) * B;
      nr = min(B, p.n - (int)r0);
      c0 = (local % ftiles) * B;
      k0 = tab.lo[g];
      kc = tab.rows(g);
      if (kc == 0 && p.accumulate) continue;
    } else {
      const Tile t = find_tile(tab, (int)tile, p.G);
      g = t.g;
      r0 = t.row0;
      nr = t.nvalid;
      c0 = t.ft * B;
      kc = DIR == LIN ? p.k : p.n;
    }
    const size_t wbase = (size_t)g * p.n * p.k;
    float acc[TM][TM];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = 0.0f;

    const int nsrc = DIR == DX && p.a1 ? 2 : 1;
    for (int src = 0; src < nsrc; ++src) {
      const TI *A = static_cast<const TI *>(src ? p.a1 : p.a0);
      const TI *Bm = static_cast<const TI *>(src ? p.b1 : p.b0);
      float ra[LD], rb[LD];
      auto load = [&](int kk0) {
#pragma unroll
        for (int i = 0; i < LD; ++i) {
          const int idx = tid + i * THREADS;
          // the contiguous index of each operand runs fastest over threads
          const int ac = DIR == DW ? idx / B : idx % BK, ar = DIR == DW ? idx % B : idx / BK;
          const int c = kk0 + ac;
          float v = 0.0f;
          if (c < kc && ar < nr)
            v = DIR == DW ? to_f(A[(size_t)(k0 + c) * p.n + r0 + ar])
                          : to_f(A[(size_t)(r0 + ar) * kc + c]);
          ra[i] = v;
          const int bc = DIR == LIN ? idx % BK : idx / B, bj = DIR == LIN ? idx / BK : idx % B;
          const int cb = kk0 + bc, j = c0 + bj;
          v = 0.0f;
          if (cb < kc && j < cols)
            v = DIR == LIN  ? to_f(Bm[wbase + (size_t)j * p.k + cb])
                : DIR == DX ? to_f(Bm[wbase + (size_t)cb * p.k + j])
                            : to_f(Bm[(size_t)(k0 + cb) * p.k + j]);
          rb[i] = v;
        }
      };
      load(0);
      for (int kk0 = 0; kk0 < kc; kk0 += BK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LD; ++i) {
          const int idx = tid + i * THREADS;
          if (DIR == DW)
            As[idx / B][idx % B] = ra[i];
          else
            As[idx % BK][idx / BK] = ra[i];
          if (DIR == LIN)
            Bs[idx % BK][idx / BK] = rb[i];
          else
            Bs[idx / B][idx % B] = rb[i];
        }
        __syncthreads();
        if (kk0 + BK < kc) load(kk0 + BK);
#pragma unroll
        for (int c = 0; c < BK; ++c) {
          float fa[TM], fb[TM];
#pragma unroll
          for (int i = 0; i < TM; i += 4) {
            *reinterpret_cast<float4 *>(fa + i) =
                *reinterpret_cast<const float4 *>(&As[c][(i / 4) * 64 + ty * 4]);
            *reinterpret_cast<float4 *>(fb + i) =
                *reinterpret_cast<const float4 *>(&Bs[c][(i / 4) * 64 + tx * 4]);
          }
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = fmaf(fa[i], fb[j], acc[i][j]);
        }
      }
      __syncthreads();
    }
    TO *C = static_cast<TO *>(p.c) + (DIR == DW ? wbase : 0);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = (i / 4) * 64 + ty * 4 + i % 4;
      if (r >= nr) continue;
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int cc = c0 + (j / 4) * 64 + tx * 4 + j % 4;
        if (cc >= cols) continue;
        TO *d = C + (size_t)(r0 + r) * cols + cc;
        *d = from_f<TO>(DIR == DW && p.accumulate ? to_f(*d) + acc[i][j] : acc[i][j]);
      }
    }
  }
}

}  // namespace simt
}  // namespace moe
