// Row groups of the training operators: the sanitised bounds of every group
// and the tiles each is cut into, built by each block in shared memory from
// the caller's offsets (no separate launch and no workspace).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {
namespace grouped {

using bf16 = __nv_bfloat16;

constexpr int MAX_GROUPS = 1024;

// Bounds of group g within [0, rows].  Offsets that decrease or leave the
// range are clamped, so that every later access stays in its buffer, and
// reported.
__device__ __forceinline__ void group_bounds(const int32_t *__restrict__ off, int g, int64_t rows,
                                             int &lo, int &n, int32_t *status) {
  const int64_t a = off[g], b = off[g + 1];
  if (a < 0 || b < a || b > rows) set_status(status, MOE_ERR_RANGE);
  const int64_t ca = a < 0 ? 0 : a > rows ? rows : a;
  const int64_t cb = b < ca ? ca : b > rows ? rows : b;
  lo = (int)ca;
  n = (int)(cb - ca);
}

// Group g's rows are lo[g] .. lo[g + 1] - 1.
// They are cut into ntt tiles of `base` rows, a multiple of 16 and at most
// rows_max; each token tile meets ft feature tiles.  start is the exclusive
// prefix of ntt * ft over the groups; start[G] the number of tiles.
struct Table {
  int32_t *start;  // [G + 1]
  int32_t *lo;     // [G + 1]
  int rows_max;
  static size_t bytes(int G) { return sizeof(int32_t) * (size_t)(2 * G + 2); }
  __device__ __forceinline__ Table(void *mem, int G, int rows_max_)
      : start(static_cast<int32_t *>(mem)), lo(start + G + 1), rows_max(rows_max_) {}
  __device__ __forceinline__ int rows(int g) const { return lo[g + 1] - lo[g]; }
};

__device__ __forceinline__ void split_rows(int n, int rows_max, int &base, int &ntt) {
  if (n <= 0) {
    base = 16;
    ntt = 0;
    return;
  }
  const int ntt0 = (n + rows_max - 1) / rows_max;
  base = ((n + ntt0 - 1) / ntt0 + 15) / 16 * 16;
  ntt = (n + base - 1) / base;
}

// Every thread of the block calls; ends with the table complete for all.
__device__ __forceinline__ void build_table(const Table &t, const int32_t *__restrict__ off, int G,
                                            int64_t rows, int ft, int32_t *status) {
  bool bad = false;
  for (int g = threadIdx.x; g <= G; g += blockDim.x) {
    const int64_t a = off[g];
    bad |= a < 0 || a > rows || (g < G && off[g + 1] < a);
    t.lo[g] = (int)(a < 0 ? 0 : a > rows ? rows : a);
  }
  if (bad) set_status(status, MOE_ERR_RANGE);
  // An offset below an earlier one counts as the earlier one: no row is then in
  // two groups, and the groups have no more tiles than rows give, which the
  // 32-bit tile numbers hold.
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0)
      for (int g = 1; g <= G; ++g) t.lo[g] = max(t.lo[g], t.lo[g - 1]);
    __syncthreads();
  }
  if (threadIdx.x < 32) {  // exclusive prefix: a lane owns a run of groups
    const int lane = threadIdx.x, per = (G + 31) / 32;
    const int g0 = min(G, lane * per), g1 = min(G, g0 + per);
    int local = 0;
    for (int g = g0; g < g1; ++g) {
      int base, ntt;
      split_rows(t.rows(g), t.rows_max, base, ntt);
      t.start[g] = ntt * ft;
      local += ntt * ft;
    }
    int inc = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    int run = inc - local;
    for (int g = g0; g < g1; ++g) {
      const int c = t.start[g];
      t.start[g] = run;
      run += c;
    }
    if (lane == 31) t.start[G] = inc;
  }
  __syncthreads();
}

struct Tile {
  int g, ft, tt, ntt;
  int row0, nvalid;  // first row of the tile in the row buffers, rows it holds
};

__device__ __forceinline__ Tile find_tile(const Table &t, int tile, int G) {
  int lo = 0, hi = G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.start[mid] <= tile)
      lo = mid;
    else
      hi = mid;
  }
  Tile r;
  r.g = lo;
  const int n = t.rows(lo);
  int base;
  split_rows(n, t.rows_max, base, r.ntt);
  const int local = tile - t.start[lo];
  r.ft = local / r.ntt;
  r.tt = local - r.ft * r.ntt;
  r.row0 = t.lo[lo] + r.tt * base;
  r.nvalid = min(base, n - r.tt * base);
  return r;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float v) {
  return __float2bfloat16_rn(v);
}

}  // namespace grouped
}  // namespace moe
