// The 8-bit activation format (e4m3 codes, one power-of-two scale for 32
// values of a row) and the elementwise kernels that write and read it.
//
// The scale of a block is 2^e with the smallest e for which amax <= 448 * 2^e.
// With amax = 1.m * 2^E this is E - 8, or E - 7 when 1.m > 1.75 (448 is
// 1.75 * 2^8), read off the bits of amax: no logarithm, no rounding, so every
// kernel that writes the format makes the same choice.  A power of two also
// makes v / scale and code * scale exact: the only rounding is the code's.
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include "grouped.cuh"
#include "sm100.cuh"

namespace moe {
namespace ckpt {

using namespace grouped;

constexpr int BLOCK = 32;  // values that share a scale

// Magnitude bits of v, 0 for an infinity or a NaN.  As integers they order
// like the magnitudes.
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

// Biased exponent byte of the scale for the largest finite magnitude's bits.
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  const int b = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(b, 0);
}

__device__ __forceinline__ float scale_of(int byte) {  // 2^(byte - 127)
  return __uint_as_float(byte > 0 ? (uint32_t)byte << 23 : 0x400000u);
}

__device__ __forceinline__ float inv_scale_of(int byte) {  // 2^(127 - byte), byte <= 247
  return __uint_as_float((uint32_t)(254 - byte) << 23);
}

// v / scale as the code conversion takes it: a finite v is within 448, an
// infinity or NaN becomes NaN (the conversion would saturate an infinity).
__device__ __forceinline__ float scaled(float v, float inv) {
  const float q = v * inv;
  return fabsf(q) <= 448.0f ? q : __uint_as_float(0x7fc00000u);
}

__device__ __forceinline__ uint8_t encode1(float v, float inv) {
  return (uint8_t)(sm100::f32x2_to_e4m3x2(scaled(v, inv), 0.0f) & 0xffu);
}

__device__ __forceinline__ float2 decode2(uint16_t codes) {
  const uint32_t h = sm100::e4m3x2_to_f16x2(codes);  // exact
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ float decode1(uint8_t code, float scale) {
  return decode2(code).x * scale;
}

template <typename T>
__device__ __forceinline__ float sigmoid(float a);
// fp32 results: the library's exponential and an IEEE division
template <>
__device__ __forceinline__ float sigmoid<float>(float a) {
  return 1.0f / (1.0f + expf(-a));
}
// bf16 results: the hardware exponential, within 2 + 1.2 |a| steps of 2^-23 by
// CUDA's table, and reciprocal, within 2: far inside the rounding that follows.
// dgate, in fp32, is summed from the same sigmoid: within 6e-7 of a term at
// |a| = 1, and 2e-6 at a = -10, where the term itself is down by exp(a).
template <>
__device__ __forceinline__ float sigmoid<bf16>(float a) {
  return __fdividef(1.0f, 1.0f + __expf(-a));
}

// ------------------------------------------------------------ rows <-> codes

template <typename T>
struct Vec8;  // eight values, loaded or stored as 16-byte vectors; bf16 rows with
              // streaming stores (32768 x 7168 restored in 92 us, 106 without, both
              // with one resident set of blocks)
template <>
struct Vec8<bf16> {
  static __device__ __forceinline__ void load(const bf16 *p, float (&v)[8]) {
    const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(bf16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};
template <>
struct Vec8<float> {
  static __device__ __forceinline__ void load(const float *p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  static __device__ __forceinline__ void store(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// un / per for the warps' work items; nearly always within 32 bits, where the
// division costs a quarter.
__device__ __forceinline__ int64_t item_row(int64_t un, int per) {
  if (un <= 0xffffffffll) return (int64_t)((uint32_t)un / (uint32_t)per);
  return un / per;
}

constexpr int ROW_THREADS = 256;
constexpr int UNROLL = 4;   // loads in flight per lane, of eight values each
constexpr int UNROLL1 = 8;  // and of one value

// Eight values a lane, four lanes a block: k % 8 == 0 and aligned rows.
template <typename TI>
__global__ void __launch_bounds__(ROW_THREADS) save_rows_v8(const TI *__restrict__ src,
                                                            int64_t rows, int k,
                                                            uint8_t *__restrict__ codes,
                                                            uint8_t *__restrict__ exps) {
  const int lane = threadIdx.x % 32, nb = (k + BLOCK - 1) / BLOCK;
  const int segs = (nb * 4 + 32 * UNROLL - 1) / (32 * UNROLL);
  const int64_t units = rows * segs, step = (int64_t)gridDim.x * (ROW_THREADS / 32);
  for (int64_t un = (int64_t)blockIdx.x * (ROW_THREADS / 32) + threadIdx.x / 32; un < units;
       un += step) {
    const int64_t row = item_row(un, segs);
    const int c0 = (int)(un - row * segs) * 32 * UNROLL + lane;
    float v[UNROLL][8];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int c = c0 + i * 32;
      if (c * 8 < k) {
        Vec8<TI>::load(src + row * k + c * 8, v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int c = c0 + i * 32;
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, finite_bits(v[i][j]));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = scale_byte(m);
      const float inv = inv_scale_of(e);
      uint32_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[j] = (uint32_t)sm100::f32x2_to_e4m3x2(scaled(v[i][4 * j], inv), scaled(v[i][4 * j + 1], inv)) |
               (uint32_t)sm100::f32x2_to_e4m3x2(scaled(v[i][4 * j + 2], inv), scaled(v[i][4 * j + 3], inv)) << 16;
      if (c * 8 < k) {
        *reinterpret_cast<uint2 *>(codes + row * k + c * 8) = make_uint2(w[0], w[1]);
        if ((c & 3) == 0) exps[row * nb + c / 4] = (uint8_t)e;
      }
    }
  }
}

// One value a lane, a block a warp, UNROLL1 blocks in flight: any k and
// alignment. Bound by the latency of its loads: 13649 rows of 2313 are restored
// in 114 us with one block in flight, 55 with four, 47.5 with eight and 51 with
// sixteen; 4000 of them are saved in 29, 18, 19 and 21 us.
template <typename TI>
__global__ void __launch_bounds__(ROW_THREADS) save_rows(const TI *__restrict__ src, int64_t rows,
                                                         int k, uint8_t *__restrict__ codes,
                                                         uint8_t *__restrict__ exps) {
  const int lane = threadIdx.x % 32, nb = (k + BLOCK - 1) / BLOCK, per = (nb + UNROLL1 - 1) / UNROLL1;
  const int64_t units = rows * per, step = (int64_t)gridDim.x * (ROW_THREADS / 32);
  for (int64_t un = (int64_t)blockIdx.x * (ROW_THREADS / 32) + threadIdx.x / 32; un < units;
       un += step) {
    const int64_t row = item_row(un, per);
    const int b0 = (int)(un - row * per) * UNROLL1;
    float v[UNROLL1];
#pragma unroll
    for (int u = 0; u < UNROLL1; ++u) {
      const int i = (b0 + u) * BLOCK + lane;
      v[u] = i < k ? to_f(src[row * k + i]) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < UNROLL1; ++u) {
      const int i = (b0 + u) * BLOCK + lane;
      const int e = scale_byte(__reduce_max_sync(0xffffffffu, finite_bits(v[u])));
      if (i < k) codes[row * k + i] = encode1(v[u], inv_scale_of(e));
      if (lane == 0 && b0 + u < nb) exps[row * nb + b0 + u] = (uint8_t)e;
    }
  }
}

// Row of the stored rows that output row i takes; -1 (reported) if there is none.
__device__ __forceinline__ int64_t source_row(const int32_t *index, int64_t i, int64_t rows,
                                              int32_t *status) {
  const int64_t r = index ? index[i] : i;
  if (r >= 0 && r < rows) return r;
  set_status(status, MOE_ERR_RANGE);
  return -1;
}

template <typename TO>
__global__ void __launch_bounds__(ROW_THREADS) load_rows_v8(const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ exps,
                                                            int64_t rows, int k,
                                                            const int32_t *__restrict__ index,
                                                            int64_t n, TO *__restrict__ out,
                                                            int32_t *status) {
  const int lane = threadIdx.x % 32, nb = (k + BLOCK - 1) / BLOCK;
  const int segs = (nb * 4 + 32 * UNROLL - 1) / (32 * UNROLL);
  const int64_t units = n * segs, step = (int64_t)gridDim.x * (ROW_THREADS / 32);
  for (int64_t un = (int64_t)blockIdx.x * (ROW_THREADS / 32) + threadIdx.x / 32; un < units;
       un += step) {
    const int64_t i = item_row(un, segs);
    const int c0 = (int)(un - i * segs) * 32 * UNROLL + lane;
    const int64_t row = source_row(index, i, rows, status);
    uint2 q[UNROLL];
    int e[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int c = c0 + j * 32;
      q[j] = make_uint2(0, 0);
      e[j] = 0;
      if (row >= 0 && c * 8 < k) {
        q[j] = __ldg(reinterpret_cast<const uint2 *>(codes + row * k + c * 8));
        e[j] = __ldg(exps + row * nb + c / 4);
      }
    }
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int c = c0 + j * 32;
      if (c * 8 >= k) continue;
      const float s = scale_of(e[j]);
      const uint16_t w[4] = {(uint16_t)(q[j].x & 0xffffu), (uint16_t)(q[j].x >> 16),
                             (uint16_t)(q[j].y & 0xffffu), (uint16_t)(q[j].y >> 16)};
      float v[8];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float2 d = decode2(w[t]);
        v[2 * t] = d.x * s;
        v[2 * t + 1] = d.y * s;
      }
      Vec8<TO>::store(out + i * k + c * 8, v);
    }
  }
}

template <typename TO>
__global__ void __launch_bounds__(ROW_THREADS) load_rows(const uint8_t *__restrict__ codes,
                                                         const uint8_t *__restrict__ exps,
                                                         int64_t rows, int k,
                                                         const int32_t *__restrict__ index,
                                                         int64_t n, TO *__restrict__ out,
                                                         int32_t *status) {
  const int lane = threadIdx.x % 32, nb = (k + BLOCK - 1) / BLOCK, per = (nb + UNROLL1 - 1) / UNROLL1;
  const int64_t units = n * per, step = (int64_t)gridDim.x * (ROW_THREADS / 32);
  for (int64_t un = (int64_t)blockIdx.x * (ROW_THREADS / 32) + threadIdx.x / 32; un < units;
       un += step) {
    const int64_t i = item_row(un, per), row = source_row(index, i, rows, status);
    const int b0 = (int)(un - i * per) * UNROLL1;
    uint8_t c[UNROLL1], e[UNROLL1];
#pragma unroll
    for (int u = 0; u < UNROLL1; ++u) {
      const int j = (b0 + u) * BLOCK + lane;
      const bool on = row >= 0 && j < k;
      c[u] = on ? codes[row * k + j] : 0;
      e[u] = on ? exps[row * nb + b0 + u] : 0;
    }
#pragma unroll
    for (int u = 0; u < UNROLL1; ++u) {
      const int j = (b0 + u) * BLOCK + lane;
      if (j < k) out[i * k + j] = from_f<TO>(decode1(c[u], scale_of(e[u])));
    }
  }
}

// ------------------------------------------------------------ plain rows

// out[i] = src[index[i]], eight values a lane (VEC) or one (32768 rows of 2313
// bf16 values: 49 us with eight loads in flight, 66 with four).
template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(ROW_THREADS) gather_rows(const TI *__restrict__ src, int64_t rows,
                                                           int k, const int32_t *__restrict__ index,
                                                           int64_t n, TO *__restrict__ out,
                                                           int32_t *status) {
  constexpr int V = VEC ? 8 : 1, U = VEC ? UNROLL : UNROLL1, PER = 32 * U * V;  // values of an item
  const int lane = threadIdx.x % 32, items = (k + PER - 1) / PER;
  const int64_t units = n * items, step = (int64_t)gridDim.x * (ROW_THREADS / 32);
  for (int64_t un = (int64_t)blockIdx.x * (ROW_THREADS / 32) + threadIdx.x / 32; un < units;
       un += step) {
    const int64_t i = item_row(un, items), row = source_row(index, i, rows, status);
    const int c0 = (int)(un - i * items) * PER + lane * V;
    float v[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * 32 * V;
#pragma unroll
      for (int j = 0; j < V; ++j) v[u][j] = 0.0f;
      if (row >= 0 && c < k) {
        if constexpr (VEC)
          Vec8<TI>::load(src + row * k + c, v[u]);
        else
          v[u][0] = to_f(src[row * k + c]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * 32 * V;
      if (c >= k) continue;
      if constexpr (VEC)
        Vec8<TO>::store(out + i * k + c, v[u]);
      else
        out[i * k + c] = from_f<TO>(v[u][0]);
    }
  }
}

// One thread per (token, slot), then one per shared row; the first threads
// copy the group offsets.
__global__ void __launch_bounds__(256) training_rows(const int32_t *__restrict__ offsets,
                                                     const int32_t *__restrict__ sorted_token,
                                                     const int32_t *__restrict__ slot_of,
                                                     const float *__restrict__ weights, int64_t T,
                                                     int k, int E, int shared, int32_t *row_token,
                                                     float *row_gate, int32_t *group_offsets,
                                                     int32_t *status) {
  const int64_t routed = T * k, total = routed + (shared ? T : 0);
  const int64_t step = (int64_t)gridDim.x * blockDim.x, me = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t i = me; i < total; i += step) {
    if (i >= routed) {
      row_token[i] = (int32_t)(i - routed);
      row_gate[i] = 1.0f;
      continue;
    }
    const int32_t t = sorted_token[i], p = slot_of[i];
    if (t < 0 || t >= T || p < 0 || p >= routed) set_status(status, MOE_ERR_RANGE);
    if (t >= 0 && t < T) row_token[i] = t;
    if (p >= 0 && p < routed) row_gate[p] = weights[i];
  }
  for (int64_t g = me; g <= E + shared; g += step)
    group_offsets[g] = g <= E ? offsets[g] : (int32_t)total;
}

// ------------------------------------------- SwiGLU around the 8-bit format
//
// The elementwise halves of swiglu_checkpoint and swiglu_backward for the
// products that run on the CUDA cores, from and to their fp32 sums.

// Rows [lo, hi) that belong to a group.
__device__ __forceinline__ void live_rows(const int32_t *off, int G, int64_t rows, int64_t &lo,
                                          int64_t &hi) {
  lo = min(max((int64_t)off[0], (int64_t)0), rows);
  hi = min(max((int64_t)off[G], lo), rows);
}

struct Saved {
  uint8_t *ca, *ea, *cu, *eu;
};

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) swiglu_save(const float *__restrict__ a,
                                                           const float *__restrict__ u,
                                                           const int32_t *offsets, int G,
                                                           int64_t rows, int n, T *__restrict__ h,
                                                           Saved s) {
  int64_t lo, hi;
  live_rows(offsets, G, rows, lo, hi);
  const int lane = threadIdx.x % 32, nb = (n + BLOCK - 1) / BLOCK;
  const int64_t step = (int64_t)gridDim.x * (ROW_THREADS / 32);
  for (int64_t un = lo * nb + (int64_t)blockIdx.x * (ROW_THREADS / 32) + threadIdx.x / 32;
       un < hi * nb; un += step) {
    const int64_t row = item_row(un, nb);
    const int i = (int)(un - row * nb) * BLOCK + lane;
    const size_t at = (size_t)row * n + i;
    const float va = i < n ? a[at] : 0.0f, vu = i < n ? u[at] : 0.0f;
    const int ea = scale_byte(__reduce_max_sync(0xffffffffu, finite_bits(va)));
    const int eu = scale_byte(__reduce_max_sync(0xffffffffu, finite_bits(vu)));
    if (i < n) {
      h[at] = from_f<T>(va * sigmoid<T>(va) * vu);
      s.ca[at] = encode1(va, inv_scale_of(ea));
      s.cu[at] = encode1(vu, inv_scale_of(eu));
    }
    if (lane == 0) {
      s.ea[un] = (uint8_t)ea;
      s.eu[un] = (uint8_t)eu;
    }
  }
}

// The gradients of one hidden value; returns its term of dgate.
template <typename T>
__device__ __forceinline__ float swiglu_grad(float a, float u, float dh, float gate, float &da,
                                             float &du, float &hg) {
  const float s = sigmoid<T>(a), as = a * s, h = as * u, gd = gate * dh;
  da = gd * u * (s + as * (1.0f - s));
  du = gd * as;
  hg = gate * h;
  return dh * h;
}

// One block a row.
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) swiglu_grads(const float *__restrict__ dh, Saved s,
                                                            const float *__restrict__ gate,
                                                            const int32_t *offsets, int G,
                                                            int64_t rows, int n, T *__restrict__ da,
                                                            T *__restrict__ du, T *__restrict__ hg,
                                                            float *__restrict__ dgate) {
  __shared__ float part[ROW_THREADS / 32];
  int64_t lo, hi;
  live_rows(offsets, G, rows, lo, hi);
  const int nb = (n + BLOCK - 1) / BLOCK;
  for (int64_t row = lo + blockIdx.x; row < hi; row += gridDim.x) {
    const float g = gate ? gate[row] : 1.0f;
    float sum = 0.0f;
    for (int i = threadIdx.x; i < n; i += ROW_THREADS) {
      const size_t at = (size_t)row * n + i, b = (size_t)row * nb + i / BLOCK;
      const float a = decode1(s.ca[at], scale_of(s.ea[b]));
      const float u = decode1(s.cu[at], scale_of(s.eu[b]));
      float va, vu, vh;
      sum += swiglu_grad<T>(a, u, dh[at], g, va, vu, vh);
      da[at] = from_f<T>(va);
      du[at] = from_f<T>(vu);
      hg[at] = from_f<T>(vh);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      float t = 0.0f;
      for (int w = 0; w < ROW_THREADS / 32; ++w) t += part[w];
      dgate[row] = t;
    }
    __syncthreads();
  }
}

}  // namespace ckpt
}  // namespace moe
