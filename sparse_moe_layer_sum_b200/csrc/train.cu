// moe_train: training operators of the experts (moe_train.h) -- host checks,
// the choice of kernel and the launches.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "ckpt.cuh"
#include "common.cuh"
#include "grouped.cuh"
#include "grouped_simt.cuh"
#include "grouped_tc.cuh"
#include "moe_train.h"

namespace moe {
namespace {

using grouped::bf16;
using grouped::Table;

bool act_type(moe_dtype dt) { return dt == MOE_BF16 || dt == MOE_F32; }
size_t elem(moe_dtype dt) { return dt == MOE_F32 ? 4 : 2; }

moe_status check_shape(const moe_grouped_shape *s) {
  if (!s) return MOE_ERR_INVALID;
  if (s->groups < 1 || s->n < 1 || s->k < 1 || s->rows < 0) return MOE_ERR_INVALID;
  if (s->groups > grouped::MAX_GROUPS || s->n > (1 << 20) || s->k > (1 << 20) ||
      s->rows >= ((int64_t)1 << 31))
    return MOE_ERR_UNSUPPORTED;
  // tile numbers are 32-bit: 64-row tiles of 64 columns at the finest
  const int64_t cols = s->n > s->k ? s->n : s->k;
  if ((s->rows / 16 + s->groups) * ((cols + 63) / 64) >= ((int64_t)1 << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// SMs of the current device, asked once per device; 0 if that fails.
int sm_count() {
  static int known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && known[dev]) return known[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev] = n;
  return n;
}

// ------------------------------------------------------------ CUDA-core path

template <typename TI, typename TO, int DIR, int T>
moe_status launch_simt(const simt::Args &a, int64_t tiles, int nsm, cudaStream_t s) {
  const int64_t most = (int64_t)nsm * simt::Cfg<T>::BLOCKS;
  const int64_t grid = tiles < most ? tiles : most;
  simt::product<TI, TO, DIR, T><<<(unsigned)grid, simt::THREADS, simt::Cfg<T>::smem(a.G), s>>>(a);
  return launch_status();
}

template <typename TI, typename TO, int DIR>
moe_status simt_tiles(const simt::Args &a, cudaStream_t s) {
  const int nsm = sm_count();
  if (nsm < 1) return MOE_ERR_CUDA;
  const int cols = DIR == simt::LIN ? a.n : a.k;
  auto tiles = [&](int t) {
    const int64_t ct = (cols + t - 1) / t;
    return DIR == simt::DW ? (int64_t)a.G * ((a.n + t - 1) / t) * ct : (a.rows / t + a.G) * ct;
  };
  // the larger tile reuses each operand value more often; the smaller ones
  // where the larger would leave SMs without work
  if (tiles(128) >= 4 * nsm) return launch_simt<TI, TO, DIR, 128>(a, tiles(128), nsm, s);
  if (tiles(64) >= nsm) return launch_simt<TI, TO, DIR, 64>(a, tiles(64), nsm, s);
  return launch_simt<TI, TO, DIR, 32>(a, tiles(32), nsm, s);
}

template <int DIR>
moe_status simt_product(const simt::Args &a, moe_dtype in, moe_dtype out, cudaStream_t s) {
  if (in == MOE_F32)
    return out == MOE_F32 ? simt_tiles<float, float, DIR>(a, s) : simt_tiles<float, bf16, DIR>(a, s);
  return out == MOE_F32 ? simt_tiles<bf16, float, DIR>(a, s) : simt_tiles<bf16, bf16, DIR>(a, s);
}

// ------------------------------------------------------------------ products

struct Product {
  const moe_grouped_shape *s;
  moe_dtype dt, out_dt;
  const void *a0, *b0, *a1, *b1;  // rows and weights (dw: dy and x)
  const int32_t *offsets;
  void *out;
  int accumulate;
  int32_t *status;
  cudaStream_t stream;
};

simt::Args simt_args(const Product &p) {
  simt::Args a;
  a.a0 = p.a0;
  a.b0 = p.b0;
  a.a1 = p.a1;
  a.b1 = p.b1;
  a.c = p.out;
  a.offsets = p.offsets;
  a.G = p.s->groups;
  a.n = p.s->n;
  a.k = p.s->k;
  a.rows = p.s->rows;
  a.accumulate = p.accumulate;
  a.status = p.status;
  return a;
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// ---------------------------------------------------------- tensor-core path

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// Row-major [planes, rows, cols] tensor (planes 0: a matrix), 128-byte
// swizzled boxes of box_rows x 128 bytes; what lies outside reads as zero and
// is not written.
bool tensor_map(CUtensorMap *m, const void *base, moe_dtype dt, uint64_t planes, uint64_t rows,
                uint64_t cols, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const uint64_t e = elem(dt);
  cuuint64_t dims[3] = {cols, rows, planes};
  cuuint64_t strides[2] = {cols * e, rows * cols * e};
  cuuint32_t box[3] = {(uint32_t)(128 / e), box_rows, 1};
  cuuint32_t step[3] = {1, 1, 1};
  return fn(m, dt == MOE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
            planes ? 3 : 2, const_cast<void *>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One block, or one pair of blocks, per SM or SM pair.
template <auto kern, typename... A>
moe_status launch_persistent(int threads, size_t smem, int cg, int64_t tiles,
                             cudaStream_t s, A... args) {
  constexpr size_t SMEM_MAX = 232448;
  if (smem > SMEM_MAX) return MOE_ERR_UNSUPPORTED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const int nsm = sm_count();
  if (nsm < 2) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  int64_t units = nsm / cg;
  if (cg == 2) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  // asked once per kernel and device: the shared-memory limit, and how many
  // SM pairs can be resident together
  static int ready[64];
  int n = dev < 64 ? ready[dev] : 0;
  if (n == 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_MAX) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    n = (int)units;
    if (cg == 2) {
      cfg.gridDim = dim3((unsigned)(units * 2));
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();  // not sticky: the launch below decides
        n = (int)units;
      }
    }
    if (dev < 64) ready[dev] = n;
  }
  if (n < units) units = n;
  if (tiles < units) units = tiles > 0 ? tiles : 1;
  cfg.gridDim = dim3((unsigned)(units * cg));
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return MOE_ERR_CUDA;
  return launch_status();
}

// Upper bound on the row tiles of all groups.
int64_t row_tiles(const moe_grouped_shape *s, int bn) {
  return s->rows / bn + (s->rows < s->groups ? s->rows : s->groups);
}

struct RowMaps {
  CUtensorMap a0, a1, b0, b1;
};

// Maps of a product with rows x0 (and x1) [rows, contract] and weights w0
// (and w1); `kmajor`: weights [G, F, contract], else [G, contract, F].
template <typename C>
bool row_maps(RowMaps *m, const moe_grouped_shape *s, const void *w0, const void *w1,
              const void *x0, const void *x1, uint64_t F, uint64_t contract) {
  auto wmap = [&](CUtensorMap *t, const void *w) {
    return C::KMAJOR ? tensor_map(t, w, MOE_BF16, s->groups, F, contract, tcg::BM)
                     : tensor_map(t, w, MOE_BF16, s->groups, contract, F, 64);
  };
  auto xmap = [&](CUtensorMap *t, const void *x) {
    return tensor_map(t, x, MOE_BF16, 0, s->rows, contract, C::BOXN);
  };
  if (!wmap(&m->a0, w0) || !xmap(&m->b0, x0)) return false;
  m->a1 = m->a0;
  m->b1 = m->b0;
  return (!w1 || wmap(&m->a1, w1)) && (!x1 || xmap(&m->b1, x1));
}

template <int OP, int CG, int AT, int BN, int STAGES, bool SEGS, typename TO>
moe_status launch_rows(const moe_grouped_shape *s, const void *w0, const void *w1, const void *x0,
                       const void *x1, int F, int contract, tcg::RowParams p, cudaStream_t st) {
  using C = tcg::RowCfg<OP, CG, AT, BN, STAGES, SEGS>;
  RowMaps m;
  if (!row_maps<C>(&m, s, w0, w1, x0, x1, F, contract)) return MOE_ERR_CUDA;
  p.G = s->groups;
  p.F = F;
  p.rows = s->rows;
  p.kb0 = (contract + tcg::BK - 1) / tcg::BK;
  p.kb = x1 ? 2 * p.kb0 : p.kb0;
  const int64_t tiles = row_tiles(s, BN) * ((F + C::FEAT - 1) / C::FEAT);
  return launch_persistent<tcg::rows_gemm<OP, CG, AT, BN, STAGES, SEGS, TO>>(C::NT, C::smem(p.G), CG, tiles,
                           st, m.a0, m.a1, m.b0, m.b1, (const tcg::RowParams)p);
}

// rows of a group on average
int64_t mean_rows(const moe_grouped_shape *s) { return (s->rows + s->groups - 1) / s->groups; }

template <int OP, typename TO>
moe_status tc_rows(const Product &p, int F, int contract) {
  tcg::RowParams r = {};
  r.offsets = p.offsets;
  r.out = p.out;
  r.status = p.status;
  const auto *s = p.s;
  auto run = [&](auto launch) { return launch(s, p.b0, p.b1, p.a0, p.a1, F, contract, r, p.stream); };
  if constexpr (sizeof(TO) == 4) {  // fp32 results: sums in segments
    if (mean_rows(s) <= 48 || F < 256) return run(launch_rows<OP, 1, 1, 64, 8, true, TO>);
    return run(launch_rows<OP, 2, 1, 256, 6, true, TO>);
  } else {
    if (mean_rows(s) <= 48) return run(launch_rows<OP, 1, 1, 64, 8, false, TO>);
    if (F < 512) return run(launch_rows<OP, 1, 1, 256, 4, false, TO>);
    return run(launch_rows<OP, 2, 2, 256, 4, false, TO>);
  }
}

int scale_blocks(int n) { return (n + ckpt::BLOCK - 1) / ckpt::BLOCK; }

// Sizes the tensor-core kernels take: rows of 16 bytes, and 4 hidden features
// written at a time.
bool tc_up_sizes(const moe_grouped_shape *s, moe_dtype dt) {
  return dt == MOE_BF16 && s->k % 8 == 0 && s->n % 4 == 0;
}
bool tc_bwd_sizes(const moe_grouped_shape *s, moe_dtype dt) {
  return dt == MOE_BF16 && s->k % 8 == 0 && s->n % 8 == 0;
}

// The first matmul with its checkpoint (n hidden features from k), and the
// gradients of the hidden rows (contracting over k).
moe_status tc_up(const moe_grouped_shape *s, const void *x, const void *w1, const void *w3,
                 const tcg::RowParams &r, cudaStream_t st) {
  if (mean_rows(s) <= 48 || s->n < 256)
    return launch_rows<tcg::UP, 1, 2, 64, 5, true, bf16>(s, w1, w3, x, nullptr, s->n, s->k, r, st);
  return launch_rows<tcg::UP, 2, 2, 128, 5, true, bf16>(s, w1, w3, x, nullptr, s->n, s->k, r, st);
}

moe_status tc_bwd(const moe_grouped_shape *s, const void *dy, const void *w2,
                  const tcg::RowParams &r, cudaStream_t st) {
  if (mean_rows(s) <= 48 || s->n < 256)
    return launch_rows<tcg::BWD, 1, 1, 64, 8, true, bf16>(s, w2, nullptr, dy, nullptr, s->n, s->k, r, st);
  return launch_rows<tcg::BWD, 2, 1, 256, 6, true, bf16>(s, w2, nullptr, dy, nullptr, s->n, s->k, r, st);
}

template <typename TO, int AT>
moe_status launch_dw(const Product &p) {
  using C = tcg::DwCfg<TO, AT>;
  const auto *s = p.s;
  CUtensorMap a, b, c;
  if (!tensor_map(&a, p.a0, MOE_BF16, 0, s->rows, s->n, tcg::BK) ||
      !tensor_map(&b, p.b0, MOE_BF16, 0, s->rows, s->k, tcg::BK) ||
      !tensor_map(&c, p.out, p.out_dt, s->groups, s->n, s->k, 32))
    return MOE_ERR_CUDA;
  const tcg::DwParams d{p.offsets, s->groups, s->n, s->k, s->rows, p.out, p.accumulate, p.status};
  const int64_t tiles = (int64_t)s->groups * ((s->n + C::FEAT - 1) / C::FEAT) * ((s->k + 255) / 256);
  return launch_persistent<tcg::dw_gemm<TO, AT>>(C::NT, (size_t)C::BYTES, 2, tiles, p.stream, a, b, c, d);
}

moe_status tc_dw(const Product &p) {
  if (p.out_dt == MOE_F32) return launch_dw<float, 1>(p);
  // a bf16 sum with what is there already adds in fp32, which the packed
  // results of the wider tile no longer are
  if (p.accumulate || p.s->n <= 256) return launch_dw<bf16, 1>(p);
  return launch_dw<bf16, 2>(p);
}

// Tensor maps need 16-byte aligned addresses and row pitches.
bool tc_operand(const void *p, int64_t cols, moe_dtype dt) {
  return aligned(p, 16) && cols * elem(dt) % 16 == 0;
}

moe_status run_linear(const Product &p) {
  if (p.dt == MOE_BF16 && tc_operand(p.a0, p.s->k, p.dt) && tc_operand(p.b0, p.s->k, p.dt))
    return p.out_dt == MOE_F32 ? tc_rows<tcg::LIN, float>(p, p.s->n, p.s->k)
                               : tc_rows<tcg::LIN, bf16>(p, p.s->n, p.s->k);
  return simt_product<simt::LIN>(simt_args(p), p.dt, p.out_dt, p.stream);
}

moe_status run_dx(const Product &p) {
  if (p.dt == MOE_BF16 && tc_operand(p.a0, p.s->n, p.dt) && tc_operand(p.b0, p.s->k, p.dt) &&
      tc_operand(p.a1, p.s->n, p.dt) && tc_operand(p.b1, p.s->k, p.dt))
    return p.out_dt == MOE_F32 ? tc_rows<tcg::DX, float>(p, p.s->k, p.s->n)
                               : tc_rows<tcg::DX, bf16>(p, p.s->k, p.s->n);
  return simt_product<simt::DX>(simt_args(p), p.dt, p.out_dt, p.stream);
}

moe_status run_dw(const Product &p) {
  // without rows there is nothing to map; the CUDA-core kernel writes the zeros
  if (p.dt == MOE_BF16 && p.s->rows > 0 && tc_operand(p.a0, p.s->n, p.dt) &&
      tc_operand(p.b0, p.s->k, p.dt) && tc_operand(p.out, p.s->k, p.out_dt))
    return tc_dw(p);
  return simt_product<simt::DW>(simt_args(p), p.dt, p.out_dt, p.stream);
}

unsigned row_grid(int64_t warps) {
  const int64_t blocks = (warps + ckpt::ROW_THREADS / 32 - 1) / (ckpt::ROW_THREADS / 32);
  const int64_t most = 148 * 8;
  return (unsigned)(blocks < most ? blocks : most);
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_EXPORT moe_status moe_grouped_linear(const moe_grouped_shape *s, const void *x, moe_dtype dt,
                                         const void *w, const int32_t *offsets, void *y,
                                         moe_dtype y_dt, int32_t *dev_status,
                                         moe_stream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (!act_type(dt) || !act_type(y_dt)) return MOE_ERR_UNSUPPORTED;
  if (s->rows == 0) return MOE_OK;
  if (!x || !w || !offsets || !y) return MOE_ERR_INVALID;
  return run_linear({s, dt, y_dt, x, w, nullptr, nullptr, offsets, y, 0, dev_status,
                     as_stream(stream)});
}

MOE_EXPORT moe_status moe_grouped_linear_dx(const moe_grouped_shape *s, const void *dy,
                                            moe_dtype dt, const void *w, const void *dy2,
                                            const void *w2, const int32_t *offsets, void *dx,
                                            moe_dtype dx_dt, int32_t *dev_status,
                                            moe_stream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (!act_type(dt) || !act_type(dx_dt)) return MOE_ERR_UNSUPPORTED;
  if (s->rows == 0) return MOE_OK;  // (an empty dy2 may well be NULL)
  if ((dy2 == nullptr) != (w2 == nullptr)) return MOE_ERR_INVALID;
  if (!dy || !w || !offsets || !dx) return MOE_ERR_INVALID;
  return run_dx({s, dt, dx_dt, dy, w, dy2, w2, offsets, dx, 0, dev_status, as_stream(stream)});
}

MOE_EXPORT moe_status moe_grouped_linear_dw(const moe_grouped_shape *s, const void *dy,
                                            moe_dtype dt, const void *x, const int32_t *offsets,
                                            void *dw, moe_dtype dw_dt, int32_t accumulate,
                                            int32_t *dev_status, moe_stream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (!act_type(dt) || !act_type(dw_dt)) return MOE_ERR_UNSUPPORTED;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID;
  // without rows the row buffers may be empty (NULL), but dw is still written
  if (!offsets || !dw || (s->rows > 0 && (!dy || !x))) return MOE_ERR_INVALID;
  return run_dw({s, dt, dw_dt, dy, x, nullptr, nullptr, offsets, dw, accumulate, dev_status,
                 as_stream(stream)});
}

MOE_EXPORT moe_status moe_checkpoint_rows(const void *src, moe_dtype dt, int64_t rows, int32_t k,
                                          uint8_t *codes, uint8_t *exps, moe_stream_t stream) {
  if (rows < 0 || k < 1) return MOE_ERR_INVALID;
  if (rows >= ((int64_t)1 << 31) || k > (1 << 20) || !act_type(dt)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!src || !codes || !exps) return MOE_ERR_INVALID;
  cudaStream_t cs = as_stream(stream);
  const int nb = scale_blocks(k);
  if (k % 8 == 0 && aligned(src, 16) && aligned(codes, 8)) {
    const int per = 32 * ckpt::UNROLL;
    const unsigned grid = row_grid(rows * ((nb * 4 + per - 1) / per));
    if (dt == MOE_F32)
      ckpt::save_rows_v8<<<grid, ckpt::ROW_THREADS, 0, cs>>>(static_cast<const float *>(src), rows, k, codes, exps);
    else
      ckpt::save_rows_v8<<<grid, ckpt::ROW_THREADS, 0, cs>>>(static_cast<const bf16 *>(src), rows, k, codes, exps);
    return launch_status();
  }
  const unsigned grid = row_grid(rows * nb);
  if (dt == MOE_F32)
    ckpt::save_rows<<<grid, ckpt::ROW_THREADS, 0, cs>>>(static_cast<const float *>(src), rows, k, codes, exps);
  else
    ckpt::save_rows<<<grid, ckpt::ROW_THREADS, 0, cs>>>(static_cast<const bf16 *>(src), rows, k, codes, exps);
  return launch_status();
}

MOE_EXPORT moe_status moe_restore_rows(const uint8_t *codes, const uint8_t *exps, int64_t rows,
                                       int32_t k, const int32_t *index, int64_t n, void *out,
                                       moe_dtype out_dt, int32_t *dev_status,
                                       moe_stream_t stream) {
  if (rows < 0 || n < 0 || k < 1) return MOE_ERR_INVALID;
  if (rows >= ((int64_t)1 << 31) || n >= ((int64_t)1 << 31) || k > (1 << 20) || !act_type(out_dt))
    return MOE_ERR_UNSUPPORTED;
  if (!index && n > rows) return MOE_ERR_INVALID;
  if (n == 0) return MOE_OK;
  if (!out || (rows > 0 && (!codes || !exps))) return MOE_ERR_INVALID;
  cudaStream_t cs = as_stream(stream);
  const int nb = scale_blocks(k);
  if (k % 8 == 0 && aligned(out, 16) && aligned(codes, 8)) {
    const int per = 32 * ckpt::UNROLL;
    const unsigned grid = row_grid(n * ((nb * 4 + per - 1) / per));
    if (out_dt == MOE_F32)
      ckpt::load_rows_v8<<<grid, ckpt::ROW_THREADS, 0, cs>>>(codes, exps, rows, k, index, n, static_cast<float *>(out), dev_status);
    else
      ckpt::load_rows_v8<<<grid, ckpt::ROW_THREADS, 0, cs>>>(codes, exps, rows, k, index, n, static_cast<bf16 *>(out), dev_status);
    return launch_status();
  }
  const unsigned grid = row_grid(n * nb);
  if (out_dt == MOE_F32)
    ckpt::load_rows<<<grid, ckpt::ROW_THREADS, 0, cs>>>(codes, exps, rows, k, index, n, static_cast<float *>(out), dev_status);
  else
    ckpt::load_rows<<<grid, ckpt::ROW_THREADS, 0, cs>>>(codes, exps, rows, k, index, n, static_cast<bf16 *>(out), dev_status);
  return launch_status();
}

MOE_EXPORT size_t moe_swiglu_checkpoint_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                                       int32_t aligned) {
  if (check_shape(s) != MOE_OK || !act_type(dt)) return 0;
  if (aligned && tc_up_sizes(s, dt)) return 0;
  return 2 * align_up((size_t)s->rows * s->n * 4, 256);  // the two projections in fp32
}

MOE_EXPORT moe_status moe_swiglu_checkpoint(const moe_grouped_shape *s, const void *x,
                                            moe_dtype dt, const void *w1, const void *w3,
                                            const int32_t *offsets, void *h, uint8_t *codes_a,
                                            uint8_t *exps_a, uint8_t *codes_u, uint8_t *exps_u,
                                            void *ws, size_t ws_bytes, int32_t *dev_status,
                                            moe_stream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (!act_type(dt)) return MOE_ERR_UNSUPPORTED;
  if (s->rows == 0) return MOE_OK;
  if (!x || !w1 || !w3 || !offsets || !h || !codes_a || !exps_a || !codes_u || !exps_u)
    return MOE_ERR_INVALID;
  cudaStream_t cs = as_stream(stream);
  const ckpt::Saved sv{codes_a, exps_a, codes_u, exps_u};
  const bool tc = tc_up_sizes(s, dt) && aligned(x, 16) && aligned(w1, 16) && aligned(w3, 16) &&
                  aligned(h, 8) && aligned(codes_a, 4) && aligned(codes_u, 4);
  const size_t need = moe_swiglu_checkpoint_workspace_size(s, dt, tc);
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (tc) {
    tcg::RowParams r = {};
    r.offsets = offsets;
    r.out = h;
    r.status = dev_status;
    r.saved = sv;
    return tc_up(s, x, w1, w3, r, cs);
  }
  float *a = static_cast<float *>(ws);
  float *u = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + align_up((size_t)s->rows * s->n * 4, 256));
  if ((st = run_linear({s, dt, MOE_F32, x, w1, nullptr, nullptr, offsets, a, 0, dev_status, cs})) != MOE_OK)
    return st;
  if ((st = run_linear({s, dt, MOE_F32, x, w3, nullptr, nullptr, offsets, u, 0, dev_status, cs})) != MOE_OK)
    return st;
  const unsigned grid = row_grid(s->rows * scale_blocks(s->n));
  if (dt == MOE_F32)
    ckpt::swiglu_save<<<grid, ckpt::ROW_THREADS, 0, cs>>>(a, u, offsets, s->groups, s->rows, s->n, static_cast<float *>(h), sv);
  else
    ckpt::swiglu_save<<<grid, ckpt::ROW_THREADS, 0, cs>>>(a, u, offsets, s->groups, s->rows, s->n, static_cast<bf16 *>(h), sv);
  return launch_status();
}

MOE_EXPORT size_t moe_swiglu_backward_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                                     int32_t aligned) {
  if (check_shape(s) != MOE_OK || !act_type(dt)) return 0;
  // one term of dgate for 32 hidden features, or dh in fp32
  if (aligned && tc_bwd_sizes(s, dt)) return (size_t)s->rows * scale_blocks(s->n) * 4;
  return (size_t)s->rows * s->n * 4;
}

MOE_EXPORT moe_status moe_swiglu_backward(const moe_grouped_shape *s, const void *dy, moe_dtype dt,
                                          const void *w2, const uint8_t *codes_a,
                                          const uint8_t *exps_a, const uint8_t *codes_u,
                                          const uint8_t *exps_u, const float *gate,
                                          const int32_t *offsets, void *da, void *du, void *hg,
                                          float *dgate, void *ws, size_t ws_bytes,
                                          int32_t *dev_status, moe_stream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (!act_type(dt)) return MOE_ERR_UNSUPPORTED;
  if (s->rows == 0) return MOE_OK;
  if (!dy || !w2 || !codes_a || !exps_a || !codes_u || !exps_u || !offsets || !da || !du || !hg ||
      !dgate)
    return MOE_ERR_INVALID;
  cudaStream_t cs = as_stream(stream);
  const ckpt::Saved sv{const_cast<uint8_t *>(codes_a), const_cast<uint8_t *>(exps_a),
                       const_cast<uint8_t *>(codes_u), const_cast<uint8_t *>(exps_u)};
  const bool tc = tc_bwd_sizes(s, dt) && aligned(dy, 16) && aligned(w2, 16) && aligned(codes_a, 4) &&
                  aligned(codes_u, 4) && aligned(da, 8) && aligned(du, 8) && aligned(hg, 8);
  if (!ws || ws_bytes < moe_swiglu_backward_workspace_size(s, dt, tc)) return MOE_ERR_WORKSPACE;
  if (tc) {
    tcg::RowParams r = {};
    r.offsets = offsets;
    r.status = dev_status;
    r.saved = sv;
    r.gate = gate;
    r.da = static_cast<bf16 *>(da);
    r.du = static_cast<bf16 *>(du);
    r.hg = static_cast<bf16 *>(hg);
    r.part = static_cast<float *>(ws);
    if ((st = tc_bwd(s, dy, w2, r, cs)) != MOE_OK) return st;
    tcg::sum_parts<<<(unsigned)((s->rows + 255) / 256), 256, 0, cs>>>(
        r.part, offsets, s->groups, s->rows, scale_blocks(s->n), dgate);
    return launch_status();
  }
  float *dh = static_cast<float *>(ws);
  // dh = dy w2: the input gradient of a linear layer from n features to k
  const moe_grouped_shape lin{s->groups, s->k, s->n, s->rows};
  if ((st = run_dx({&lin, dt, MOE_F32, dy, w2, nullptr, nullptr, offsets, dh, 0, dev_status, cs})) != MOE_OK)
    return st;
  const unsigned grid = row_grid(s->rows * (ckpt::ROW_THREADS / 32));
  if (dt == MOE_F32)
    ckpt::swiglu_grads<<<grid, ckpt::ROW_THREADS, 0, cs>>>(
        dh, sv, gate, offsets, s->groups, s->rows, s->n, static_cast<float *>(da),
        static_cast<float *>(du), static_cast<float *>(hg), dgate);
  else
    ckpt::swiglu_grads<<<grid, ckpt::ROW_THREADS, 0, cs>>>(
        dh, sv, gate, offsets, s->groups, s->rows, s->n, static_cast<bf16 *>(da),
        static_cast<bf16 *>(du), static_cast<bf16 *>(hg), dgate);
  return launch_status();
}

MOE_EXPORT moe_status moe_training_rows(const moe_cfg *cfg, int64_t T, const int32_t *offsets,
                                        const int32_t *sorted_token, const int32_t *slot_of,
                                        const float *weights, int32_t *row_token, float *row_gate,
                                        int32_t *group_offsets, int32_t *dev_status,
                                        moe_stream_t stream) {
  const moe_status st = check_cfg(cfg);
  if (st != MOE_OK) return st;
  if (T < 0) return MOE_ERR_INVALID;
  if (cfg->n_shared > 1 || T * ((int64_t)cfg->topk + cfg->n_shared) >= ((int64_t)1 << 31))
    return MOE_ERR_UNSUPPORTED;
  if (!offsets || !group_offsets) return MOE_ERR_INVALID;
  if (T > 0 && (!sorted_token || !slot_of || !weights || !row_token || !row_gate))
    return MOE_ERR_INVALID;
  const int64_t items = T * (cfg->topk + cfg->n_shared) + cfg->n_routed + 2;
  const int64_t blocks = (items + 255) / 256;
  ckpt::training_rows<<<(unsigned)(blocks < 1184 ? blocks : 1184), 256, 0, as_stream(stream)>>>(
      offsets, sorted_token, slot_of, weights, T, cfg->topk, cfg->n_routed, cfg->n_shared, row_token,
      row_gate, group_offsets, dev_status);
  return launch_status();
}

template <typename TI, typename TO>
static void launch_gather(bool vec, unsigned grid, const void *src, int64_t rows, int32_t k,
                          const int32_t *index, int64_t n, void *out, int32_t *status,
                          cudaStream_t s) {
  if (vec)
    ckpt::gather_rows<TI, TO, true><<<grid, ckpt::ROW_THREADS, 0, s>>>(
        static_cast<const TI *>(src), rows, k, index, n, static_cast<TO *>(out), status);
  else
    ckpt::gather_rows<TI, TO, false><<<grid, ckpt::ROW_THREADS, 0, s>>>(
        static_cast<const TI *>(src), rows, k, index, n, static_cast<TO *>(out), status);
}

MOE_EXPORT moe_status moe_gather_rows(const void *src, moe_dtype dt, int64_t rows, int32_t k,
                                      const int32_t *index, int64_t n, void *out, moe_dtype out_dt,
                                      int32_t *dev_status, moe_stream_t stream) {
  if (rows < 0 || n < 0 || k < 1) return MOE_ERR_INVALID;
  if (rows >= ((int64_t)1 << 31) || n >= ((int64_t)1 << 31) || k > (1 << 20) || !act_type(dt) ||
      !act_type(out_dt))
    return MOE_ERR_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  if (!index || !out || (rows > 0 && !src)) return MOE_ERR_INVALID;
  const bool vec = k % 8 == 0 && aligned(src, 16) && aligned(out, 16);
  const int per = 32 * ckpt::UNROLL * (vec ? 8 : 1);
  const unsigned grid = row_grid(n * ((k + per - 1) / per));
  cudaStream_t cs = as_stream(stream);
  if (dt == MOE_F32 && out_dt == MOE_F32)
    launch_gather<float, float>(vec, grid, src, rows, k, index, n, out, dev_status, cs);
  else if (dt == MOE_F32)
    launch_gather<float, bf16>(vec, grid, src, rows, k, index, n, out, dev_status, cs);
  else if (out_dt == MOE_F32)
    launch_gather<bf16, float>(vec, grid, src, rows, k, index, n, out, dev_status, cs);
  else
    launch_gather<bf16, bf16>(vec, grid, src, rows, k, index, n, out, dev_status, cs);
  return launch_status();
}
