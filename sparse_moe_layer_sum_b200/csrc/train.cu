// moe_train: training operators of the experts (moe_train.h) -- host checks,
// the choice of kernel and the launches.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "ckpt.cuh"
#include "common.cuh"
#include "grouped.cuh"
#include "grouped_simt.cuh"
#include "grouped_tc.cuh"
#include "moe_train.h"

namespace moe {
namespace {

using grouped::bf16;

// SMs of a B200: what the choices that size a workspace go by, without asking
// a device
constexpr int SMS = 148;

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
  if (a.splits > 1) return launch_simt<TI, TO, DIR, 32>(a, tiles(32) * a.splits, nsm, s);
  // the larger tile reuses each operand value more often; the smaller ones
  // where the larger would leave SMs without work.  (Empty groups count here:
  // with many groups of a row or two the larger tiles mostly multiply rows that
  // do not exist.)
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
  void *ws;
  size_t ws_bytes;
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
  a.splits = 1;
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
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
    // a device that was reset has forgotten the shared-memory limit
    cudaGetLastError();
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_MAX) !=
            cudaSuccess ||
        cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return launch_status();
}

// Upper bound on the row tiles of all groups.
int64_t row_tiles(const moe_grouped_shape *s, int bn) {
  return s->rows / bn + (s->rows < s->groups ? s->rows : s->groups);
}

// ------------------------------------------------------------------ staging

// A matrix that a tensor-core product reads: rows x cols, row-major.
struct Operand {
  const void *p;
  int64_t rows;
  int cols;
};

int padded(int cols) { return (cols + 7) / 8 * 8; }

// How a product runs.  direct: TMA reads the operands as they are.  staged:
// through bf16 copies in the workspace (see stage_rows).  Otherwise on the
// CUDA cores.
struct Plan {
  bool direct = false, staged = false;
  int terms = 1;         // planes of a staged operand
  size_t bytes = 0;      // of the staged operands
  int splits = 1;        // parts of the contraction that are computed apart
  size_t part = 0;       // bytes of their fp32 planes
  size_t total() const { return bytes + part; }
  bool tensor() const { return direct || staged; }
};

// The kinds of product, and the number of operations from which staging beats
// the CUDA cores, by operand type.  Below, the copies and their launches cost
// more than they save; dw crosses late because its results off the pitch are
// stored without TMA.  Measured on 28 random shapes either side, none of them
// with many groups of few rows, whose weights are all copied; for example
// linear, bf16: 1.2e7 12.3 (CUDA cores) / 10.6 us (staged), 2.2e8 30 / 13 us;
// dw, bf16: 2.2e8 18.4 / 18.2 us, 8.3e8 48 / 29 us; linear, fp32: 2e8 16.6 /
// 16.7 us, 2.1e9 122 / 61 us; backward, fp32: 9e8 52 / 86 us, 2.1e9 121 / 82 us.
enum Kind { K_LINEAR, K_DX, K_DW, K_UP, K_BWD };
double staging_from(Kind k, moe_dtype dt) {
  if (dt == MOE_F32) return k == K_BWD || k == K_DW ? 1e9 : 2e8;
  return k == K_DW ? 5e8 : k == K_BWD ? 1e8 : 1e7;
}

// aligned: every operand is 16-byte aligned (their addresses are not looked at).
Plan plan(Kind kind, const Operand *ops, int n, moe_dtype dt, double flops, bool aligned) {
  Plan p;
  p.terms = dt == MOE_F32 ? tcg::SPLIT_TERMS : 1;
  bool fits = dt == MOE_BF16;
  for (int i = 0; i < n; ++i) {
    fits = fits && aligned && ops[i].cols % 8 == 0;
    if (ops[i].rows * p.terms >= ((int64_t)1 << 31)) {  // row coordinates are 32-bit
      p.bytes = 0;
      return p;
    }
    p.bytes += align_up((size_t)ops[i].rows * padded(ops[i].cols) * p.terms * 2, 256);
  }
  if (fits) {
    p.direct = true;
    p.bytes = 0;
    return p;
  }
  p.staged = flops >= staging_from(kind, dt);
  if (!p.staged) p.bytes = 0;
  return p;
}

bool all_aligned(const Operand *ops, int n) {
  for (int i = 0; i < n; ++i)
    if (!aligned(ops[i].p, 16)) return false;
  return true;
}

// Copies every operand into the workspace and points it there.
moe_status stage(Operand *ops, int n, moe_dtype dt, void *ws, cudaStream_t s) {
  uint8_t *at = static_cast<uint8_t *>(ws);
  const int nsm = sm_count();
  if (nsm < 1) return MOE_ERR_CUDA;
  for (int i = 0; i < n; ++i) {
    const int kp = padded(ops[i].cols);
    const int64_t blocks = (ops[i].rows * (kp / 8) + 255) / 256, most = (int64_t)nsm * 8;
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    bf16 *dst = reinterpret_cast<bf16 *>(at);
    if (dt == MOE_F32)
      tcg::stage_rows<float, tcg::SPLIT_TERMS><<<grid, 256, 0, s>>>(static_cast<const float *>(ops[i].p), ops[i].rows, ops[i].cols, kp, dst);
    else
      tcg::stage_rows<bf16, 1><<<grid, 256, 0, s>>>(static_cast<const bf16 *>(ops[i].p), ops[i].rows, ops[i].cols, kp, dst);
    const moe_status st = launch_status();
    if (st != MOE_OK) return st;
    at += align_up((size_t)ops[i].rows * kp * (dt == MOE_F32 ? tcg::SPLIT_TERMS : 1) * 2, 256);
    ops[i].p = dst;
    ops[i].cols = kp;
  }
  return MOE_OK;
}

// --------------------------------------------------------- tensor-core launches

// A product with one result row per input row: F features, contracting over
// `contract` values; x and w as planned (w1, x1: a second weight or source).
struct RowJob {
  const moe_grouped_shape *s;
  int F, contract, terms;
  Operand x0, w0, x1, w1;  // w1, x1: p NULL if there is none
  tcg::RowParams p;
  cudaStream_t stream;
};

template <int OP, int CG, int AT, int BN, int STAGES, bool SEGS, typename TO>
moe_status launch_rows(const RowJob &j) {
  using C = tcg::RowCfg<OP, CG, AT, BN, STAGES, SEGS>;
  const moe_grouped_shape *s = j.s;
  const uint64_t planes = (uint64_t)j.terms * s->groups, wrows = C::KMAJOR ? j.F : j.contract;
  auto wmap = [&](CUtensorMap *t, const Operand &w) {
    return tensor_map(t, w.p, MOE_BF16, planes, wrows, w.cols, C::KMAJOR ? tcg::BM : 64);
  };
  auto xmap = [&](CUtensorMap *t, const Operand &x) {
    return tensor_map(t, x.p, MOE_BF16, 0, (uint64_t)j.terms * s->rows, x.cols, C::BOXN);
  };
  CUtensorMap a0, a1, b0, b1;
  if (!wmap(&a0, j.w0) || !xmap(&b0, j.x0)) return MOE_ERR_CUDA;
  a1 = a0;
  b1 = b0;
  if ((j.w1.p && !wmap(&a1, j.w1)) || (j.x1.p && !xmap(&b1, j.x1))) return MOE_ERR_CUDA;
  tcg::RowParams p = j.p;
  p.G = s->groups;
  p.F = j.F;
  p.rows = s->rows;
  p.passes = j.terms == 1 ? 1 : tcg::SPLIT_PASSES;
  p.kb0 = (j.contract + tcg::BK - 1) / tcg::BK;
  p.kb = p.kb0 * p.passes * (j.x1.p ? 2 : 1);
  const int64_t tiles = row_tiles(s, BN) * ((j.F + C::FEAT - 1) / C::FEAT) * (p.splits ? p.splits : 1);
  return launch_persistent<tcg::rows_gemm<OP, CG, AT, BN, STAGES, SEGS, TO>>(
      C::NT, C::smem(p.G), CG, tiles, j.stream, a0, a1, b0, b1, (const tcg::RowParams)p);
}

// rows of a group on average
int64_t mean_rows(const moe_grouped_shape *s) { return (s->rows + s->groups - 1) / s->groups; }

// Whether tiles of bn rows by feat features are the better choice: the groups
// are long enough to fill them, and there are enough for half the SM pairs.
// The narrow tiles (64 rows, 128 features, one SM) read the weights once for
// every 64 rows but keep more SMs busy.  Linear, narrow / wide: 4 groups, 1000
// rows, 1024 x 1024: 12 / 23 us; 32 groups, 2000 rows: 18.6 / 19.9 us; dx,
// 4 groups, 300 rows, 2048 -> 7168: 54 / 28.5 us.
bool wide(const RowJob &j, int bn, int feat) {
  return mean_rows(j.s) > 48 && row_tiles(j.s, bn) * ((j.F + feat - 1) / feat) >= SMS / 4;
}

template <int OP, typename TO>
moe_status tc_rows(const RowJob &j) {
  // fp32 results, and long sums: in segments (65600 values, 640 rows to 1024
  // 431 -> 438 us, 4096 rows to 2048 774 -> 1029 us)
  if (sizeof(TO) == 4 || (int64_t)j.contract * (j.x1.p ? 2 : 1) > tcg::LONG_SUM) {
    if (wide(j, 256, 256)) return launch_rows<OP, 2, 1, 256, 6, true, TO>(j);
    return launch_rows<OP, 1, 1, 64, 8, true, TO>(j);
  }
  if constexpr (sizeof(TO) == 2) {
    if (wide(j, 256, 512)) return launch_rows<OP, 2, 2, 256, 4, false, TO>(j);
    return launch_rows<OP, 1, 1, 64, 8, false, TO>(j);
  }
  return MOE_ERR_UNSUPPORTED;  // not reached
}

// The first matmul with its checkpoint, and the gradients of the hidden rows.
template <typename TO>
moe_status tc_up(const RowJob &j) {
  if (wide(j, 128, 256)) return launch_rows<tcg::UP, 2, 2, 128, 5, true, TO>(j);
  return launch_rows<tcg::UP, 1, 2, 64, 5, true, TO>(j);
}

template <typename TO>
moe_status tc_bwd(const RowJob &j) {
  if (wide(j, 256, 256)) return launch_rows<tcg::BWD, 2, 1, 256, 6, true, TO>(j);
  return launch_rows<tcg::BWD, 1, 1, 64, 8, true, TO>(j);
}

template <typename TO, int AT, bool SEGS>
moe_status launch_dw(const Product &p, const Operand *ops, int terms, int splits = 1, int above = -1,
                     int upto = INT32_MAX) {
  using C = tcg::DwCfg<TO, AT, SEGS>;
  const auto *s = p.s;
  const uint64_t rows = (uint64_t)terms * s->rows;
  const bool store = aligned(p.out, 16) && (int64_t)s->k * sizeof(TO) % 16 == 0;
  CUtensorMap a, b, c;
  if (!tensor_map(&a, ops[0].p, MOE_BF16, 0, rows, ops[0].cols, tcg::BK) ||
      !tensor_map(&b, ops[1].p, MOE_BF16, 0, rows, ops[1].cols, tcg::BK))
    return MOE_ERR_CUDA;
  c = a;
  if (store && !tensor_map(&c, p.out, p.out_dt, (uint64_t)splits * s->groups, s->n, s->k, 32)) return MOE_ERR_CUDA;
  const tcg::DwParams d{p.offsets, s->groups, s->n, s->k, s->rows, p.out, p.accumulate,
                        terms == 1 ? 1 : tcg::SPLIT_PASSES, splits, above, upto, store, p.status};
  const int64_t tiles = (int64_t)s->groups * splits * ((s->n + C::FEAT - 1) / C::FEAT) * ((s->k + 255) / 256);
  return launch_persistent<tcg::dw_gemm<TO, AT, SEGS>>(C::NT, (size_t)C::BYTES, 2, tiles, p.stream, a, b, c, d);
}

moe_status tc_dw(const Product &p, const Operand *ops, int terms) {
  if (p.out_dt == MOE_F32) return launch_dw<float, 1, true>(p, ops, terms);
  // a bf16 sum with what is there already adds in fp32, which the packed
  // results of the wider tile no longer are
  const bool narrow = p.accumulate || p.s->n <= 256;
  if (p.s->rows <= tcg::LONG_SUM)
    return narrow ? launch_dw<bf16, 1, false>(p, ops, terms) : launch_dw<bf16, 2, false>(p, ops, terms);
  // Groups that may be long: those that are, by a launch whose sums go in
  // segments.  2048 x 4096: 32 groups of 2200 rows, none of them long, 831 ->
  // 836 us; with one of 73728 rows among them 1630 -> 1900 us; one of 200000
  // rows 2.27 -> 3.11 ms, where one launch cuts positive sums by 7e-4.
  const moe_status st = narrow ? launch_dw<bf16, 1, false>(p, ops, terms, 1, -1, tcg::LONG_SUM)
                               : launch_dw<bf16, 2, false>(p, ops, terms, 1, -1, tcg::LONG_SUM);
  return st != MOE_OK ? st : launch_dw<bf16, 1, true>(p, ops, terms, 1, tcg::LONG_SUM);
}

// ---------------------------------------------------- operands of the products

double flops_of(const moe_grouped_shape *s, int products) {
  return 2.0 * products * (double)s->rows * s->n * s->k;
}

int linear_ops(const moe_grouped_shape *s, const void *x, const void *w, Operand *o) {
  o[0] = {x, s->rows, s->k};
  o[1] = {w, (int64_t)s->groups * s->n, s->k};
  return 2;
}
int dx_ops(const moe_grouped_shape *s, const void *dy, const void *w, const void *dy2, const void *w2,
           bool two, Operand *o) {
  o[0] = {dy, s->rows, s->n};
  o[1] = {w, (int64_t)s->groups * s->n, s->k};
  o[2] = {dy2, s->rows, s->n};
  o[3] = {w2, (int64_t)s->groups * s->n, s->k};
  return two ? 4 : 2;
}
int dw_ops(const moe_grouped_shape *s, const void *dy, const void *x, Operand *o) {
  o[0] = {dy, s->rows, s->n};
  o[1] = {x, s->rows, s->k};
  return 2;
}
int up_ops(const moe_grouped_shape *s, const void *x, const void *w1, const void *w3, Operand *o) {
  o[0] = {x, s->rows, s->k};
  o[1] = {w1, (int64_t)s->groups * s->n, s->k};
  o[2] = {w3, (int64_t)s->groups * s->n, s->k};
  return 3;
}
int bwd_ops(const moe_grouped_shape *s, const void *dy, const void *w2, Operand *o) {
  o[0] = {dy, s->rows, s->k};
  o[1] = {w2, (int64_t)s->groups * s->k, s->n};
  return 2;
}

// Few tiles leave SMs idle while each works through a long contraction: it is
// cut into parts, the partial results go to the workspace in fp32 and are
// added in a fixed order.  Linear, one group of 200 rows, 7168 -> 2048: 42 ->
// 29 us.  dw, one group of 4096 rows, 512 x 512: 43 -> 17 us; it takes three
// parts of 512 rows to pay (two of 256: 8.8 -> 12.3 us).
void split_rows_product(Plan &p, const moe_grouped_shape *s, int F, int contract, int sources) {
  if (!p.tensor()) return;
  const int64_t tiles = row_tiles(s, 64) * ((F + 127) / 128);
  const int64_t kb = (int64_t)((contract + tcg::BK - 1) / tcg::BK) * sources *
                     (p.terms == 1 ? 1 : tcg::SPLIT_PASSES);
  // parts of a segment (8 k-blocks) at least
  int64_t n = std::min<int64_t>({16, SMS / (tiles < 1 ? 1 : tiles), kb / 8});
  if (n < 2) return;
  const int64_t per = (kb + n - 1) / n;
  n = (kb + per - 1) / per;  // none of them empty
  p.splits = (int)n;
  p.part = align_up((size_t)n * s->rows * F * 4, 256);
}

void split_dw_product(Plan &p, const moe_grouped_shape *s) {
  if (!p.tensor()) return;
  const int64_t tiles = (int64_t)s->groups * ((s->n + 255) / 256) * ((s->k + 255) / 256);
  const int64_t n = std::min<int64_t>({16, SMS / 2 / tiles, mean_rows(s) / 512});
  if (n < 3) return;
  p.splits = (int)n;
  p.part = align_up((size_t)n * s->groups * s->n * s->k * 4, 256);
}

// The same on the CUDA cores, whose smallest tile is 32 x 32 and whose slices
// are 64 deep (dx of two products, 6 groups, 5 rows, 1104 -> 64, fp32: 41 ->
// 10 us).
void split_simt_product(Plan &p, Kind kind, const moe_grouped_shape *s, int products) {
  if (p.tensor()) return;
  const int cols = kind == K_LINEAR ? s->n : s->k;
  const int64_t contract = kind == K_LINEAR ? s->k : kind == K_DX ? s->n : mean_rows(s);
  auto tiles = [&](int t) {
    const int64_t ct = (cols + t - 1) / t;
    return kind == K_DW ? (int64_t)s->groups * ((s->n + t - 1) / t) * ct : row_tiles(s, t) * ct;
  };
  if (tiles(64) >= SMS) return;  // enough of the larger ones
  int64_t n = std::min<int64_t>({16, 2 * SMS / std::max<int64_t>(1, tiles(32)),
                                 (contract + 63) / 64 * products / 3});
  if (n < 3) return;
  p.splits = (int)n;
  p.part = align_up((size_t)n * 4 * (kind == K_DW ? (size_t)s->groups * s->n * s->k : (size_t)s->rows * cols), 256);
}

Plan plan_product(Kind kind, const moe_grouped_shape *s, const Operand *o, int n, moe_dtype dt,
                  int products, bool aligned) {
  Plan p = plan(kind, o, n, dt, flops_of(s, products), aligned);
  if (kind == K_LINEAR) split_rows_product(p, s, s->n, s->k, products);
  if (kind == K_DX) split_rows_product(p, s, s->k, s->n, products);
  if (kind == K_DW) split_dw_product(p, s);
  split_simt_product(p, kind, s, products);
  return p;
}

// Bytes of workspace that a product takes: with aligned operands, or with any
// (aligned ones can take the more: parts of a tensor-core product).
size_t product_workspace(Kind kind, const moe_grouped_shape *s, const Operand *o, int n, moe_dtype dt,
                         int products, bool aligned) {
  const size_t least = plan_product(kind, s, o, n, dt, products, true).total();
  return aligned ? least : std::max(least, plan_product(kind, s, o, n, dt, products, false).total());
}

// The plan for operands whose addresses are known.  Without the workspace a
// staged product runs on the CUDA cores, a direct one undivided.
Plan plan_call(Kind kind, const moe_grouped_shape *s, const Operand *o, int n, moe_dtype dt, int products,
               const void *ws, size_t ws_bytes) {
  Plan p = plan_product(kind, s, o, n, dt, products, all_aligned(o, n));
  if (p.total() && (!ws || !aligned(ws, 16) || ws_bytes < p.total())) {
    p.staged = false;
    p.splits = 1;
    p.bytes = p.part = 0;
  }
  return p;
}

// out = the sum of the splits' planes behind the staged operands.
moe_status join(const Plan &pl, const Product &p, int64_t rows, int64_t cols, const int32_t *offsets) {
  const float *part = reinterpret_cast<const float *>(static_cast<const uint8_t *>(p.ws) + pl.bytes);
  const int64_t blocks = (rows * cols + 255) / 256, most = SMS * 8;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  if (p.out_dt == MOE_F32)
    tcg::sum_splits<<<grid, 256, 0, p.stream>>>(part, pl.splits, offsets, p.s->groups, rows, cols, static_cast<float *>(p.out), p.accumulate);
  else
    tcg::sum_splits<<<grid, 256, 0, p.stream>>>(part, pl.splits, offsets, p.s->groups, rows, cols, static_cast<bf16 *>(p.out), p.accumulate);
  return launch_status();
}

// On the CUDA cores, in parts if the plan says so.
template <int DIR>
moe_status run_simt(const Plan &pl, const Product &p, int64_t rows, int64_t cols,
                    const int32_t *offsets) {
  simt::Args a = simt_args(p);
  if (pl.splits == 1) return simt_product<DIR>(a, p.dt, p.out_dt, p.stream);
  a.splits = pl.splits;
  a.c = static_cast<uint8_t *>(p.ws) + pl.bytes;
  a.accumulate = 0;
  const moe_status st = simt_product<DIR>(a, p.dt, MOE_F32, p.stream);
  return st != MOE_OK ? st : join(pl, p, rows, cols, offsets);
}

template <int OP>
moe_status run_rows(const Plan &pl, const Product &p, RowJob &j) {
  j.p.offsets = p.offsets;
  j.p.status = p.status;
  j.p.splits = pl.splits;
  j.p.out = p.out;
  if (pl.splits > 1) {
    j.p.out = static_cast<uint8_t *>(p.ws) + pl.bytes;
    const moe_status st = launch_rows<OP, 1, 1, 64, 8, true, float>(j);
    return st != MOE_OK ? st : join(pl, p, p.s->rows, j.F, p.offsets);
  }
  return p.out_dt == MOE_F32 ? tc_rows<OP, float>(j) : tc_rows<OP, bf16>(j);
}

moe_status run_linear(const Product &p) {
  Operand o[4];
  const int n = linear_ops(p.s, p.a0, p.b0, o);
  const Plan pl = plan_call(K_LINEAR, p.s, o, n, p.dt, 1, p.ws, p.ws_bytes);
  if (!pl.tensor()) return run_simt<simt::LIN>(pl, p, p.s->rows, p.s->n, p.offsets);
  if (pl.staged) {
    const moe_status st = stage(o, n, p.dt, p.ws, p.stream);
    if (st != MOE_OK) return st;
  }
  RowJob j{p.s, p.s->n, p.s->k, pl.terms, o[0], o[1], {}, {}, {}, p.stream};
  return run_rows<tcg::LIN>(pl, p, j);
}

moe_status run_dx(const Product &p) {
  Operand o[4];
  const bool two = p.a1 != nullptr;
  const int n = dx_ops(p.s, p.a0, p.b0, p.a1, p.b1, two, o);
  const Plan pl = plan_call(K_DX, p.s, o, n, p.dt, two ? 2 : 1, p.ws, p.ws_bytes);
  if (!pl.tensor()) return run_simt<simt::DX>(pl, p, p.s->rows, p.s->k, p.offsets);
  if (pl.staged) {
    const moe_status st = stage(o, n, p.dt, p.ws, p.stream);
    if (st != MOE_OK) return st;
  }
  RowJob j{p.s, p.s->k, p.s->n, pl.terms, o[0], o[1], o[2], o[3], {}, p.stream};
  return run_rows<tcg::DX>(pl, p, j);
}

moe_status run_dw(const Product &p) {
  Operand o[4];
  const int n = dw_ops(p.s, p.a0, p.b0, o);
  const Plan pl = plan_call(K_DW, p.s, o, n, p.dt, 1, p.ws, p.ws_bytes);
  // without rows there is nothing to map; the CUDA-core kernel writes the zeros
  if (p.s->rows == 0) return simt_product<simt::DW>(simt_args(p), p.dt, p.out_dt, p.stream);
  if (!pl.tensor()) return run_simt<simt::DW>(pl, p, (int64_t)p.s->groups * p.s->n, p.s->k, nullptr);
  if (pl.staged) {
    const moe_status st = stage(o, n, p.dt, p.ws, p.stream);
    if (st != MOE_OK) return st;
  }
  if (pl.splits > 1) {
    Product q = p;
    q.out = static_cast<uint8_t *>(p.ws) + pl.bytes;
    q.out_dt = MOE_F32;
    q.accumulate = 0;
    const moe_status st = launch_dw<float, 1, true>(q, o, pl.terms, pl.splits);
    return st != MOE_OK ? st : join(pl, p, (int64_t)p.s->groups * p.s->n, p.s->k, nullptr);
  }
  return tc_dw(p, o, pl.terms);
}

int scale_blocks(int n) { return (n + ckpt::BLOCK - 1) / ckpt::BLOCK; }

// Blocks of a kernel over rows: a resident set that walks on, or, for kernels
// that mostly write (READ_BACK), six sets, so that the SMs that are done take
// more (32768 x 7168 restored from 4096 rows: 92 us with one set, 79 with six,
// 78 with twelve; saving gains nothing).
constexpr int RESIDENT = 8, READ_BACK = 48;
unsigned row_grid(int64_t warps, int per_sm = RESIDENT) {
  const int64_t blocks = (warps + ckpt::ROW_THREADS / 32 - 1) / (ckpt::ROW_THREADS / 32);
  const int64_t most = SMS * per_sm;
  return (unsigned)(blocks < most ? blocks : most);
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_EXPORT size_t moe_grouped_linear_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                                    int32_t aligned) {
  if (check_shape(s) != MOE_OK || !act_type(dt)) return 0;
  Operand o[4];
  const int n = linear_ops(s, nullptr, nullptr, o);
  return product_workspace(K_LINEAR, s, o, n, dt, 1, aligned != 0);
}

MOE_EXPORT size_t moe_grouped_linear_dx_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                                       int32_t two, int32_t aligned) {
  if (check_shape(s) != MOE_OK || !act_type(dt)) return 0;
  Operand o[4];
  const int n = dx_ops(s, nullptr, nullptr, nullptr, nullptr, two != 0, o);
  return product_workspace(K_DX, s, o, n, dt, two ? 2 : 1, aligned != 0);
}

MOE_EXPORT size_t moe_grouped_linear_dw_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                                       int32_t aligned) {
  if (check_shape(s) != MOE_OK || !act_type(dt)) return 0;
  Operand o[4];
  const int n = dw_ops(s, nullptr, nullptr, o);
  return product_workspace(K_DW, s, o, n, dt, 1, aligned != 0);
}

MOE_EXPORT moe_status moe_grouped_linear(const moe_grouped_shape *s, const void *x, moe_dtype dt,
                                         const void *w, const int32_t *offsets, void *y,
                                         moe_dtype y_dt, void *ws, size_t ws_bytes,
                                         int32_t *dev_status, moe_stream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (!act_type(dt) || !act_type(y_dt)) return MOE_ERR_UNSUPPORTED;
  if (s->rows == 0) return MOE_OK;
  if (!x || !w || !offsets || !y) return MOE_ERR_INVALID;
  return run_linear({s, dt, y_dt, x, w, nullptr, nullptr, offsets, y, 0, ws, ws_bytes, dev_status,
                     as_stream(stream)});
}

MOE_EXPORT moe_status moe_grouped_linear_dx(const moe_grouped_shape *s, const void *dy,
                                            moe_dtype dt, const void *w, const void *dy2,
                                            const void *w2, const int32_t *offsets, void *dx,
                                            moe_dtype dx_dt, void *ws, size_t ws_bytes,
                                            int32_t *dev_status, moe_stream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (!act_type(dt) || !act_type(dx_dt)) return MOE_ERR_UNSUPPORTED;
  if (s->rows == 0) return MOE_OK;  // (an empty dy2 may well be NULL)
  if ((dy2 == nullptr) != (w2 == nullptr)) return MOE_ERR_INVALID;
  if (!dy || !w || !offsets || !dx) return MOE_ERR_INVALID;
  return run_dx({s, dt, dx_dt, dy, w, dy2, w2, offsets, dx, 0, ws, ws_bytes, dev_status, as_stream(stream)});
}

MOE_EXPORT moe_status moe_grouped_linear_dw(const moe_grouped_shape *s, const void *dy,
                                            moe_dtype dt, const void *x, const int32_t *offsets,
                                            void *dw, moe_dtype dw_dt, int32_t accumulate, void *ws,
                                            size_t ws_bytes, int32_t *dev_status,
                                            moe_stream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  if (!act_type(dt) || !act_type(dw_dt)) return MOE_ERR_UNSUPPORTED;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID;
  // without rows the row buffers may be empty (NULL), but dw is still written
  if (!offsets || !dw || (s->rows > 0 && (!dy || !x))) return MOE_ERR_INVALID;
  return run_dw({s, dt, dw_dt, dy, x, nullptr, nullptr, offsets, dw, accumulate, ws, ws_bytes,
                 dev_status, as_stream(stream)});
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
  const unsigned grid = row_grid(rows * ((nb + ckpt::UNROLL1 - 1) / ckpt::UNROLL1));
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
    const unsigned grid = row_grid(n * ((nb * 4 + per - 1) / per), READ_BACK);
    if (out_dt == MOE_F32)
      ckpt::load_rows_v8<<<grid, ckpt::ROW_THREADS, 0, cs>>>(codes, exps, rows, k, index, n, static_cast<float *>(out), dev_status);
    else
      ckpt::load_rows_v8<<<grid, ckpt::ROW_THREADS, 0, cs>>>(codes, exps, rows, k, index, n, static_cast<bf16 *>(out), dev_status);
    return launch_status();
  }
  const unsigned grid = row_grid(n * ((nb + ckpt::UNROLL1 - 1) / ckpt::UNROLL1), READ_BACK);
  if (out_dt == MOE_F32)
    ckpt::load_rows<<<grid, ckpt::ROW_THREADS, 0, cs>>>(codes, exps, rows, k, index, n, static_cast<float *>(out), dev_status);
  else
    ckpt::load_rows<<<grid, ckpt::ROW_THREADS, 0, cs>>>(codes, exps, rows, k, index, n, static_cast<bf16 *>(out), dev_status);
  return launch_status();
}

// A single product on the CUDA cores.
static Plan cores_plan(Kind kind, const moe_grouped_shape *s) {
  Plan p;
  split_simt_product(p, kind, s, 1);
  return p;
}

MOE_EXPORT size_t moe_swiglu_checkpoint_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                                       int32_t aligned) {
  if (check_shape(s) != MOE_OK || !act_type(dt)) return 0;
  Operand o[4];
  const Plan p = plan(K_UP, o, up_ops(s, nullptr, nullptr, nullptr, o), dt, flops_of(s, 2), aligned);
  // on the CUDA cores: the two projections in fp32, and what their product takes
  return p.tensor() ? p.bytes : 2 * align_up((size_t)s->rows * s->n * 4, 256) + cores_plan(K_LINEAR, s).part;
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
  Operand o[4];
  const int n = up_ops(s, x, w1, w3, o);
  const bool fits = all_aligned(o, n);
  const Plan p = plan(K_UP, o, n, dt, flops_of(s, 2), fits);
  const size_t need = moe_swiglu_checkpoint_workspace_size(s, dt, fits);
  if (need && (!ws || !aligned(ws, 16) || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (p.tensor()) {
    if (p.staged && (st = stage(o, n, dt, ws, cs)) != MOE_OK) return st;
    RowJob j{s, s->n, s->k, p.terms, o[0], o[1], {}, o[2], {}, cs};
    j.p.offsets = offsets;
    j.p.out = h;
    j.p.status = dev_status;
    j.p.saved = sv;
    j.p.vec = s->n % 4 == 0 && aligned(h, 4 * elem(dt)) && aligned(codes_a, 4) && aligned(codes_u, 4);
    return dt == MOE_F32 ? tc_up<float>(j) : tc_up<bf16>(j);
  }
  const size_t plane = align_up((size_t)s->rows * s->n * 4, 256);
  float *a = static_cast<float *>(ws);
  float *u = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + plane);
  const Plan cores = cores_plan(K_LINEAR, s);
  Product lin{s, dt, MOE_F32, x, w1, nullptr, nullptr, offsets, a, 0, u + plane / 4, cores.part, dev_status, cs};
  if ((st = run_simt<simt::LIN>(cores, lin, s->rows, s->n, offsets)) != MOE_OK) return st;
  lin.b0 = w3;
  lin.out = u;
  if ((st = run_simt<simt::LIN>(cores, lin, s->rows, s->n, offsets)) != MOE_OK) return st;
  const unsigned grid = row_grid(s->rows * scale_blocks(s->n));
  if (dt == MOE_F32)
    ckpt::swiglu_save<<<grid, ckpt::ROW_THREADS, 0, cs>>>(a, u, offsets, s->groups, s->rows, s->n, static_cast<float *>(h), sv);
  else
    ckpt::swiglu_save<<<grid, ckpt::ROW_THREADS, 0, cs>>>(a, u, offsets, s->groups, s->rows, s->n, static_cast<bf16 *>(h), sv);
  return launch_status();
}

// one term of dgate for 32 hidden features
static size_t part_bytes(const moe_grouped_shape *s) {
  return align_up((size_t)s->rows * scale_blocks(s->n) * 4, 256);
}

MOE_EXPORT size_t moe_swiglu_backward_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                                     int32_t aligned) {
  if (check_shape(s) != MOE_OK || !act_type(dt)) return 0;
  Operand o[4];
  const Plan p = plan(K_BWD, o, bwd_ops(s, nullptr, nullptr, o), dt, flops_of(s, 1), aligned);
  if (p.tensor()) return part_bytes(s) + p.bytes;
  // dh in fp32, and what its product takes
  const moe_grouped_shape lin{s->groups, s->k, s->n, s->rows};
  return align_up((size_t)s->rows * s->n * 4, 256) + cores_plan(K_DX, &lin).part;
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
  Operand o[4];
  const int n = bwd_ops(s, dy, w2, o);
  const bool fits = all_aligned(o, n);
  const Plan p = plan(K_BWD, o, n, dt, flops_of(s, 1), fits);
  if (!ws || !aligned(ws, 16) || ws_bytes < moe_swiglu_backward_workspace_size(s, dt, fits))
    return MOE_ERR_WORKSPACE;
  if (p.tensor()) {
    if (p.staged && (st = stage(o, n, dt, static_cast<uint8_t *>(ws) + part_bytes(s), cs)) != MOE_OK)
      return st;
    RowJob j{s, s->n, s->k, p.terms, o[0], o[1], {}, {}, {}, cs};
    j.p.offsets = offsets;
    j.p.status = dev_status;
    j.p.saved = sv;
    j.p.gate = gate;
    j.p.da = da;
    j.p.du = du;
    j.p.hg = hg;
    j.p.part = static_cast<float *>(ws);
    const size_t v = 4 * elem(dt);
    j.p.vec = s->n % 4 == 0 && aligned(codes_a, 4) && aligned(codes_u, 4) && aligned(da, v) &&
              aligned(du, v) && aligned(hg, v);
    if ((st = dt == MOE_F32 ? tc_bwd<float>(j) : tc_bwd<bf16>(j)) != MOE_OK) return st;
    tcg::sum_parts<<<(unsigned)((s->rows + 255) / 256), 256, 0, cs>>>(
        j.p.part, offsets, s->groups, s->rows, scale_blocks(s->n), dgate);
    return launch_status();
  }
  const size_t plane = align_up((size_t)s->rows * s->n * 4, 256);
  float *dh = static_cast<float *>(ws);
  // dh = dy w2: the input gradient of a linear layer from n features to k
  const moe_grouped_shape lin{s->groups, s->k, s->n, s->rows};
  const Plan cores = cores_plan(K_DX, &lin);
  const Product q{&lin, dt, MOE_F32, dy, w2, nullptr, nullptr, offsets, dh, 0, static_cast<uint8_t *>(ws) + plane,
                  cores.part, dev_status, cs};
  if ((st = run_simt<simt::DX>(cores, q, s->rows, s->n, offsets)) != MOE_OK) return st;
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
  if (cfg->n_shared > 1 || T >= ((int64_t)1 << 31) ||  // (the product below would wrap)
      T * ((int64_t)cfg->topk + cfg->n_shared) >= ((int64_t)1 << 31))
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
  const int per = 32 * (vec ? ckpt::UNROLL * 8 : ckpt::UNROLL1);
  const unsigned grid = row_grid(n * ((k + per - 1) / per), READ_BACK);
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
