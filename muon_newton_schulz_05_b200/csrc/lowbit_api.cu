// C ABI of the dropout and 4-bit (MXFP4) operators: argument validation,
// tensor maps and launches. Nothing here allocates or synchronises; every
// check comes before the first launch.
#include <cmath>
#include <cstring>
#include <mutex>

#include "lowbit.cuh"
#include "mxfp4_gemm.cuh"

using namespace muon;

namespace {

constexpr int64_t kLimit = int64_t(1) << 31;
constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr size_t kHeader = 4096;   // workspace: the device status word at offset 0

inline bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool known_dtype(int32_t d) { return d == MUON_F32 || d == MUON_BF16; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t dtype_size(int32_t d) { return d == MUON_BF16 ? 2 : 4; }

struct Span {
  const void* p;
  size_t n;
};

bool overlaps(const Span& a, const Span& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}

bool shape_ok(int64_t count, int64_t rows, int64_t cols) {
  if (count < 1 || rows < 1 || cols < 1) return false;
  if (count >= kLimit || rows >= kMaxDim || cols >= kMaxDim) return false;
  // the factors are bounded, so these products do not overflow
  return count * rows < kLimit && count * cols < kLimit &&
         count * (ceil_div(rows, kMxTile) * ceil_div(cols, kMxTile)) < kLimit;
}

size_t data_bytes(int64_t count, int64_t rows, int64_t cols) {
  return static_cast<size_t>(count) * rows * ceil_div(cols, kMxBlock) * 16;
}

size_t scale_bytes(int64_t count, int64_t rows, int64_t cols) {
  return static_cast<size_t>(count) * ceil_div(rows, kMxTile) * ceil_div(cols, kMxTile) * kMxTileBytes;
}

muon_status check_mxfp4(const muon_mxfp4* q) {
  if (!q) return MUON_ERR_NULL;
  if (!shape_ok(q->count, q->rows, q->cols)) return MUON_ERR_SHAPE;
  if (!q->data || !q->scales) return MUON_ERR_NULL;
  if (!aligned(q->data) || !aligned(q->scales)) return MUON_ERR_ALIGN;
  return MUON_OK;
}

Span data_span(const muon_mxfp4* q) { return {q->data, data_bytes(q->count, q->rows, q->cols)}; }
Span scale_span(const muon_mxfp4* q) { return {q->scales, scale_bytes(q->count, q->rows, q->cols)}; }

// Dropout threshold (p in units of 2^-16) and the factor that belongs to it.
bool dropout_terms(double p, uint32_t* threshold, float* scale) {
  if (!(p >= 0.0 && p < 1.0)) return false;   // also refuses NaN
  const double t = std::nearbyint(p * 65536.0);
  if (t > 65535.0) return false;
  *threshold = static_cast<uint32_t>(t);
  *scale = static_cast<float>(65536.0 / (65536.0 - t));
  return true;
}

// Devices whose kernels have their attributes set.
struct LowbitDevice {
  bool quantize = false, gemm = false;
  int pairs = 0;
};
LowbitDevice g_lowbit[64];
std::mutex g_lowbit_mu;

// The current device, prepared for quantisation or (pairs given) for products.
muon_status lowbit_device(int* sms, int* pairs = nullptr) {
  const muon_status st = library_device(sms);
  if (st != MUON_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MUON_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_lowbit_mu);
  LowbitDevice& d = g_lowbit[dev];
  if (pairs) {
    if (!d.gemm && mx_gemm_prepare(&d.pairs) != cudaSuccess) return MUON_ERR_CUDA;
    d.gemm = true;
    *pairs = d.pairs;
  } else {
    if (!d.quantize && quantize_prepare() != cudaSuccess) return MUON_ERR_CUDA;
    d.quantize = true;
  }
  return MUON_OK;
}

muon_status run_quantize(QuantParams& q, int32_t dtype, int64_t count, int64_t rows, int64_t cols,
                         const muon_mxfp4* out, const muon_mxfp4* out_t, void* stream) {
  if (!q.x || (!out && !out_t)) return MUON_ERR_NULL;
  if (!shape_ok(count, rows, cols)) return MUON_ERR_SHAPE;
  if (!known_dtype(dtype)) return MUON_ERR_DTYPE;
  if (!aligned(q.x) || !aligned(q.ema) || !aligned(q.rng)) return MUON_ERR_ALIGN;
  const size_t n = static_cast<size_t>(count) * rows * cols;
  Span in[2] = {{q.x, n * dtype_size(dtype)}, {q.ema, n * 4}};
  Span w[4] = {};
  const muon_mxfp4* outs[2] = {out, out_t};
  for (int i = 0; i < 2; ++i) {
    if (!outs[i]) continue;
    const muon_status st = check_mxfp4(outs[i]);
    if (st != MUON_OK) return st;
    const int64_t r = i ? cols : rows, c = i ? rows : cols;
    if (outs[i]->count != count || outs[i]->rows != r || outs[i]->cols != c) return MUON_ERR_SHAPE;
    w[2 * i] = data_span(outs[i]);
    w[2 * i + 1] = scale_span(outs[i]);
  }
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 2; ++j)
      if (overlaps(w[i], in[j])) return MUON_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlaps(w[i], w[j])) return MUON_ERR_ALIAS;
    if (overlaps(w[i], {q.rng, 16})) return MUON_ERR_ALIAS;
  }
  int sms = 0;
  const muon_status st = lowbit_device(&sms);
  if (st != MUON_OK) return st;
  q.q = out ? static_cast<uint8_t*>(out->data) : nullptr;
  q.s = out ? static_cast<uint8_t*>(out->scales) : nullptr;
  q.qt = out_t ? static_cast<uint8_t*>(out_t->data) : nullptr;
  q.st = out_t ? static_cast<uint8_t*>(out_t->scales) : nullptr;
  q.count = static_cast<int>(count);
  q.rows = static_cast<int>(rows);
  q.cols = static_cast<int>(cols);
  q.tiles_r = static_cast<int>(ceil_div(rows, kMxTile));
  q.tiles_c = static_cast<int>(ceil_div(cols, kMxTile));
  q.fd_tiles = make_fastdiv(static_cast<uint32_t>(q.tiles_r) * static_cast<uint32_t>(q.tiles_c));
  q.fd_tiles_c = make_fastdiv(static_cast<uint32_t>(q.tiles_c));
  q.blocks_r = static_cast<int>(ceil_div(rows, kMxBlock));
  q.blocks_c = static_cast<int>(ceil_div(cols, kMxBlock));
  return launch_quantize(q, dtype == MUON_BF16, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MUON_OK
             : MUON_ERR_CUDA;
}

// ------------------------------------------------------------------- product
bool gemm_shape_ok(const MxGemmShape& s) {
  return shape_ok(s.count, s.m, s.k) && shape_ok(s.count, s.n, s.k) && shape_ok(s.count, s.m, s.n);
}

// The workspace must not depend on the device the size is asked on: the plan
// is made for a B200's 148 SMs (74 pairs); fewer only take the tiles in more
// turns.
constexpr int kPlanSms = 148;

MxGemmPlan plan_for(const MxGemmShape& s) { return plan_mx_gemm(s, kPlanSms / 2, kPlanSms); }

// Tensor maps of an operand's codes and, unless tile_box is 0, of its scale tiles.
muon_status operand_maps(const muon_mxfp4* q, int row_box, int tile_box, CUtensorMap* rows, CUtensorMap* scales) {
  const int64_t blocks = ceil_div(q->cols, kMxBlock), groups = ceil_div(blocks, 4);
  const cuuint64_t rd[3] = {static_cast<cuuint64_t>(blocks * 16), static_cast<cuuint64_t>(q->rows),
                            static_cast<cuuint64_t>(q->count)};
  const cuuint64_t rs[2] = {static_cast<cuuint64_t>(blocks * 16), static_cast<cuuint64_t>(blocks * 16 * q->rows)};
  const cuuint32_t rb[3] = {128, static_cast<cuuint32_t>(row_box), 1};
  muon_status st = encode_tiled(rows, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, q->data, rd, rs, rb,
                                CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != MUON_OK || tile_box == 0) return st;
  const cuuint64_t sd[2] = {static_cast<cuuint64_t>(groups * (kMxTileBytes / 4)),
                            static_cast<cuuint64_t>(q->count * ceil_div(q->rows, kMxTile))};
  const cuuint64_t ss[1] = {static_cast<cuuint64_t>(groups * kMxTileBytes)};
  const cuuint32_t sb[2] = {256, static_cast<cuuint32_t>(tile_box)};
  return encode_tiled(scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, q->scales, sd, ss, sb, CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace

extern "C" {

size_t muon_mxfp4_data_size(int64_t count, int64_t rows, int64_t cols) {
  return shape_ok(count, rows, cols) ? data_bytes(count, rows, cols) : 0;
}

size_t muon_mxfp4_scales_size(int64_t count, int64_t rows, int64_t cols) {
  return shape_ok(count, rows, cols) ? scale_bytes(count, rows, cols) : 0;
}

muon_status muon_dropout(const void* x, const void* residual, void* out, int32_t dtype, int64_t rows,
                         int64_t cols, double p, const int64_t* rng, uint64_t site, void* stream) {
  if (!x || !out || !rng) return MUON_ERR_NULL;
  if (rows < 1 || cols < 1 || rows >= kLimit || cols >= kMaxDim || rows * ceil_div(cols, 8) >= kLimit)
    return MUON_ERR_SHAPE;
  if (!known_dtype(dtype)) return MUON_ERR_DTYPE;
  if (!aligned(x) || !aligned(residual) || !aligned(out) || !aligned(rng)) return MUON_ERR_ALIGN;
  DropoutParams d{};
  if (!dropout_terms(p, &d.threshold, &d.scale)) return MUON_ERR_HPARAM;
  const size_t bytes = static_cast<size_t>(rows) * cols * dtype_size(dtype);
  const Span o{out, bytes};
  if ((out != x && overlaps(o, {x, bytes})) || (out != residual && overlaps(o, {residual, bytes})) ||
      overlaps(o, {rng, 16}))
    return MUON_ERR_ALIAS;
  int sms = 0;
  const muon_status st = library_device(&sms);
  if (st != MUON_OK) return st;
  d.x = x;
  d.residual = residual;
  d.out = out;
  d.rng = reinterpret_cast<const long long*>(rng);
  d.site = site;
  d.rows = rows;
  d.cols = static_cast<int>(cols);
  d.groups = static_cast<int>(ceil_div(cols, 8));
  d.fd_groups = make_fastdiv(static_cast<uint32_t>(d.groups));
  d.fd_cols = make_fastdiv(static_cast<uint32_t>(cols));
  d.total = static_cast<uint32_t>(rows * d.groups);
  return launch_dropout(d, dtype == MUON_BF16, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MUON_OK
             : MUON_ERR_CUDA;
}

muon_status muon_mxfp4_quantize(const void* x, int32_t dtype, int64_t count, int64_t rows,
                                int64_t cols, const muon_mxfp4* out, const muon_mxfp4* out_t, double p,
                                int32_t stochastic, const int64_t* rng, uint64_t site, void* stream) {
  QuantParams q{};
  if (!dropout_terms(p, &q.threshold, &q.scale) || stochastic < 0 || stochastic > 1) return MUON_ERR_HPARAM;
  if ((p > 0.0 || stochastic) && !rng) return MUON_ERR_NULL;
  q.x = x;
  q.stochastic = stochastic;
  q.rng = reinterpret_cast<const long long*>(rng);
  q.site = site;
  return run_quantize(q, dtype, count, rows, cols, out, out_t, stream);
}

muon_status muon_mxfp4_readout(const void* theta, int32_t dtype, const float* ema, float w_final,
                               int64_t count, int64_t rows, int64_t cols, const muon_mxfp4* out,
                               const muon_mxfp4* out_t, void* stream) {
  if (!ema) return MUON_ERR_NULL;
  if (!std::isfinite(w_final)) return MUON_ERR_HPARAM;
  QuantParams q{};
  q.x = theta;
  q.ema = ema;
  q.w_final = w_final;
  q.w_ema = 1.0f - w_final;
  q.scale = 1.0f;
  return run_quantize(q, dtype, count, rows, cols, out, out_t, stream);
}

muon_status muon_mxfp4_dequantize(const muon_mxfp4* q, void* out, int32_t dtype, void* stream) {
  if (!out) return MUON_ERR_NULL;
  muon_status st = check_mxfp4(q);
  if (st != MUON_OK) return st;
  if (!known_dtype(dtype)) return MUON_ERR_DTYPE;
  if (!aligned(out)) return MUON_ERR_ALIGN;
  const int64_t groups = ceil_div(q->cols, 8);
  if (q->count * q->rows * groups >= kLimit) return MUON_ERR_SHAPE;
  const Span o{out, static_cast<size_t>(q->count) * q->rows * q->cols * dtype_size(dtype)};
  if (overlaps(o, data_span(q)) || overlaps(o, scale_span(q))) return MUON_ERR_ALIAS;
  int sms = 0;
  if ((st = library_device(&sms)) != MUON_OK) return st;
  DequantParams d{};
  d.q = static_cast<const uint8_t*>(q->data);
  d.s = static_cast<const uint8_t*>(q->scales);
  d.out = out;
  d.count = static_cast<int>(q->count);
  d.rows = static_cast<int>(q->rows);
  d.cols = static_cast<int>(q->cols);
  d.blocks = static_cast<int>(ceil_div(q->cols, kMxBlock));
  d.tiles_r = static_cast<int>(ceil_div(q->rows, kMxTile));
  d.tiles_c = static_cast<int>(ceil_div(q->cols, kMxTile));
  d.groups = static_cast<int>(groups);
  d.fd_groups = make_fastdiv(static_cast<uint32_t>(groups));
  d.fd_rows = make_fastdiv(static_cast<uint32_t>(q->rows));
  d.fd_cols = make_fastdiv(static_cast<uint32_t>(q->cols));
  d.total = static_cast<uint32_t>(q->count * q->rows * groups);
  return launch_dequantize(d, dtype == MUON_BF16, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MUON_OK
             : MUON_ERR_CUDA;
}

size_t muon_mxfp4_matmul_workspace_size(int64_t count, int64_t m, int64_t n, int64_t k) {
  const MxGemmShape s{count, m, n, k};
  return gemm_shape_ok(s) ? kHeader + plan_for(s).part_bytes : 0;
}

muon_status muon_mxfp4_matmul(const muon_mxfp4* a, const muon_mxfp4* b, const void* add, void* out,
                              int32_t out_dtype, void* ws, size_t ws_bytes, void* stream) {
  muon_status st = check_mxfp4(a);
  if (st == MUON_OK) st = check_mxfp4(b);
  if (st != MUON_OK) return st;
  if (!out) return MUON_ERR_NULL;
  const MxGemmShape s{a->count > b->count ? a->count : b->count, a->rows, b->rows, a->cols};
  if (a->cols != b->cols || (a->count != s.count && a->count != 1) || (b->count != s.count && b->count != 1) ||
      !gemm_shape_ok(s))
    return MUON_ERR_SHAPE;
  if (!known_dtype(out_dtype)) return MUON_ERR_DTYPE;
  if (!aligned(out) || !aligned(add) || !aligned(ws)) return MUON_ERR_ALIGN;
  const MxGemmPlan pl = plan_for(s);
  if (!ws || ws_bytes < kHeader + pl.part_bytes) return MUON_ERR_WORKSPACE;
  const Span o{out, static_cast<size_t>(s.count) * s.m * s.n * dtype_size(out_dtype)};
  const Span w{ws, ws_bytes};
  const Span in[4] = {data_span(a), scale_span(a), data_span(b), scale_span(b)};
  for (const Span& i : in)
    if (overlaps(o, i) || overlaps(w, i)) return MUON_ERR_ALIAS;
  if ((add && add != out && overlaps(o, {add, o.n})) || overlaps(o, w) || overlaps(w, {add, o.n}))
    return MUON_ERR_ALIAS;
  int sms = 0, pairs = 0;
  if ((st = lowbit_device(&sms, &pairs)) != MUON_OK) return st;

  MxGemmParams p;
  std::memset(&p, 0, sizeof(p));
  const muon_mxfp4* l = pl.swap ? b : a;
  const muon_mxfp4* r = pl.swap ? a : b;
  if ((st = operand_maps(l, 128, pl.few ? 0 : 1, &p.rows_l, &p.scales_l)) != MUON_OK) return st;
  if ((st = operand_maps(r, pl.few ? pl.nt : 128, pl.few ? 0 : 2, &p.rows_r, &p.scales_r)) != MUON_OK) return st;
  // results are stored, and addends loaded, by TMA where out's rows start on 16-byte boundaries
  p.tma_out = !pl.few && pl.split == 1 && s.n * dtype_size(out_dtype) % 16 == 0 ? 1 : 0;
  if (p.tma_out) {
    const bool bf16 = out_dtype == MUON_BF16;
    const cuuint64_t d[3] = {static_cast<cuuint64_t>(s.n), static_cast<cuuint64_t>(s.m),
                             static_cast<cuuint64_t>(s.count)};
    const cuuint64_t st2[2] = {static_cast<cuuint64_t>(s.n * dtype_size(out_dtype)),
                               static_cast<cuuint64_t>(s.m * s.n * dtype_size(out_dtype))};
    const cuuint32_t box[3] = {bf16 ? 64u : 32u, 32, 1};   // 128-byte rows
    const CUtensorMapDataType type = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    st = encode_tiled(&p.result, type, 3, out, d, st2, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st == MUON_OK && add) st = encode_tiled(&p.addend, type, 3, add, d, st2, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != MUON_OK) return st;
  }
  p.add = add;
  p.out = out;
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kHeader);
  p.m = static_cast<int>(l->rows);
  p.n = static_cast<int>(r->rows);
  p.count = static_cast<int>(s.count);
  p.share_l = l->count == 1 ? 1 : 0;
  p.share_r = r->count == 1 ? 1 : 0;
  p.tiles_l = static_cast<int>(ceil_div(l->rows, kMxTile));
  p.tiles_r = static_cast<int>(ceil_div(r->rows, kMxTile));
  p.sf_l = static_cast<const uint8_t*>(l->scales);
  p.sf_r = static_cast<const uint8_t*>(r->scales);
  p.sf_groups = static_cast<int>(ceil_div(s.k, kMxTile));
  p.k64 = static_cast<int>(ceil_div(s.k, 64));
  p.kstages = static_cast<int>(ceil_div(s.k, 256));
  p.split = pl.split;
  p.kc = pl.kc;
  p.ring = pl.ring;
  p.tm = pl.tm;
  p.tn = pl.tn;
  p.group = 8;
  if (!pl.few) {
    p.fd_split = make_fastdiv(static_cast<uint32_t>(pl.split));
    p.fd_mat = make_fastdiv(static_cast<uint32_t>(pl.tm) * static_cast<uint32_t>(pl.tn));
    p.fd_band = make_fastdiv(static_cast<uint32_t>(p.group) * static_cast<uint32_t>(pl.tn));
    p.fd_group = make_fastdiv(static_cast<uint32_t>(p.group));
    p.fd_rest = make_fastdiv(static_cast<uint32_t>(pl.tm % p.group));
  }
  p.stride_l = pl.swap ? 1 : s.n;
  p.stride_r = pl.swap ? s.n : 1;
  p.stride_c = s.m * s.n;
  p.status = static_cast<int*>(ws);
  p.wait_limit_ns = static_cast<unsigned long long>(wait_limit_seconds() * 1e9);
  p.fault = fault_mode();
  return launch_mx_gemm(p, pl, out_dtype == MUON_BF16, pairs, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MUON_OK
             : MUON_ERR_CUDA;
}

}  // extern "C"
