// Host side of the four-bit operators: argument checks, tensor maps and launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "fp4_kernels.h"
#include "mlp_handle.h"

using namespace tpmlp;
using namespace tpmlp::host;

namespace {

constexpr long long MAX_DIM = 1ll << 28;

int bad(int code, const char* msg) {
  set_detail_msg(msg);
  return code;
}

int launched(const char* name, cudaError_t e) {
  if (e == cudaSuccess) return TPMLP_OK;
  set_detail(name, e);
  return TPMLP_ERR_CUDA;
}

bool format_ok(int format) { return format == TPFP4_NV || format == TPFP4_MX; }
bool dim_ok(long long n) { return n >= 1 && n <= MAX_DIM; }

bool aligned(const void* p, size_t n) {
  return reinterpret_cast<uintptr_t>(p) % n == 0;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a);
  const uintptr_t pb = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && na > 0 && nb > 0 && pa < pb + nb &&
         pb < pa + na;
}

// Bytes from the first to past the last element of a strided matrix.
size_t extent(long long rows, long long cols, long long stride, size_t es) {
  return rows == 0 ? 0 : static_cast<size_t>((rows - 1) * stride + cols) * es;
}

int dtype_ok(int dtype) {
  return dtype == TPMLP_BF16 || dtype == TPMLP_FP32
             ? TPMLP_OK
             : bad(TPMLP_ERR_ARG, "fp4: dtype must be TPMLP_BF16 or TPMLP_FP32");
}

constexpr int AUTO_SCALE = 1 << 20;   // "g is the matrix's own", as an exponent

// The exponent of g; AUTO_SCALE for 0 (NV).
int scale_exponent(int format, double scale, bool may_be_auto, int* e) {
  if (format == TPFP4_MX) {
    if (scale != 0.0 && scale != 1.0)
      return bad(TPMLP_ERR_ARG, "fp4: MX has no scale of the whole matrix");
    *e = 0;
    return TPMLP_OK;
  }
  if (scale == 0.0 && may_be_auto) {
    *e = AUTO_SCALE;
    return TPMLP_OK;
  }
  int x = 0;
  if (!std::isfinite(scale) || std::frexp(scale, &x) != 0.5 || x - 1 < -126 ||
      x - 1 > 127)
    return bad(TPMLP_ERR_ARG, may_be_auto
                   ? "fp4: scale must be 0 or a power of two from 2^-126 to 2^127"
                   : "fp4: scale must be a power of two from 2^-126 to 2^127");
  *e = x - 1;
  return TPMLP_OK;
}

int packed_ok(const char* what, long long rows, long long cols, int format,
              const void* packed, size_t bytes) {
  if (packed == nullptr) return bad(TPMLP_ERR_ARG, what);
  if (!aligned(packed, 256))
    return bad(TPMLP_ERR_ALIGN, "fp4: a packed matrix must be 256-byte aligned");
  if (bytes < fp4::packed_bytes(rows, cols, format))
    return bad(TPMLP_ERR_WORKSPACE, "fp4: a packed matrix has too few bytes");
  return TPMLP_OK;
}

// Quantise along rows or columns, arguments checked.  both (nullable, with
// transpose): along the rows too, into it.
int quantize(HandleCore* core, const char* name, long long rows, long long cols,
             bool bf16, const void* x, long long stride, bool transpose,
             int format, int exponent, const void* like, void* packed, float* part,
             cudaStream_t s, void* both = nullptr) {
  const fp4::Packed p = transpose ? fp4::view(packed, cols, rows)
                                  : fp4::view(packed, rows, cols);
  const fp4::Packed rp = both != nullptr ? fp4::view(both, rows, cols) : p;
  auto step = [&](const char* n, auto&& f) {
    return core != nullptr ? run(core, n, s, f) : launched(n, f());
  };
  fp4::Gain g = {exponent, 0, nullptr};
  if (exponent == AUTO_SCALE && like != nullptr) {
    g.like = static_cast<const fp4::Header*>(like);
  } else if (exponent == AUTO_SCALE) {
    TRY(step("fp4_amax", [&] {
      return fp4::launch_amax(bf16, x, stride, rows, cols, p.head, &g.slots, s);
    }));
  }
  return step(name, [&] {
    return transpose
               ? fp4::launch_quantize_columns(bf16, format, x, stride,
                                              static_cast<int>(rows), p, g, part,
                                              both != nullptr ? &rp : nullptr, s)
               : fp4::launch_quantize_rows(bf16, format, x, stride, p, g, s);
  });
}

// Tiles of `inner` bytes or rows of them, one below the other: `rows` rows, boxes
// of `box`.  In 8-byte elements (a box has at most 256 a side); rows past the end
// are filled with zeros.
int tiles_map(CUtensorMap* m, const void* base, size_t inner, size_t rows,
              int box) {
  EncodeTiledFn enc = get_encoder();
  if (enc == nullptr)
    return bad(TPMLP_ERR_CUDA, "cuTensorMapEncodeTiled entry point not available");
  const cuuint64_t dims[2] = {inner / 8, rows};
  const cuuint64_t strides[1] = {inner};
  const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(inner / 8),
                               static_cast<cuuint32_t>(box)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, 2, const_cast<void*>(base), dims,
          strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS
             ? TPMLP_OK
             : bad(TPMLP_ERR_CUDA, "cuTensorMapEncodeTiled failed (fp4 tiles)");
}

int scales_map(CUtensorMap* m, const fp4::Packed& p, int format) {
  return tiles_map(m, p.scales, fp4::tile_bytes(format),
                   fp4::tiles_of(p.rows, p.cols), 1);
}

int codes_map(CUtensorMap* m, const fp4::Packed& p, int box_rows) {
  return tiles_map(m, p.codes, fp4::TILE_COLS / 2,
                   fp4::tiles_of(p.rows, p.cols) * fp4::TILE_ROWS, box_rows);
}

// Rows of A up to which the split kernel is the faster one.  Times in us (NV, one
// product in L2, launches back to back), split against pairs:
//   up to 32 rows (B of 1024 to 20480 rows, K 1024 to 20480): 2.9 to 40 against 4.1
//     to 55;
//   64 rows, K = 4096: 4.9 to 11.8 against 7.0 to 11.9; K = 1024: 4.5 to 8.1 against
//     4.4 to 6.7;
//   128 rows, 7 tiles of 256 x 256 and 16 k-tiles: 6.5 against 8.3; 16 tiles: 9.4
//     against 7.4; 20 tiles and 80 k-tiles: 14.1 against 21.5;
//   more: few tiles with long sums: 20 tiles (256 x 5120) and 80 k-tiles 19.0
//     against 21.4, 32 tiles 24.3 against 21.8; 4 tiles and 16 k-tiles 8.1 against
//     7.3.
bool few(const fp4::ProductArgs& a) {
  const long long tiles = ((a.M + 255ll) / 256) * ((a.N + 255ll) / 256);
  const int ktiles = a.a.ktiles;
  if (a.M <= 32) return true;
  if (a.M <= 64) return ktiles >= 8;
  if (a.M <= 128) return ktiles >= 16 && 2 * tiles <= ktiles;
  return ktiles >= 64 && 4 * tiles <= ktiles;
}

int product(HandleCore* core, const char* name, int format,
            const fp4::ProductArgs& a, int sms, cudaStream_t s) {
  auto step = [&](auto&& f) {
    return core != nullptr ? run(core, name, s, f) : launched(name, f());
  };
  if (a.x != nullptr || few(a))
    return step([&] { return fp4::launch_product_split(format, a, sms, s); });
  CUtensorMap ta, tsa, tb, tsb, to;
  TRY(codes_map(&ta, a.a, 128));
  TRY(codes_map(&tb, a.b, 64));
  TRY(scales_map(&tsa, a.a, format));
  TRY(scales_map(&tsb, a.b, format));
  const size_t es = a.epilogue == fp4::OUT_FP32 ? 4 : 2;
  // (a TMA store ends a row at the next 16-byte boundary, not at the map's last
  // element: rows that end elsewhere would overwrite what lies behind them)
  const bool tma = a.epilogue != fp4::OUT_GELU_FP4 && aligned16(a.out) &&
                   a.ldo * es % 16 == 0 && a.N * es % 16 == 0;
  if (tma) TRY(out_map(&to, a.out, es == 4, a.M, a.N, a.ldo));
  return step([&] {
    return fp4::launch_product_pairs(format, ta, tsa, tb, tsb, tma ? &to : nullptr,
                                     a, sms / 2, s);
  });
}

// x [rows, cols] as the left operand of a product: quantised first, or by the
// product itself where that is a product of very few rows with a given g: one launch
// instead of two.  In us, weights not in L2, launches back to back: 1 x 1024 x 4096
// 3.5 and 5.0, 1 x 5120 x 20480 12.6 and 14.1, 8 (bf16) x 1024 x 4096 4.1 and 5.2, 8 x
// 5120 x 20480 13.7 and 14.4 (in L2: 10.6 and 9.5).  `xq` keeps the quantised rows and
// the status word.
int left_operand(HandleCore* core, const char* name, long long rows,
                 long long cols, bool bf16, const void* x, long long stride,
                 int format, int exponent, void* xq, fp4::ProductArgs* a,
                 cudaStream_t s) {
  a->a = fp4::view(xq, rows, cols);
  a->status = a->a.head->status;
  const int most = bf16 ? fp4::PLAIN_ROWS_BF16 : fp4::PLAIN_ROWS_FP32;
  if (rows <= most && exponent != AUTO_SCALE) {
    a->x = x;
    a->x_bf16 = bf16 ? 1 : 0;
    a->x_stride = stride;
    a->x_exponent = exponent;
    a->dependent = 0;
    return TPMLP_OK;
  }
  a->dependent = 1;
  return quantize(core, name, rows, cols, bf16, x, stride, false, format, exponent,
                  nullptr, xq, nullptr, s);
}

// A column quantisation's sums over 256 rows each, added up.
int finish_colsum(const void* part, float* colsum, long long rows, long long cols,
                  cudaStream_t s) {
  return launched("fp4_colsum",
                  launch_colsum_finalize(static_cast<const float*>(part), colsum,
                                         static_cast<int>((rows + 255) / 256),
                                         static_cast<int>(cols), s));
}

// tp_fp4_quantize's arguments.
int check_quantize(long long rows, long long cols, int dtype, const void* x,
                   long long row_stride, int transpose, int format, double scale,
                   const void* like, const void* packed, size_t packed_bytes,
                   const float* colsum, const void* workspace,
                   size_t workspace_bytes, int* exponent) {
  if (!format_ok(format)) return bad(TPMLP_ERR_ARG, "fp4: unknown format");
  TRY(dtype_ok(dtype));
  if (transpose != 0 && transpose != 1)
    return bad(TPMLP_ERR_ARG, "fp4: transpose must be 0 or 1");
  if (!dim_ok(cols) || rows < transpose || rows > MAX_DIM)
    return bad(TPMLP_ERR_SHAPE, "fp4: rows or cols out of range");
  if (row_stride < cols || row_stride > (1ll << 40))
    return bad(TPMLP_ERR_SHAPE, "fp4: row stride below the columns or too large");
  TRY(scale_exponent(format, scale, true, exponent));
  if (like != nullptr && (format != TPFP4_NV || scale != 0.0))
    return bad(TPMLP_ERR_ARG, "fp4: like is NV's, with scale = 0");
  if (!aligned(like, 256))
    return bad(TPMLP_ERR_ALIGN, "fp4: a packed matrix must be 256-byte aligned");
  const size_t es = dtype == TPMLP_BF16 ? 2 : 4;
  const long long prows = transpose ? cols : rows, pcols = transpose ? rows : cols;
  TRY(packed_ok("fp4: packed is null", prows, pcols, format, packed, packed_bytes));
  if (colsum != nullptr && !transpose)
    return bad(TPMLP_ERR_ARG, "fp4: colsum needs transpose = 1");
  if (rows == 0) return TPMLP_OK;
  if (x == nullptr) return bad(TPMLP_ERR_ARG, "fp4: x is null");
  if (!aligned(x, es) || !aligned(colsum, 4) || !aligned(workspace, 16))
    return bad(TPMLP_ERR_ALIGN, "fp4: x, colsum or workspace off its alignment");
  const size_t nx = extent(rows, cols, row_stride, es);
  const size_t np = fp4::packed_bytes(prows, pcols, format);
  const size_t ns = static_cast<size_t>(cols) * 4;
  const size_t nw = tp_fp4_colsum_workspace_bytes(rows, cols);
  if (overlap(x, nx, packed, np) || overlap(like, fp4::HEADER_BYTES, packed, np))
    return bad(TPMLP_ERR_ARG, "fp4: packed overlaps x or like");
  if (colsum != nullptr) {
    if (workspace == nullptr) return bad(TPMLP_ERR_ARG, "fp4: workspace is null");
    if (workspace_bytes < nw)
      return bad(TPMLP_ERR_WORKSPACE, "fp4: workspace too small for colsum");
    if (overlap(colsum, ns, x, nx) || overlap(colsum, ns, packed, np) ||
        overlap(colsum, ns, workspace, nw) || overlap(workspace, nw, x, nx) ||
        overlap(workspace, nw, packed, np))
      return bad(TPMLP_ERR_ARG, "fp4: colsum or workspace overlaps another buffer");
  }
  // one block a 64-column, 256-row piece (columns, up to a multiple of 256) or 16
  // rows x 256 (rows)
  const long long blocks = transpose
                               ? (cols + 255) / 256 * 4 * ((rows + 255) / 256)
                               : (rows + 15) / 16 * ((cols + 255) / 256);
  if (blocks > INT_MAX) return bad(TPMLP_ERR_SHAPE, "fp4: matrix too large");
  return TPMLP_OK;
}

// tp_fp4_matmul's arguments.
int check_matmul(long long T, long long N, long long K, int format, const void* A,
                 size_t a_bytes, const void* B, size_t b_bytes, const float* bias,
                 int dtype, const void* C, long long ldc, const void* status) {
  if (!format_ok(format)) return bad(TPMLP_ERR_ARG, "fp4: unknown format");
  TRY(dtype_ok(dtype));
  if (T < 0 || T > MAX_DIM || !dim_ok(N) || !dim_ok(K))
    return bad(TPMLP_ERR_SHAPE, "fp4: T, N or K out of range");
  if (ldc < N || ldc > (1ll << 40))
    return bad(TPMLP_ERR_SHAPE, "fp4: ldc below N or too large");
  TRY(packed_ok("fp4: A is null", T, K, format, A, a_bytes));
  TRY(packed_ok("fp4: B is null", N, K, format, B, b_bytes));
  if (T == 0) return TPMLP_OK;
  if (C == nullptr) return bad(TPMLP_ERR_ARG, "fp4: C is null");
  const size_t es = dtype == TPMLP_BF16 ? 2 : 4;
  if (!aligned(C, es) || !aligned(bias, 4) || !aligned(status, 16))
    return bad(TPMLP_ERR_ALIGN, "fp4: C, bias or status off its alignment");
  const size_t nc = extent(T, N, ldc, es);
  if (overlap(status, 16, C, nc) || overlap(status, 16, bias, size_t(N) * 4) ||
      overlap(status, 16, A, fp4::packed_bytes(T, K, format)) ||
      overlap(status, 16, B, fp4::packed_bytes(N, K, format)))
    return bad(TPMLP_ERR_ARG, "fp4: status overlaps another buffer");
  if (overlap(C, nc, A, fp4::packed_bytes(T, K, format)) ||
      overlap(C, nc, B, fp4::packed_bytes(N, K, format)) ||
      overlap(C, nc, bias, static_cast<size_t>(N) * 4))
    return bad(TPMLP_ERR_ARG, "fp4: C overlaps an input");
  // rows of all tiles and output tiles are counted in 32 bits
  const long long ktiles = (K + 255) / 256;
  if ((std::max(T, N) + 127) / 128 * ktiles > INT_MAX / 256 ||
      (T + 127) / 128 * ((N + 127) / 128) > INT_MAX / 16)
    return bad(TPMLP_ERR_SHAPE, "fp4: product too large");
  return TPMLP_OK;
}

// A product's fields but its left operand's, arguments checked.
fp4::ProductArgs matmul_args(long long T, long long N, long long K, const void* B,
                             const float* bias, int dtype, void* C,
                             long long ldc) {
  fp4::ProductArgs a = {};
  a.b = fp4::view(B, N, K);
  a.M = static_cast<int>(T);
  a.N = static_cast<int>(N);
  a.epilogue = dtype == TPMLP_BF16 ? fp4::OUT_BF16 : fp4::OUT_FP32;
  a.out = C;
  a.ldo = ldc;
  a.bias = bias;
  a.budget_ns = HandleCore().budget_ns;
  return a;
}

// ----------------------------------------------------------- MLP block --

struct MlpPack {
  size_t a = 0, a_bytes = 0, b = 0, b_bytes = 0, total = 0;
};
// A^T [f, h] | B^T [h, f]
MlpPack mlp_pack(const tp_mlp_config& c, int format) {
  MlpPack p;
  p.a_bytes = fp4::up256(fp4::packed_bytes(c.ffn, c.hidden, format));
  p.b_bytes = fp4::up256(fp4::packed_bytes(c.hidden, c.ffn, format));
  p.b = p.a_bytes;
  p.total = p.a_bytes + p.b_bytes;
  return p;
}

struct MlpLayout {
  size_t xq = 0, yq = 0, xn = 0, mean = 0, rstd = 0, total = 0;
};
// Xq [T, h], whose header's status word is the call's (but for
// tp_fp4_mlp_set_status) | Yq [T, f] | [Xn bf16,
// mean, rstd]
MlpLayout mlp_layout(const tp_mlp_config& c, int tokens, int format) {
  MlpLayout l;
  const size_t T = static_cast<size_t>(tokens);
  l.yq = fp4::up256(fp4::packed_bytes(tokens, c.hidden, format));
  l.xn = l.yq + fp4::up256(fp4::packed_bytes(tokens, c.ffn, format));
  l.mean = l.xn + (c.use_layernorm ? fp4::up256(T * c.hidden * 2) : 0);
  l.rstd = l.mean + (c.use_layernorm ? fp4::up256(T * 4) : 0);
  l.total = l.rstd + (c.use_layernorm ? fp4::up256(T * 4) : 0);
  return l;
}

int mlp_config_ok(const tp_mlp_config& c, int format) {
  if (!format_ok(format)) return bad(TPMLP_ERR_ARG, "fp4: unknown format");
  if (c.dtype != TPMLP_BF16 || c.dropout_p > 0.f)
    return bad(TPMLP_ERR_ARG, "fp4: the block must be bf16 without dropout");
  return TPMLP_OK;
}

}  // namespace

extern "C" {

size_t tp_fp4_bytes(long long rows, long long cols, int format) {
  if (!format_ok(format) || !dim_ok(cols) || rows < 0 || rows > MAX_DIM) return 0;
  return fp4::packed_bytes(rows, cols, format);
}

long long tp_fp4_offset(long long rows, long long cols, int format, int which) {
  if (tp_fp4_bytes(rows, cols, format) == 0) return -1;
  if (which == TPFP4_CODES) return static_cast<long long>(fp4::HEADER_BYTES);
  if (which == TPFP4_SCALES)
    return static_cast<long long>(fp4::scales_offset(rows, cols));
  return -1;
}

size_t tp_fp4_colsum_workspace_bytes(long long rows, long long cols) {
  if (!dim_ok(rows) || !dim_ok(cols)) return 0;
  return static_cast<size_t>((rows + fp4::TILE_COLS - 1) / fp4::TILE_COLS) * cols *
         4;
}

int tp_fp4_quantize(long long rows, long long cols, int dtype, const void* x,
                    long long row_stride, int transpose, int format,
                    double scale, const void* like, void* packed,
                    size_t packed_bytes, float* colsum, void* workspace, size_t workspace_bytes,
                    void* stream) {
  int exponent = 0;
  TRY(check_quantize(rows, cols, dtype, x, row_stride, transpose, format, scale,
                     like, packed, packed_bytes, colsum, workspace, workspace_bytes,
                     &exponent));
  if (rows == 0) return TPMLP_OK;
  int sms = 0;
  TRY(check_device(&sms));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  TRY(quantize(nullptr, "fp4_quantize", rows, cols, dtype == TPMLP_BF16, x,
               row_stride, transpose != 0, format, exponent, like, packed,
               colsum != nullptr ? static_cast<float*>(workspace) : nullptr, s));
  return colsum == nullptr ? TPMLP_OK
                           : finish_colsum(workspace, colsum, rows, cols, s);
}

int tp_fp4_quantize_both(long long rows, long long cols, int dtype, const void* x,
                         long long row_stride, int format, double scale,
                         void* packed, size_t packed_bytes, void* packed_t,
                         size_t packed_t_bytes, float* colsum, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int exponent = 0;
  TRY(check_quantize(rows, cols, dtype, x, row_stride, 1, format, scale, nullptr,
                     packed_t, packed_t_bytes, colsum, workspace, workspace_bytes,
                     &exponent));
  TRY(check_quantize(rows, cols, dtype, x, row_stride, 0, format, scale, nullptr,
                     packed, packed_bytes, nullptr, nullptr, 0, &exponent));
  const size_t np = fp4::packed_bytes(rows, cols, format);
  if (overlap(packed, np, packed_t, fp4::packed_bytes(cols, rows, format)) ||
      overlap(packed, np, colsum, static_cast<size_t>(cols) * 4) ||
      (colsum != nullptr &&
       overlap(packed, np, workspace, tp_fp4_colsum_workspace_bytes(rows, cols))))
    return bad(TPMLP_ERR_ARG, "fp4: packed overlaps another output");
  int sms = 0;
  TRY(check_device(&sms));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  TRY(quantize(nullptr, "fp4_quantize_both", rows, cols, dtype == TPMLP_BF16, x,
               row_stride, true, format, exponent, nullptr, packed_t,
               colsum != nullptr ? static_cast<float*>(workspace) : nullptr, s,
               packed));
  return colsum == nullptr ? TPMLP_OK
                           : finish_colsum(workspace, colsum, rows, cols, s);
}

int tp_fp4_dequantize(long long rows, long long cols, int format,
                      const void* packed, size_t packed_bytes, int dtype,
                      void* out, long long row_stride, void* stream) {
  if (!format_ok(format)) return bad(TPMLP_ERR_ARG, "fp4: unknown format");
  TRY(dtype_ok(dtype));
  if (!dim_ok(cols) || rows < 0 || rows > MAX_DIM)
    return bad(TPMLP_ERR_SHAPE, "fp4: rows or cols out of range");
  if (row_stride < cols || row_stride > (1ll << 40))
    return bad(TPMLP_ERR_SHAPE, "fp4: row stride below the columns or too large");
  TRY(packed_ok("fp4: packed is null", rows, cols, format, packed, packed_bytes));
  if (rows == 0) return TPMLP_OK;
  if (out == nullptr) return bad(TPMLP_ERR_ARG, "fp4: out is null");
  const size_t es = dtype == TPMLP_BF16 ? 2 : 4;
  if (!aligned(out, es)) return bad(TPMLP_ERR_ALIGN, "fp4: out off its alignment");
  if (overlap(out, extent(rows, cols, row_stride, es), packed,
              fp4::packed_bytes(rows, cols, format)))
    return bad(TPMLP_ERR_ARG, "fp4: out overlaps packed");
  if ((rows + 15) / 16 * ((cols + 255) / 256) > INT_MAX)
    return bad(TPMLP_ERR_SHAPE, "fp4: matrix too large");
  int sms = 0;
  TRY(check_device(&sms));
  return launched("fp4_dequantize",
                  fp4::launch_dequantize(fp4::view(packed, rows, cols), format,
                                         dtype == TPMLP_BF16, out, row_stride,
                                         static_cast<cudaStream_t>(stream)));
}

int tp_fp4_matmul(long long T, long long N, long long K, int format,
                  const void* A, size_t a_bytes, const void* B, size_t b_bytes,
                  const float* bias, int dtype, void* C, long long ldc,
                  void* status, void* stream) {
  TRY(check_matmul(T, N, K, format, A, a_bytes, B, b_bytes, bias, dtype, C, ldc,
                   status));
  if (T == 0) return TPMLP_OK;
  int sms = 0;
  TRY(check_device(&sms));
  fp4::ProductArgs a = matmul_args(T, N, K, B, bias, dtype, C, ldc);
  a.a = fp4::view(A, T, K);
  a.status = status != nullptr ? static_cast<int*>(status) : a.a.head->status;
  return product(nullptr, "fp4_matmul", format, a, sms,
                 static_cast<cudaStream_t>(stream));
}

int tp_fp4_linear(long long T, long long N, long long K, int x_dtype,
                  const void* x, long long x_stride, int format, double x_scale,
                  void* xq, size_t xq_bytes, const void* W, size_t w_bytes,
                  const float* bias, int dtype, void* C, long long ldc,
                  void* status, void* stream) {
  int exponent = 0;
  TRY(check_quantize(T, K, x_dtype, x, x_stride, 0, format, x_scale, nullptr,
                     xq, xq_bytes, nullptr, nullptr, 0, &exponent));
  TRY(check_matmul(T, N, K, format, xq, xq_bytes, W, w_bytes, bias, dtype, C, ldc,
                   status));
  if (T == 0) return TPMLP_OK;
  const size_t nx = extent(T, K, x_stride, x_dtype == TPMLP_BF16 ? 2 : 4);
  const size_t nq = fp4::packed_bytes(T, K, format);
  if (overlap(xq, nq, W, fp4::packed_bytes(N, K, format)) ||
      overlap(xq, nq, bias, static_cast<size_t>(N) * 4) ||
      overlap(C, extent(T, N, ldc, dtype == TPMLP_BF16 ? 2 : 4), x, nx))
    return bad(TPMLP_ERR_ARG, "fp4: xq or C overlaps an input");
  int sms = 0;
  TRY(check_device(&sms));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  fp4::ProductArgs a = matmul_args(T, N, K, W, bias, dtype, C, ldc);
  TRY(left_operand(nullptr, "fp4_quantize", T, K, x_dtype == TPMLP_BF16, x,
                   x_stride, format, exponent, xq, &a, s));
  if (status != nullptr) a.status = static_cast<int*>(status);
  return product(nullptr, "fp4_matmul", format, a, sms, s);
}

int tp_fp4_check(void* status, void* stream) {
  if (status == nullptr) return TPMLP_ERR_ARG;
  return check_status(status, static_cast<cudaStream_t>(stream));
}

size_t tp_fp4_mlp_weights_bytes(const tp_mlp_handle* H, int format) {
  if (H == nullptr || mlp_config_ok(H->cfg, format) != TPMLP_OK) return 0;
  return mlp_pack(H->cfg, format).total;
}

int tp_fp4_mlp_pack_weights(tp_mlp_handle* H, int format, const void* A,
                            const void* B, void* packed, size_t packed_bytes,
                            void* stream) {
  if (H == nullptr) return TPMLP_ERR_ARG;
  const tp_mlp_config& c = H->cfg;
  TRY(mlp_config_ok(c, format));
  if (!A || !B || !packed) return bad(TPMLP_ERR_ARG, "fp4: null pointer");
  if (!aligned16(A) || !aligned16(B) || !aligned(packed, 256))
    return bad(TPMLP_ERR_ALIGN, "fp4: A, B or packed off its alignment");
  const MlpPack p = mlp_pack(c, format);
  if (packed_bytes < p.total)
    return bad(TPMLP_ERR_WORKSPACE, "fp4: packed weights need more bytes");
  const size_t n = static_cast<size_t>(c.hidden) * c.ffn * 2;
  if (overlap(packed, p.total, A, n) || overlap(packed, p.total, B, n))
    return bad(TPMLP_ERR_ARG, "fp4: packed overlaps A or B");
  int sms = 0;
  TRY(check_device(&sms));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* pk = static_cast<char*>(packed);
  const int e = format == TPFP4_NV ? AUTO_SCALE : 0;
  TRY(quantize(&H->core, "fp4_quantize_weights", c.hidden, c.ffn, true, A, c.ffn,
               true, format, e, nullptr, pk + p.a, nullptr, s));
  return quantize(&H->core, "fp4_quantize_weights", c.ffn, c.hidden, true, B,
                  c.hidden, true, format, e, nullptr, pk + p.b, nullptr, s);
}

size_t tp_fp4_mlp_workspace_bytes(const tp_mlp_handle* H, int tokens,
                                  int format) {
  if (H == nullptr || tokens < 0 || mlp_config_ok(H->cfg, format) != TPMLP_OK)
    return 0;
  return mlp_layout(H->cfg, tokens, format).total;
}

int tp_fp4_mlp_set_status(tp_mlp_handle* H, void* status) {
  if (H == nullptr) return TPMLP_ERR_ARG;
  if (!aligned16(status))
    return bad(TPMLP_ERR_ALIGN, "fp4: status must be 16-byte aligned");
  H->fp4_status = static_cast<int*>(status);
  return TPMLP_OK;
}

int tp_fp4_mlp_forward(tp_mlp_handle* H, int tokens, int format, const void* X,
                       const void* packed, const float* bias1,
                       const float* bias2, const float* ln_gamma,
                       const float* ln_beta, double x_scale, double y_scale,
                       void* Z, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (H == nullptr) return TPMLP_ERR_ARG;
  const tp_mlp_config& c = H->cfg;
  TRY(mlp_config_ok(c, format));
  int xe = 0, ye = 0;
  TRY(scale_exponent(format, x_scale, false, &xe));
  TRY(scale_exponent(format, y_scale, false, &ye));
  if (tokens < 0 || tokens > c.max_tokens) return TPMLP_ERR_SHAPE;
  if (!packed || !workspace || (tokens > 0 && (!X || !Z))) return TPMLP_ERR_ARG;
  if (c.use_layernorm && (!ln_gamma || !ln_beta)) return TPMLP_ERR_ARG;
  const void* ptrs[] = {X, Z, bias1, bias2, ln_gamma, ln_beta};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return TPMLP_ERR_ALIGN;
  if (!aligned(packed, 256) || !aligned(workspace, 256))
    return bad(TPMLP_ERR_ALIGN, "fp4: packed and workspace: 256-byte alignment");
  const MlpLayout L = mlp_layout(c, tokens, format);
  if (workspace_bytes < L.total) return TPMLP_ERR_WORKSPACE;
  const MlpPack P = mlp_pack(c, format);
  const size_t nx = static_cast<size_t>(tokens) * c.hidden * 2;
  const size_t nh = static_cast<size_t>(c.hidden) * 4;
  const struct { const void* p; size_t n; } inputs[] = {
      {X, nx}, {packed, P.total}, {bias1, static_cast<size_t>(c.ffn) * 4},
      {bias2, nh}, {ln_gamma, nh}, {ln_beta, nh}};
  int* const status = H->fp4_status;   // (null: the workspace's)
  if (overlap(status, 16, Z, nx) || overlap(status, 16, workspace, L.total))
    return bad(TPMLP_ERR_ARG, "fp4: Z or workspace overlaps the status");
  for (const auto& in : inputs)
    if (overlap(Z, nx, in.p, in.n) || overlap(workspace, L.total, in.p, in.n))
      return bad(TPMLP_ERR_ARG, "fp4: Z or workspace overlaps an input");
  if (overlap(Z, nx, workspace, L.total))
    return bad(TPMLP_ERR_ARG, "fp4: Z overlaps the workspace");
  int sms = 0;
  TRY(check_device(&sms));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const char* pk = static_cast<const char*>(packed);
  if (tokens == 0)
    return launched("cudaMemsetAsync(status)", cudaMemsetAsync(ws, 0, 16, s));
  const int h = c.hidden, f = c.ffn;
  const void* Xop = X;
  if (c.use_layernorm) {
    TRY(run(&H->core, "layernorm_fwd", s, [&] {
      return launch_ln_fwd(true, X, ln_gamma, ln_beta, ws + L.xn,
                           reinterpret_cast<float*>(ws + L.mean),
                           reinterpret_cast<float*>(ws + L.rstd), tokens, h,
                           c.ln_eps, s);
    }));
    Xop = ws + L.xn;
  }
  fp4::ProductArgs a = {};
  TRY(left_operand(&H->core, "fp4_quantize_x", tokens, h, true, Xop, h, format, xe,
                   ws + L.xq, &a, s));
  if (status != nullptr) a.status = status;
  a.b = fp4::view(pk + P.a, f, h);
  a.M = tokens;
  a.N = f;
  a.epilogue = fp4::OUT_GELU_FP4;
  a.bias = bias1;
  a.y = fp4::view(ws + L.yq, tokens, f);
  a.y_exponent = ye;
  a.gelu_mode = c.gelu_mode;
  a.budget_ns = H->core.budget_ns;
  TRY(product(&H->core, "gemm1_gelu_fp4", format, a, sms, s));
  a.a = a.y;
  a.x = nullptr;
  a.dependent = 1;
  a.b = fp4::view(pk + P.b, h, f);
  a.N = h;
  a.epilogue = fp4::OUT_BF16;
  a.out = Z;
  a.ldo = h;
  a.bias = bias2;
  if (c.use_residual) {
    a.residual = X;
    a.ldr = h;
  }
  return product(&H->core, "gemm2_fp4", format, a, sms, s);
}

}  // extern "C"
