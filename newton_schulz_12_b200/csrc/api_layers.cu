// C ABI of the operators around a Muon-trained linear layer: layer norm with
// its gradient, and 4-bit microscaled quantisation and products.  Arguments
// are checked on the host before anything is enqueued; no call takes a workspace
// (a product has its stream's status word, which the first one allocates).
#include <algorithm>
#include <cmath>
#include <iterator>
#include <new>
#include <vector>

#include "internal.h"
#include "muon.h"

using namespace muon;

namespace {

constexpr long long kMaxSide = 1ll << 30;  // rows and columns: tensor-copy coordinates are 32-bit

#define TRY(expr)                 \
  do {                            \
    const int r_ = (expr);        \
    if (r_ != MUON_OK) return r_; \
  } while (0)

#define TRY_CUDA(call)                                                                              \
  do {                                                                                              \
    const cudaError_t e_ = (call);                                                                  \
    if (e_ != cudaSuccess)                                                                          \
      return host::set_error(MUON_ERR_CUDA, "%s failed: %s", #call, cudaGetErrorString(e_));        \
  } while (0)

long long element_size(int dtype) { return dtype == MUON_FP32 ? 4 : 2; }

int check_dtype(int dtype) {
  if (dtype != MUON_BF16 && dtype != MUON_FP32 && dtype != MUON_FP16)
    return host::set_error(MUON_ERR_ARG, "dtype %d unknown", dtype);
  return MUON_OK;
}

int check_pointer(const void* p, long long align, const char* what) {
  if (!p) return host::set_error(MUON_ERR_ARG, "%s is NULL", what);
  if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(align))
    return host::set_error(MUON_ERR_ARG, "%s is not %lld-byte aligned", what, align);
  return MUON_OK;
}

int check_side(long long v, long long lo, const char* what) {
  if (v < lo || v > kMaxSide)
    return host::set_error(MUON_ERR_SHAPE, "%s %lld out of range %lld..%lld", what, v, lo, kMaxSide);
  return MUON_OK;
}

// A row-major matrix's stride in elements: at least its columns where rows follow one another.
int check_stride(long long rows, long long cols, long long ld, const char* what) {
  if (rows > 1 && (ld < cols || ld > (1ll << 44) / rows))
    return host::set_error(MUON_ERR_SHAPE, "row stride %lld of %s is below its %lld columns or too large", ld, what, cols);
  return MUON_OK;
}

long long extent(long long rows, long long cols, long long ld) { return rows ? (rows - 1) * ld + cols : 0; }

// Memory that a call reads or writes: a matrix from its first to its last element.
struct Span {
  uintptr_t at, end;
  bool out;
  const char* what;
};

Span reads(const void* p, long long bytes, const char* what) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return {at, p && bytes > 0 ? at + static_cast<uintptr_t>(bytes) : at, false, what};
}

Span writes(const void* p, long long bytes, const char* what) {
  Span s = reads(p, bytes, what);
  s.out = true;
  return s;
}

// What is written shares no byte with anything else of the call.
int check_apart(Span* spans, size_t count) {
  std::sort(spans, spans + count, [](const Span& a, const Span& b) { return a.at < b.at; });
  const Span *any = nullptr, *out = nullptr;  // those that reach farthest so far, of all and of the written ones
  for (size_t i = 0; i < count; ++i) {
    const Span& s = spans[i];
    if (s.end == s.at) continue;
    const Span* other = s.out ? any : out;
    if (other && other->end > s.at)
      return host::set_error(MUON_ERR_ARG, "%s must not overlap %s", s.out ? s.what : other->what, s.out ? other->what : s.what);
    if (!any || s.end > any->end) any = &s;
    if (s.out && (!out || s.end > out->end)) out = &s;
  }
  return MUON_OK;
}

long long scale_bytes(long long rows, long long cols) {
  return ((rows + mx::kTile - 1) / mx::kTile) * ((cols + mx::kTile - 1) / mx::kTile) * 512;
}

int check_params(const void* weight, const void* bias, int dtype, int param_dtype) {
  TRY(check_dtype(dtype));
  TRY(check_dtype(param_dtype));
  if (param_dtype != MUON_FP32 && param_dtype != dtype)
    return host::set_error(MUON_ERR_ARG, "param_dtype %d must be fp32 or the type of x (%d)", param_dtype, dtype);
  if (weight) TRY(check_pointer(weight, element_size(param_dtype), "weight"));
  if (bias) TRY(check_pointer(bias, element_size(param_dtype), "bias"));
  return MUON_OK;
}

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

int forward_impl(long long rows, long long cols, const void* x, long long ldx, int dtype, const void* weight, const void* bias,
                 int param_dtype, float eps, void* y, long long ldy, float* mean, float* rstd, void* stream) {
  TRY(check_side(rows, 0, "rows"));
  TRY(check_side(cols, 1, "cols"));
  TRY(check_params(weight, bias, dtype, param_dtype));
  if (!std::isfinite(eps) || eps < 0.f) return host::set_error(MUON_ERR_ARG, "eps must be finite and not negative");
  TRY(check_stride(rows, cols, ldx, "x"));
  TRY(check_stride(rows, cols, ldy, "y"));
  if (rows == 0) return MUON_OK;
  const long long e = element_size(dtype);
  TRY(check_pointer(x, e, "x"));
  TRY(check_pointer(y, e, "y"));
  TRY(check_pointer(mean, 4, "mean"));
  TRY(check_pointer(rstd, 4, "rstd"));
  const long long pe = element_size(param_dtype) * cols;
  Span spans[] = {writes(y, extent(rows, cols, ldy) * e, "y"), writes(mean, rows * 4, "mean"), writes(rstd, rows * 4, "rstd"),
                  reads(x, extent(rows, cols, ldx) * e, "x"),  reads(weight, pe, "weight"),    reads(bias, pe, "bias")};
  TRY(check_apart(spans, std::size(spans)));
  int sms = 0;
  TRY(host::device_sms(&sms));
  ln::FwdParams p{};
  p.rows = rows;
  p.cols = static_cast<int>(cols);
  p.x = x;
  p.ldx = ldx;
  p.weight = weight;
  p.bias = bias;
  p.eps = eps;
  p.y = y;
  p.ldy = ldy;
  p.mean = mean;
  p.rstd = rstd;
  host::Timed timed(MUON_KERNEL_LAYER_NORM, as_stream(stream));
  TRY_CUDA(ln::launch_forward(p, dtype, param_dtype, sms, as_stream(stream)));
  return MUON_OK;
}

long long backward_scratch(long long rows, long long cols, int sms) {
  return static_cast<long long>(ln::partial_count(rows, static_cast<int>(cols), sms)) * 2 * cols * 4;
}

int backward_impl(long long rows, long long cols, const void* dy, long long lddy, const void* x, long long ldx, int dtype,
                  const void* weight, int param_dtype, const float* mean, const float* rstd, void* dx, long long lddx,
                  void* dweight, void* dbias, void* scratch, long long scratch_bytes, void* stream) {
  TRY(check_side(rows, 0, "rows"));
  TRY(check_side(cols, 1, "cols"));
  TRY(check_params(weight, nullptr, dtype, param_dtype));
  if (dweight) TRY(check_pointer(dweight, element_size(param_dtype), "dweight"));
  if (dbias) TRY(check_pointer(dbias, element_size(param_dtype), "dbias"));
  TRY(check_stride(rows, cols, lddy, "dy"));
  TRY(check_stride(rows, cols, ldx, "x"));
  TRY(check_stride(rows, cols, lddx, "dx"));
  const long long e = element_size(dtype);
  if (rows > 0) {
    TRY(check_pointer(dy, e, "dy"));
    TRY(check_pointer(x, e, "x"));
    TRY(check_pointer(mean, 4, "mean"));
    TRY(check_pointer(rstd, 4, "rstd"));
    TRY(check_pointer(dx, e, "dx"));
  }
  const long long pe = element_size(param_dtype) * cols;
  Span spans[9] = {writes(dx, extent(rows, cols, lddx) * e, "dx"), writes(dweight, pe, "dweight"),
                   writes(dbias, pe, "dbias"),                    reads(dy, extent(rows, cols, lddy) * e, "dy"),
                   reads(x, extent(rows, cols, ldx) * e, "x"),    reads(weight, pe, "weight"),
                   reads(mean, rows * 4, "mean"),                 reads(rstd, rows * 4, "rstd")};
  TRY(check_apart(spans, 8));
  if (rows == 0 && !dweight && !dbias) return MUON_OK;
  int sms = 0;
  TRY(host::device_sms(&sms));
  const bool sums = dweight || dbias;
  if (sums && rows > 0) {
    const long long need = backward_scratch(rows, cols, sms);
    if (scratch_bytes < need)
      return host::set_error(MUON_ERR_ARG, "scratch of %lld bytes: %lld are needed (muon_layer_norm_scratch_bytes)", scratch_bytes, need);
    TRY(check_pointer(scratch, 16, "scratch"));
    spans[8] = writes(scratch, need, "scratch");
    TRY(check_apart(spans, 9));
  }
  ln::BwdParams p{};
  p.rows = rows;
  p.cols = static_cast<int>(cols);
  p.dy = dy;
  p.lddy = lddy;
  p.x = x;
  p.ldx = ldx;
  p.weight = weight;
  p.mean = mean;
  p.rstd = rstd;
  p.dx = dx;
  p.lddx = lddx;
  p.dweight = dweight;
  p.dbias = dbias;
  p.partials = static_cast<float*>(scratch);
  p.parts = sums ? ln::partial_count(rows, p.cols, sms) : 0;
  host::Timed timed(MUON_KERNEL_LAYER_NORM_GRAD, as_stream(stream));
  TRY_CUDA(ln::launch_backward(p, dtype, param_dtype, sms, as_stream(stream)));
  return MUON_OK;
}

int tile_count(long long v) { return static_cast<int>((v + mx::kTile - 1) / mx::kTile); }

int check_matrix(const int64_t* shapes, int i) {
  const long long r = shapes[2 * i], c = shapes[2 * i + 1];
  if (r < 0 || c < 0 || r > kMaxSide || c > kMaxSide)
    return host::set_error(MUON_ERR_SHAPE, "matrix %d: bad shape %lld x %lld", i, r, c);
  return MUON_OK;
}

int quantize_impl(int count, const void* const* x, const int64_t* shapes, const int64_t* strides, int dtype,
                  void* const* row_data, void* const* row_scales, void* const* col_data, void* const* col_scales,
                  void* stream) {
  if (count < 0) return host::set_error(MUON_ERR_ARG, "count %d < 0", count);
  TRY(check_dtype(dtype));
  if ((row_data == nullptr) != (row_scales == nullptr) || (col_data == nullptr) != (col_scales == nullptr))
    return host::set_error(MUON_ERR_ARG, "data and scales of a form come together");
  if (!row_data && !col_data) return host::set_error(MUON_ERR_ARG, "no form is wanted");
  if (count == 0) return MUON_OK;
  if (!x || !shapes) return host::set_error(MUON_ERR_ARG, "x and shapes must be non-NULL");
  const long long e = element_size(dtype);
  std::vector<Span> spans;  // all matrices' together: they may be written at the same time
  spans.reserve(static_cast<size_t>(count) * 5);
  for (int i = 0; i < count; ++i) {
    TRY(check_matrix(shapes, i));
    const long long r = shapes[2 * i], c = shapes[2 * i + 1];
    if (r == 0 || c == 0) continue;
    TRY(check_stride(r, c, strides ? strides[i] : c, "x"));
    TRY(check_pointer(x[i], e, "x"));
    if (row_data) TRY(check_pointer(row_data[i], 16, "row_data"));
    if (row_data) TRY(check_pointer(row_scales[i], 16, "row_scales"));
    if (col_data) TRY(check_pointer(col_data[i], 16, "col_data"));
    if (col_data) TRY(check_pointer(col_scales[i], 16, "col_scales"));
    if (static_cast<long long>(tile_count(r)) * tile_count(c) >= (1ll << 31))
      return host::set_error(MUON_ERR_SHAPE, "matrix %d: %lld x %lld has too many tiles", i, r, c);
    spans.push_back(reads(x[i], extent(r, c, strides ? strides[i] : c) * e, "x"));
    if (row_data) {
      spans.push_back(writes(row_data[i], r * mx::data_stride(c), "row_data"));
      spans.push_back(writes(row_scales[i], scale_bytes(r, c), "row_scales"));
    }
    if (col_data) {
      spans.push_back(writes(col_data[i], c * mx::data_stride(r), "col_data"));
      spans.push_back(writes(col_scales[i], scale_bytes(r, c), "col_scales"));
    }
  }
  TRY(check_apart(spans.data(), spans.size()));
  int sms = 0;
  TRY(host::device_sms(&sms));
  cudaStream_t s = as_stream(stream);
  int i = 0;
  while (i < count) {  // as many matrices a launch as its table holds
    mx::QuantParams p{};
    long long tiles = 0;
    for (; i < count && p.nmat < mx::kMaxMats; ++i) {
      const long long r = shapes[2 * i], c = shapes[2 * i + 1];
      if (r == 0 || c == 0) continue;
      const long long more = static_cast<long long>(tile_count(r)) * tile_count(c);
      if (tiles + more >= (1ll << 31)) break;
      mx::QuantMat& M = p.mat[p.nmat++];
      M.x = x[i];
      M.ldx = strides ? strides[i] : c;
      M.rows = static_cast<int>(r);
      M.cols = static_cast<int>(c);
      M.tiles_c = tile_count(c);
      M.tile_begin = static_cast<int>(tiles);
      M.row_data = row_data ? row_data[i] : nullptr;
      M.row_scales = row_data ? row_scales[i] : nullptr;
      M.col_data = col_data ? col_data[i] : nullptr;
      M.col_scales = col_data ? col_scales[i] : nullptr;
      tiles += more;
    }
    p.ntiles = static_cast<int>(tiles);
    if (p.ntiles == 0) continue;
    host::Timed timed(MUON_KERNEL_MX_QUANTIZE, s);
    TRY_CUDA(mx::launch_quantize(p, dtype, s));
  }
  return MUON_OK;
}

int dequantize_impl(int count, const void* const* data, const void* const* scales, const int64_t* shapes, void* const* y,
                    int dtype, void* stream) {
  if (count < 0) return host::set_error(MUON_ERR_ARG, "count %d < 0", count);
  TRY(check_dtype(dtype));
  if (count == 0) return MUON_OK;
  if (!data || !scales || !shapes || !y) return host::set_error(MUON_ERR_ARG, "data, scales, shapes and y must be non-NULL");
  std::vector<Span> spans;
  spans.reserve(static_cast<size_t>(count) * 3);
  for (int i = 0; i < count; ++i) {
    TRY(check_matrix(shapes, i));
    const long long r = shapes[2 * i], c = shapes[2 * i + 1];
    if (r == 0 || c == 0) continue;
    TRY(check_pointer(data[i], 16, "data"));
    TRY(check_pointer(scales[i], 16, "scales"));
    TRY(check_pointer(y[i], element_size(dtype), "y"));
    if (static_cast<long long>(tile_count(r)) * tile_count(c) >= (1ll << 31))
      return host::set_error(MUON_ERR_SHAPE, "matrix %d: %lld x %lld has too many tiles", i, r, c);
    spans.push_back(reads(data[i], r * mx::data_stride(c), "data"));
    spans.push_back(reads(scales[i], scale_bytes(r, c), "scales"));
    spans.push_back(writes(y[i], r * c * element_size(dtype), "y"));
  }
  TRY(check_apart(spans.data(), spans.size()));
  int sms = 0;
  TRY(host::device_sms(&sms));
  cudaStream_t s = as_stream(stream);
  int i = 0;
  while (i < count) {
    mx::DequantParams p{};
    long long tiles = 0;
    for (; i < count && p.nmat < mx::kMaxMats; ++i) {
      const long long r = shapes[2 * i], c = shapes[2 * i + 1];
      if (r == 0 || c == 0) continue;
      const long long more = static_cast<long long>(tile_count(r)) * tile_count(c);
      if (tiles + more >= (1ll << 31)) break;
      mx::DequantMat& M = p.mat[p.nmat++];
      M.data = data[i];
      M.scales = scales[i];
      M.y = y[i];
      M.rows = static_cast<int>(r);
      M.cols = static_cast<int>(c);
      M.tiles_c = tile_count(c);
      M.tile_begin = static_cast<int>(tiles);
      tiles += more;
    }
    p.ntiles = static_cast<int>(tiles);
    if (p.ntiles == 0) continue;
    host::Timed timed(MUON_KERNEL_MX_DEQUANTIZE, s);
    TRY_CUDA(mx::launch_dequantize(p, dtype, s));
  }
  return MUON_OK;
}

int product_impl(long long m, long long n, long long k, const void* a_data, const void* a_scales, const void* b_data,
                 const void* b_scales, void* out, long long ldo, int dtype, void* stream) {
  TRY(check_side(m, 0, "m"));
  TRY(check_side(n, 0, "n"));
  TRY(check_side(k, 0, "k"));
  TRY(check_dtype(dtype));
  if (((m + 31) / 32) * ((n + 31) / 32) >= (1ll << 31))
    return host::set_error(MUON_ERR_SHAPE, "%lld x %lld has too many tiles", m, n);
  TRY(check_stride(m, n, ldo, "out"));
  if (m == 0 || n == 0) return MUON_OK;
  const long long e = element_size(dtype), ob = extent(m, n, ldo) * e;
  TRY(check_pointer(out, e, "out"));
  int sms = 0;
  cudaStream_t s = as_stream(stream);
  if (k == 0) {  // a sum of nothing
    TRY(host::device_sms(&sms));
    TRY_CUDA(cudaMemset2DAsync(out, m > 1 ? ldo * e : n * e, 0, n * e, m, s));
    return MUON_OK;
  }
  TRY(check_pointer(a_data, 16, "a_data"));
  TRY(check_pointer(a_scales, 16, "a_scales"));
  TRY(check_pointer(b_data, 16, "b_data"));
  TRY(check_pointer(b_scales, 16, "b_scales"));
  Span spans[] = {writes(out, ob, "out"), reads(a_data, m * mx::data_stride(k), "a_data"),
                  reads(a_scales, scale_bytes(m, k), "a_scales"), reads(b_data, n * mx::data_stride(k), "b_data"),
                  reads(b_scales, scale_bytes(n, k), "b_scales")};
  TRY(check_apart(spans, std::size(spans)));
  TRY(host::device_sms(&sms));
  mx::ProductParams p{};
  TRY(host::workspace_status(s, &p.status));
  p.timeout_ns = host::wait_timeout_ns();
  p.inject = host::take_injection();
  // few rows of A: B's rows take the tensor cores' 128-row side
  p.transposed = m <= 64 && n > m;
  p.m = static_cast<int>(p.transposed ? n : m);
  p.n = static_cast<int>(p.transposed ? m : n);
  p.k = static_cast<int>(k);
  p.out = out;
  p.ldo = ldo;
  p.a_scales = p.transposed ? b_scales : a_scales;
  p.b_scales = p.transposed ? a_scales : b_scales;
  const uint64_t row = static_cast<uint64_t>(mx::data_stride(k));
  const int tile_n = mx::product_tile_n(p.m, p.n, p.k, sms);
  TRY(host::encode_2d(&p.a, p.transposed ? b_data : a_data, false, row, p.m, row, 128, 128));
  TRY(host::encode_2d(&p.b, p.transposed ? a_data : b_data, false, row, p.n, row, 128, tile_n == 256 ? 128 : tile_n));
  if (tile_n == 256) {
    const uint64_t words = static_cast<uint64_t>(tile_count(k)) * 128;
    TRY(host::encode_2d(&p.sa, p.a_scales, true, words, tile_count(p.m), words * 4, 256, 1));
    TRY(host::encode_2d(&p.sb, p.b_scales, true, words, tile_count(p.n), words * 4, 256, 2));
  }
  host::Timed timed(MUON_KERNEL_MX_PRODUCT, s);
  TRY_CUDA(mx::launch_product(p, dtype, sms, s));
  return MUON_OK;
}

// No C++ exception leaves a C entry.
template <typename F>
int guarded(F&& f) {
  try {
    host::clear_error();
    return f();
  } catch (const std::bad_alloc&) {
    return MUON_ERR_ALLOC;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

}  // namespace

extern "C" {

int muon_layer_norm(long long rows, long long cols, const void* x, long long ldx, int dtype, const void* weight,
                    const void* bias, int param_dtype, float eps, void* y, long long ldy, float* mean, float* rstd,
                    void* stream) {
  return guarded([&] {
    return forward_impl(rows, cols, x, ldx, dtype, weight, bias, param_dtype, eps, y, ldy, mean, rstd, stream);
  });
}

int muon_layer_norm_scratch_bytes(long long rows, long long cols, long long* bytes) {
  return guarded([&]() -> int {
    if (!bytes) return host::set_error(MUON_ERR_ARG, "bytes is NULL");
    TRY(check_side(rows, 0, "rows"));
    TRY(check_side(cols, 1, "cols"));
    int sms = 0;
    TRY(host::device_sms(&sms));
    *bytes = backward_scratch(rows, cols, sms);
    return MUON_OK;
  });
}

int muon_layer_norm_backward(long long rows, long long cols, const void* dy, long long lddy, const void* x, long long ldx,
                             int dtype, const void* weight, int param_dtype, const float* mean, const float* rstd, void* dx,
                             long long lddx, void* dweight, void* dbias, void* scratch, long long scratch_bytes,
                             void* stream) {
  return guarded([&] {
    return backward_impl(rows, cols, dy, lddy, x, ldx, dtype, weight, param_dtype, mean, rstd, dx, lddx, dweight, dbias,
                         scratch, scratch_bytes, stream);
  });
}

int muon_mx_quantize(int count, const void* const* x, const int64_t* shapes, const int64_t* strides, int dtype,
                     void* const* row_data, void* const* row_scales, void* const* col_data, void* const* col_scales,
                     void* stream) {
  return guarded([&] {
    return quantize_impl(count, x, shapes, strides, dtype, row_data, row_scales, col_data, col_scales, stream);
  });
}

int muon_mx_dequantize(int count, const void* const* data, const void* const* scales, const int64_t* shapes,
                       void* const* y, int dtype, void* stream) {
  return guarded([&] { return dequantize_impl(count, data, scales, shapes, y, dtype, stream); });
}

int muon_mx_product(long long m, long long n, long long k, const void* a_data, const void* a_scales, const void* b_data,
                    const void* b_scales, void* out, long long ldo, int dtype, void* stream) {
  return guarded([&] { return product_impl(m, n, k, a_data, a_scales, b_data, b_scales, out, ldo, dtype, stream); });
}

}  // extern "C"
