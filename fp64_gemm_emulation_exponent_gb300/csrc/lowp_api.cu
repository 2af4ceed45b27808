// C-ABI of the low-precision products: argument checks of the microscaled
// 4-bit matrices and of the products of rows grouped by expert.
#include <cuda_runtime.h>

#include <cmath>

#include "lowp.h"

namespace ozk {
namespace {

constexpr int64_t kMaxRows = INT32_MAX / 2;
constexpr int64_t kMaxFeatures = 1 << 22;
constexpr int64_t kMaxTiles = INT32_MAX / 2;  // tile numbers are ints

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
size_t size_of(int dtype) { return dtype == OZK_F64 ? 8 : dtype == OZK_F32 ? 4 : 2; }

struct Span {
  uintptr_t lo, hi;
};
// Bytes of `groups` matrices of rows x cols (leading dimension ld, `group` elements apart).
Span span(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t esize, int64_t groups = 1, int64_t group = 0) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (rows <= 0 || cols <= 0 || groups <= 0) return {a, a};
  return {a, a + esize * static_cast<size_t>((groups - 1) * group + (rows - 1) * ld + cols)};
}
// Memory of no bytes overlaps nothing, whatever its address.
bool overlap(const Span& x, const Span& y) {
  return x.lo < x.hi && y.lo < y.hi && x.lo < y.hi && y.lo < x.hi;
}

bool known_format(int f) { return f == OZK_NVFP4 || f == OZK_MXFP4; }
bool known_dtype(int t) { return t >= OZK_BF16 && t <= OZK_F64; }

int check_mx4(int64_t rows, int64_t K, int format, const int32_t* offsets, int groups) {
  if (rows < 0 || K < 0 || !known_format(format) || groups < 1) return OZK_ERR_INVALID_ARG;
  if (rows > kMaxRows || K > kMaxFeatures || groups > kMaxGroups) return OZK_ERR_UNSUPPORTED;
  if (offsets == nullptr && rows % groups != 0) return OZK_ERR_INVALID_ARG;
  return OZK_OK;
}

Mx4Matrix matrix(int64_t rows, int64_t K, int format, const int32_t* offsets, int groups, const uint8_t* codes,
                 const uint8_t* scales) {
  return {rows, K, format, groups, offsets, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales)};
}

bool countable(int64_t tiles_m, int64_t tiles_n) { return tiles_m == 0 || tiles_n <= kMaxTiles / tiles_m; }
int64_t tiles_of(int64_t n) { return (n + 127) / 128; }

int run(const Product& q, cudaStream_t stream, int sms) {
  const int64_t tiles_n = q.op == kGradWeights ? tiles_of(q.N) * q.groups : q.T / 128 + q.groups;
  if (!countable(tiles_of(q.op == kGated ? 2 * q.M : q.M), tiles_n)) return OZK_ERR_UNSUPPORTED;
  try {  // the launcher's tables may allocate; nothing is thrown across the C boundary
    return launch_product(q, sms, stream) == cudaSuccess ? OZK_OK : OZK_ERR_CUDA;
  } catch (...) {
    return OZK_ERR_CUDA;
  }
}

// What the three 16-bit products share: T rows of x (K columns) and of y or
// its gradient (N columns), weights N x K per group.
int check_grouped(int64_t T, int64_t N, int64_t K, int groups, const int32_t* offsets, int dtype, int out_dtype) {
  if (T < 0 || N < 0 || K < 0 || groups < 1 || offsets == nullptr) return OZK_ERR_INVALID_ARG;
  if (dtype != OZK_BF16 && dtype != OZK_F16) return OZK_ERR_UNSUPPORTED;
  if (out_dtype != dtype && out_dtype != OZK_F32) return OZK_ERR_UNSUPPORTED;
  if (T > kMaxRows || N > kMaxFeatures || K > kMaxFeatures || groups > kMaxGroups) return OZK_ERR_UNSUPPORTED;
  return OZK_OK;
}
// An operand of the 16-bit products: rows of `cols` elements, read by bulk
// tensor copies (16-byte aligned base and strides).
int check_operand(const void* p, int64_t cols, int64_t ld) {
  if (p == nullptr || ld < cols) return OZK_ERR_INVALID_ARG;
  if (!aligned16(p) || ld % 8 != 0) return OZK_ERR_UNSUPPORTED;
  return OZK_OK;
}
int check_weights(const void* w, int64_t N, int64_t K, int64_t ldw, int groups, int64_t stride) {
  const int rc = check_operand(w, K, ldw);
  if (rc) return rc;
  if (groups > 1 && stride < (N - 1) * ldw + K) return OZK_ERR_INVALID_ARG;
  if (groups > 1 && stride % 8 != 0) return OZK_ERR_UNSUPPORTED;
  return OZK_OK;
}

bool known_activation(int a) { return a >= OZK_SILU && a <= OZK_GELU_TANH; }

// The two slopes of a gated product: rows of N elements, lds apart, `plane` between the two.
int check_slopes(const float* s, int64_t T, int64_t N, int64_t lds, int64_t plane) {
  if (!s || reinterpret_cast<uintptr_t>(s) % 4 != 0 || lds < N || plane < (T - 1) * lds + N) return OZK_ERR_INVALID_ARG;
  return OZK_OK;
}

// A few 16-bit rows times 4-bit weights, plain or gated.
int gemv(int64_t T, int64_t N, int64_t K, int groups, const int32_t* offsets, const void* X, int64_t ldx, int dtype,
         const uint8_t* codes, const uint8_t* scales, int format, float alpha, bool gated, int act, void* Y, int64_t ldy,
         int out_dtype, cudaStream_t stream) {
  if (T < 0 || N < 0 || K < 0 || !known_format(format) || groups < 1) return OZK_ERR_INVALID_ARG;
  if (offsets == nullptr && groups != 1) return OZK_ERR_INVALID_ARG;
  if (gated && !known_activation(act)) return OZK_ERR_INVALID_ARG;
  if (dtype != OZK_BF16 && dtype != OZK_F16) return OZK_ERR_UNSUPPORTED;
  if (out_dtype != OZK_BF16 && out_dtype != OZK_F16 && out_dtype != OZK_F32) return OZK_ERR_UNSUPPORTED;
  const int64_t per = gated ? 2 : 1;  // rows of w of an output column
  if (T > kMaxRows || N > kMaxFeatures || K > kMaxFeatures || groups > kMaxGroups || per * N > kMaxRows / groups)
    return OZK_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return OZK_OK;
  if (!Y || ldy < N || reinterpret_cast<uintptr_t>(Y) % size_of(out_dtype) != 0) return OZK_ERR_INVALID_ARG;
  const int64_t rows = per * N * groups;
  if (K > 0) {
    if (!X || ldx < K || reinterpret_cast<uintptr_t>(X) % 2 != 0) return OZK_ERR_INVALID_ARG;
    if (!codes || !scales || !aligned16(codes) || !aligned16(scales)) return OZK_ERR_INVALID_ARG;
    const Span y = span(Y, T, N, ldy, size_of(out_dtype));
    if (overlap(y, span(X, T, K, ldx, 2)) || overlap(y, span(codes, 1, rows * (ozk_kpad(K) / 2), 0, 1)) ||
        overlap(y, span(scales, 1, static_cast<int64_t>(ozk_mx4_scale_bytes(rows, K, format, groups)), 0, 1)))
      return OZK_ERR_INVALID_ARG;
  }
  int sms = 0;
  const int rc = current_device_supported(&sms);
  if (rc) return rc;
  const Gemv q = {T, N, K, offsets, X, ldx, dtype, matrix(rows, K, format, nullptr, groups, codes, scales), alpha, gated,
                  act, Y, ldy, out_dtype};
  try {  // the launcher's table may allocate; nothing is thrown across the C boundary
    return launch_mx4_gemv(q, sms, stream) == cudaSuccess ? OZK_OK : OZK_ERR_CUDA;
  } catch (...) {
    return OZK_ERR_CUDA;
  }
}

}  // namespace
}  // namespace ozk

using namespace ozk;

extern "C" {

size_t ozk_mx4_scale_bytes(int64_t rows, int64_t K, int format, int groups) {
  if (rows < 0 || rows > kMaxRows || K < 0 || K > kMaxFeatures || !known_format(format) || groups < 1 ||
      groups > kMaxGroups)
    return 0;
  return static_cast<size_t>(mx4_row_blocks(rows, groups)) * static_cast<size_t>(mx4_kgroups(K, format)) * 512;
}

int ozk_mx4_quantize(int64_t rows, int64_t K, const void* X, int64_t ldx, int dtype, int format, float prescale,
                     const int32_t* offsets, int groups, uint8_t* codes, uint8_t* scales, ozk_stream_t stream) {
  int rc = check_mx4(rows, K, format, offsets, groups);
  if (rc) return rc;
  if (!known_dtype(dtype) || !(prescale > 0.0f) || !std::isfinite(prescale)) return OZK_ERR_INVALID_ARG;
  if (rows == 0 || K == 0) return OZK_OK;
  if (!X || ldx < K || !codes || !scales || !aligned16(codes) || !aligned16(scales)) return OZK_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(X) % size_of(dtype) != 0) return OZK_ERR_INVALID_ARG;
  const Span x = span(X, rows, K, ldx, size_of(dtype));
  const Span c = span(codes, 1, rows * (ozk_kpad(K) / 2), 0, 1);
  const Span s = span(scales, 1, static_cast<int64_t>(ozk_mx4_scale_bytes(rows, K, format, groups)), 0, 1);
  if (overlap(x, c) || overlap(x, s) || overlap(c, s)) return OZK_ERR_INVALID_ARG;
  int sms = 0;
  rc = current_device_supported(&sms);
  if (rc) return rc;
  const Mx4Matrix m = matrix(rows, K, format, offsets, groups, codes, scales);
  return launch_mx4_quantize(m, X, ldx, dtype, prescale, sms, stream) == cudaSuccess ? OZK_OK : OZK_ERR_CUDA;
}

int ozk_mx4_dequantize(int64_t rows, int64_t K, const uint8_t* codes, const uint8_t* scales, int format,
                       const int32_t* offsets, int groups, void* X, int64_t ldx, int dtype, ozk_stream_t stream) {
  int rc = check_mx4(rows, K, format, offsets, groups);
  if (rc) return rc;
  if (!known_dtype(dtype)) return OZK_ERR_INVALID_ARG;
  if (rows == 0 || K == 0) return OZK_OK;
  if (!X || ldx < K || !codes || !scales || !aligned16(codes) || !aligned16(scales)) return OZK_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(X) % size_of(dtype) != 0) return OZK_ERR_INVALID_ARG;
  const Span x = span(X, rows, K, ldx, size_of(dtype));
  const Span c = span(codes, 1, rows * (ozk_kpad(K) / 2), 0, 1);
  const Span s = span(scales, 1, static_cast<int64_t>(ozk_mx4_scale_bytes(rows, K, format, groups)), 0, 1);
  if (overlap(x, c) || overlap(x, s)) return OZK_ERR_INVALID_ARG;
  int sms = 0;
  rc = current_device_supported(&sms);
  if (rc) return rc;
  const Mx4Matrix m = matrix(rows, K, format, offsets, groups, codes, scales);
  return launch_mx4_dequantize(m, X, ldx, dtype, sms, stream) == cudaSuccess ? OZK_OK : OZK_ERR_CUDA;
}

int ozk_mx4_grouped_gemm(int64_t T, int64_t N, int64_t K, int groups, const int32_t* offsets, const uint8_t* x_codes,
                         const uint8_t* x_scales, const uint8_t* w_codes, const uint8_t* w_scales, int format,
                         float alpha, void* Y, int64_t ldy, int out_dtype, ozk_stream_t stream) {
  if (T < 0 || N < 0 || K < 0 || !known_format(format) || groups < 1) return OZK_ERR_INVALID_ARG;
  if (offsets == nullptr && groups != 1) return OZK_ERR_INVALID_ARG;
  if (out_dtype != OZK_BF16 && out_dtype != OZK_F16 && out_dtype != OZK_F32) return OZK_ERR_UNSUPPORTED;
  if (T > kMaxRows || N > kMaxFeatures || K > kMaxFeatures || groups > kMaxGroups || N > kMaxRows / groups)
    return OZK_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return OZK_OK;
  if (!Y || ldy < N || reinterpret_cast<uintptr_t>(Y) % size_of(out_dtype) != 0) return OZK_ERR_INVALID_ARG;
  Product q = {};
  q.op = kMx4;
  q.out_type = out_dtype;
  q.T = T;
  q.M = N;
  q.K = K;
  q.groups = groups;
  q.offsets = offsets;
  q.out = Y;
  q.ldo = ldy;
  q.alpha = alpha;
  q.a = matrix(T, K, format, offsets, groups, x_codes, x_scales);
  q.b = matrix(N * groups, K, format, nullptr, groups, w_codes, w_scales);
  if (K > 0) {
    if (!x_codes || !x_scales || !w_codes || !w_scales) return OZK_ERR_INVALID_ARG;
    if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(w_codes) || !aligned16(w_scales))
      return OZK_ERR_INVALID_ARG;
    const Span y = span(Y, T, N, ldy, size_of(out_dtype));
    for (const Mx4Matrix* m : {&q.a, &q.b}) {
      const int64_t cb = m->rows * (ozk_kpad(K) / 2);
      const int64_t sb = static_cast<int64_t>(ozk_mx4_scale_bytes(m->rows, K, format, groups));
      if (overlap(y, span(m->codes, 1, cb, 0, 1)) || overlap(y, span(m->scales, 1, sb, 0, 1)))
        return OZK_ERR_INVALID_ARG;
    }
  }
  int sms = 0;
  const int rc = current_device_supported(&sms);
  return rc ? rc : run(q, stream, sms);
}

int ozk_mx4_gemm(int64_t M, int64_t N, int64_t K, const uint8_t* a_codes, const uint8_t* a_scales,
                 const uint8_t* b_codes, const uint8_t* b_scales, int format, float alpha, void* C, int64_t ldc,
                 int out_dtype, ozk_stream_t stream) {
  return ozk_mx4_grouped_gemm(M, N, K, 1, nullptr, a_codes, a_scales, b_codes, b_scales, format, alpha, C, ldc,
                              out_dtype, stream);
}

int ozk_mx4_gemv(int64_t T, int64_t N, int64_t K, int groups, const int32_t* offsets, const void* X, int64_t ldx,
                 int dtype, const uint8_t* w_codes, const uint8_t* w_scales, int format, float alpha, void* Y,
                 int64_t ldy, int out_dtype, ozk_stream_t stream) {
  return gemv(T, N, K, groups, offsets, X, ldx, dtype, w_codes, w_scales, format, alpha, false, OZK_SILU, Y, ldy,
              out_dtype, stream);
}

int ozk_mx4_gated_gemv(int64_t T, int64_t N, int64_t K, int groups, const int32_t* offsets, const void* X, int64_t ldx,
                       int dtype, const uint8_t* w_codes, const uint8_t* w_scales, int format, float alpha,
                       int activation, void* Y, int64_t ldy, int out_dtype, ozk_stream_t stream) {
  return gemv(T, N, K, groups, offsets, X, ldx, dtype, w_codes, w_scales, format, alpha, true, activation, Y, ldy,
              out_dtype, stream);
}

int ozk_grouped_gemm(int64_t T, int64_t N, int64_t K, int groups, const int32_t* offsets, const void* X, int64_t ldx,
                     const void* W, int64_t ldw, int64_t w_stride, int dtype, void* Y, int64_t ldy, int out_dtype,
                     ozk_stream_t stream) {
  int rc = check_grouped(T, N, K, groups, offsets, dtype, out_dtype);
  if (rc) return rc;
  if (T == 0 || N == 0) return OZK_OK;
  if (!Y || ldy < N || reinterpret_cast<uintptr_t>(Y) % size_of(out_dtype) != 0) return OZK_ERR_INVALID_ARG;
  if (K > 0) {
    if ((rc = check_operand(X, K, ldx)) || (rc = check_weights(W, N, K, ldw, groups, w_stride))) return rc;
    const Span y = span(Y, T, N, ldy, size_of(out_dtype));
    if (overlap(y, span(X, T, K, ldx, 2)) || overlap(y, span(W, N, K, ldw, 2, groups, w_stride)))
      return OZK_ERR_INVALID_ARG;
  }
  Product q = {};
  q.op = kForward;
  q.dtype = dtype;
  q.out_type = out_dtype;
  q.T = T;
  q.M = N;
  q.K = K;
  q.groups = groups;
  q.offsets = offsets;
  q.rows = X;
  q.ld_rows = ldx;
  q.other = W;
  q.ld_other = ldw;
  q.other_group = groups > 1 ? w_stride : N * ldw;
  q.out = Y;
  q.ldo = ldy;
  q.alpha = 1.0f;
  int sms = 0;
  rc = current_device_supported(&sms);
  return rc ? rc : run(q, stream, sms);
}

int ozk_grouped_gated_gemm(int64_t T, int64_t N, int64_t K, int groups, const int32_t* offsets, const void* X,
                           int64_t ldx, const void* W, int64_t ldw, int64_t w_stride, int dtype, int activation,
                           void* Y, int64_t ldy, float* slopes, int64_t lds, int64_t slope_stride,
                           ozk_stream_t stream) {
  int rc = check_grouped(T, N, K, groups, offsets, dtype, dtype);
  if (rc) return rc;
  if (!known_activation(activation)) return OZK_ERR_INVALID_ARG;
  if (2 * N > kMaxFeatures) return OZK_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return OZK_OK;
  if (!Y || ldy < N || reinterpret_cast<uintptr_t>(Y) % 2 != 0) return OZK_ERR_INVALID_ARG;
  const Span y = span(Y, T, N, ldy, 2), s = span(slopes, T, N, lds, 4, 2, slope_stride);
  if (slopes) {
    if ((rc = check_slopes(slopes, T, N, lds, slope_stride))) return rc;
    if (overlap(y, s)) return OZK_ERR_INVALID_ARG;
  }
  if (K > 0) {
    if ((rc = check_operand(X, K, ldx)) || (rc = check_weights(W, 2 * N, K, ldw, groups, w_stride))) return rc;
    const Span x = span(X, T, K, ldx, 2), w = span(W, 2 * N, K, ldw, 2, groups, w_stride);
    if (overlap(y, x) || overlap(y, w) || (slopes && (overlap(s, x) || overlap(s, w)))) return OZK_ERR_INVALID_ARG;
  }
  Product q = {};
  q.op = kGated;
  q.dtype = dtype;
  q.out_type = dtype;
  q.T = T;
  q.M = N;
  q.K = K;
  q.groups = groups;
  q.offsets = offsets;
  q.rows = X;
  q.ld_rows = ldx;
  q.other = W;
  q.ld_other = ldw;
  q.other_group = groups > 1 ? w_stride : 2 * N * ldw;
  q.out = Y;
  q.ldo = ldy;
  q.alpha = 1.0f;
  q.act = activation;
  q.slopes = slopes;
  q.lds = lds;
  q.slope_plane = slope_stride;
  int sms = 0;
  rc = current_device_supported(&sms);
  return rc ? rc : run(q, stream, sms);
}

int ozk_gated_grad(int64_t T, int64_t N, int groups, const int32_t* offsets, const void* dH, int64_t lddh,
                   const float* slopes, int64_t lds, int64_t slope_stride, int dtype, void* dpre, int64_t ldp,
                   ozk_stream_t stream) {
  if (T < 0 || N < 0 || groups < 1 || (offsets == nullptr && groups != 1)) return OZK_ERR_INVALID_ARG;
  if (dtype != OZK_BF16 && dtype != OZK_F16) return OZK_ERR_UNSUPPORTED;
  if (T > kMaxRows || 2 * N > kMaxFeatures || groups > kMaxGroups) return OZK_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return OZK_OK;
  if (!dH || lddh < N || reinterpret_cast<uintptr_t>(dH) % 2 != 0) return OZK_ERR_INVALID_ARG;
  if (!dpre || ldp < 2 * N || reinterpret_cast<uintptr_t>(dpre) % 2 != 0) return OZK_ERR_INVALID_ARG;
  int rc = check_slopes(slopes, T, N, lds, slope_stride);
  if (rc) return rc;
  const Span d = span(dpre, T, 2 * N, ldp, 2);
  if (overlap(d, span(dH, T, N, lddh, 2)) || overlap(d, span(slopes, T, N, lds, 4, 2, slope_stride)))
    return OZK_ERR_INVALID_ARG;
  int sms = 0;
  if ((rc = current_device_supported(&sms))) return rc;
  const GatedGrad q = {T, N, groups, offsets, dtype, dH, slopes, lddh, lds, slope_stride, dpre, ldp, nullptr, 0, 0};
  return launch_gated_grad(q, sms, stream) == cudaSuccess ? OZK_OK : OZK_ERR_CUDA;
}

int ozk_grouped_gated_gemm_grad(int64_t T, int64_t N, int64_t K, int groups, const int32_t* offsets, const void* dH,
                                int64_t lddh, const float* slopes, int64_t lds, int64_t slope_stride, const void* X,
                                int64_t ldx, const void* W, int64_t ldw, int64_t w_stride, int dtype, void* dpre,
                                int64_t ldp, void* dX, int64_t lddx, void* dW, int64_t lddw, int64_t dw_stride,
                                ozk_stream_t stream) {
  int rc = check_grouped(T, N, K, groups, offsets, dtype, dtype);
  if (rc) return rc;
  if (2 * N > kMaxFeatures) return OZK_ERR_UNSUPPORTED;
  if (T > 0 && N > 0) {
    if (!dH || lddh < N || reinterpret_cast<uintptr_t>(dH) % 2 != 0) return OZK_ERR_INVALID_ARG;
    if ((rc = check_slopes(slopes, T, N, lds, slope_stride)) || (rc = check_operand(dpre, 2 * N, ldp))) return rc;
    if (dX && K > 0 && (rc = check_weights(W, 2 * N, K, ldw, groups, w_stride))) return rc;
    if (dW && K > 0 && (rc = check_operand(X, K, ldx))) return rc;
  }
  // all three results are written before the last operand has been read; dX without columns and dW without rows too
  const Span out[3] = {span(dpre, T, 2 * N, ldp, 2), span(dX, dX ? T : 0, K, lddx, 2),
                       span(dW, dW ? 2 * N : 0, K, lddw, 2, groups, dw_stride)};
  const Span in[4] = {span(dH, T, N, lddh, 2), span(slopes, T, N, lds, 4, 2, slope_stride), span(X, T, K, ldx, 2),
                      span(W, 2 * N, K, ldw, 2, groups, w_stride)};
  for (int i = 0; i < 3; ++i) {
    for (const Span& s : in)
      if (overlap(out[i], s)) return OZK_ERR_INVALID_ARG;
    if (overlap(out[i], out[(i + 1) % 3])) return OZK_ERR_INVALID_ARG;
  }
  // whatever the calls below would refuse is refused here, before the first of them has written
  if (dX && T > 0 && K > 0 && (lddx < K || reinterpret_cast<uintptr_t>(dX) % 2 != 0)) return OZK_ERR_INVALID_ARG;
  if (dW && N > 0 && K > 0 &&
      (lddw < K || reinterpret_cast<uintptr_t>(dW) % 2 != 0 || (groups > 1 && dw_stride < (2 * N - 1) * lddw + K)))
    return OZK_ERR_INVALID_ARG;
  if (dX && T > 0 && !countable(tiles_of(K), T / 128 + groups)) return OZK_ERR_UNSUPPORTED;
  if (dW && !countable(tiles_of(K), tiles_of(2 * N) * groups)) return OZK_ERR_UNSUPPORTED;
  int sms = 0;
  if ((rc = current_device_supported(&sms))) return rc;
  if (T > 0 && (N > 0 || (dX && K > 0))) {
    const GatedGrad q = {T, N, groups, offsets, dtype, dH, slopes, lddh, lds, slope_stride, dpre, ldp, K > 0 ? dX : nullptr, K, lddx};
    if (launch_gated_grad(q, sms, stream) != cudaSuccess) return OZK_ERR_CUDA;
  }
  if (dX && (rc = ozk_grouped_gemm_dx(T, 2 * N, K, groups, offsets, dpre, ldp, W, ldw, w_stride, dtype, dX, lddx, dtype, stream)))
    return rc;
  return dW ? ozk_grouped_gemm_dw(T, 2 * N, K, groups, offsets, dpre, ldp, X, ldx, dtype, dW, lddw, dw_stride, dtype, stream)
            : OZK_OK;
}

int ozk_grouped_gemm_dx(int64_t T, int64_t N, int64_t K, int groups, const int32_t* offsets, const void* dY,
                        int64_t lddy, const void* W, int64_t ldw, int64_t w_stride, int dtype, void* dX, int64_t lddx,
                        int out_dtype, ozk_stream_t stream) {
  int rc = check_grouped(T, N, K, groups, offsets, dtype, out_dtype);
  if (rc) return rc;
  if (T == 0 || K == 0) return OZK_OK;
  if (!dX || lddx < K || reinterpret_cast<uintptr_t>(dX) % size_of(out_dtype) != 0) return OZK_ERR_INVALID_ARG;
  if (N > 0) {
    if ((rc = check_operand(dY, N, lddy)) || (rc = check_weights(W, N, K, ldw, groups, w_stride))) return rc;
    const Span x = span(dX, T, K, lddx, size_of(out_dtype));
    if (overlap(x, span(dY, T, N, lddy, 2)) || overlap(x, span(W, N, K, ldw, 2, groups, w_stride)))
      return OZK_ERR_INVALID_ARG;
  }
  Product q = {};
  q.op = kGradRows;
  q.dtype = dtype;
  q.out_type = out_dtype;
  q.T = T;
  q.M = K;
  q.K = N;
  q.groups = groups;
  q.offsets = offsets;
  q.rows = dY;
  q.ld_rows = lddy;
  q.other = W;
  q.ld_other = ldw;
  q.other_group = groups > 1 ? w_stride : N * ldw;
  q.out = dX;
  q.ldo = lddx;
  q.alpha = 1.0f;
  int sms = 0;
  rc = current_device_supported(&sms);
  return rc ? rc : run(q, stream, sms);
}

int ozk_grouped_gemm_dw(int64_t T, int64_t N, int64_t K, int groups, const int32_t* offsets, const void* dY,
                        int64_t lddy, const void* X, int64_t ldx, int dtype, void* dW, int64_t lddw, int64_t dw_stride,
                        int out_dtype, ozk_stream_t stream) {
  int rc = check_grouped(T, N, K, groups, offsets, dtype, out_dtype);
  if (rc) return rc;
  if (N == 0 || K == 0) return OZK_OK;
  if (!dW || lddw < K || reinterpret_cast<uintptr_t>(dW) % size_of(out_dtype) != 0) return OZK_ERR_INVALID_ARG;
  if (groups > 1 && dw_stride < (N - 1) * lddw + K) return OZK_ERR_INVALID_ARG;
  if (T > 0) {
    if ((rc = check_operand(dY, N, lddy)) || (rc = check_operand(X, K, ldx))) return rc;
    const Span w = span(dW, N, K, lddw, size_of(out_dtype), groups, dw_stride);
    if (overlap(w, span(dY, T, N, lddy, 2)) || overlap(w, span(X, T, K, ldx, 2))) return OZK_ERR_INVALID_ARG;
  }
  Product q = {};
  q.op = kGradWeights;
  q.dtype = dtype;
  q.out_type = out_dtype;
  q.T = T;
  q.M = K;
  q.N = N;
  q.K = 1;
  q.groups = groups;
  q.offsets = offsets;
  q.rows = dY;
  q.ld_rows = lddy;
  q.other = X;
  q.ld_other = ldx;
  q.out = dW;
  q.ldo = lddw;
  q.out_group = dw_stride;
  q.alpha = 1.0f;
  int sms = 0;
  rc = current_device_supported(&sms);
  return rc ? rc : run(q, stream, sms);
}

int ozk_withhold_next_product(int pairs, int cta, int kblock, uint32_t timeout_us) {
  if (pairs < 0 || pairs > 1 || cta < 0 || cta > pairs || kblock < -1 || timeout_us > 1000000u)
    return OZK_ERR_INVALID_ARG;
  withhold_next_product(pairs, cta, kblock, timeout_us);
  return OZK_OK;
}

}  // extern "C"
