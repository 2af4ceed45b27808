// Internal declarations of the low-precision products: microscaled 4-bit
// matrices and products of rows grouped by expert.
#pragma once

#include "ozk_internal.h"

namespace ozk {

constexpr int kMaxGroups = 1024;  // the group table of a product lies in shared memory

// A microscaled 4-bit matrix: rows x K in `groups` groups, starting at
// offsets[0..groups] (device) or, where that is null, of rows / groups rows each.
struct Mx4Matrix {
  int64_t rows, K;
  int format, groups;
  const int32_t* offsets;
  uint8_t* codes;
  uint8_t* scales;
};

// Scale words (4 blocks) per row: 64 columns a word for nvfp4, 128 for mxfp4.
inline int mx4_kgroups(int64_t K, int format) {
  const int64_t kpad = ozk_kpad(K), span = format == OZK_MXFP4 ? 128 : 64;
  return static_cast<int>((kpad + span - 1) / span);
}
inline int64_t mx4_row_blocks(int64_t rows, int groups) { return rows / 128 + groups; }

cudaError_t launch_mx4_quantize(const Mx4Matrix& m, const void* x, int64_t ldx, int dtype, float prescale,
                                int num_sms, cudaStream_t stream);
cudaError_t launch_mx4_dequantize(const Mx4Matrix& m, void* out, int64_t ldo, int dtype, int num_sms,
                                  cudaStream_t stream);
int take_mx4_status(int* status);  // the stream is idle; bit 1: bad group offsets

// The products.  kForward: out[t, m] = sum_k x[t, k] w[e][m, k]; kGradRows:
// out[t, m] = sum_k dy[t, k] w[e][k, m]; kGradWeights: out[e][n, m] =
// sum over the rows t of group e of dy[t, n] x[t, m]; kMx4: kForward on 4-bit
// operands, times alpha; kGated: out[t, m] = act(g) u with g the kForward
// product with row m of w[e] (2 M rows) and u that with row M + m, and where
// slopes is given its derivatives by g, u act'(g), and by u, act(g).
enum ProductOp { kForward = 0, kGradRows = 1, kGradWeights = 2, kMx4 = 3, kGated = 4 };
struct Product {
  ProductOp op;
  int dtype;                  // of the 16-bit operands
  int out_type;
  int64_t T;                  // rows over all groups
  int64_t M, N, K;            // output columns; output rows of a group (kGradWeights); terms (else)
  int groups;
  const int32_t* offsets;     // device, groups + 1; null: one group of T rows
  const void* rows;           // x or dy: T rows, the operand with one row per output row (kGradWeights: dy)
  int64_t ld_rows;
  const void* other;          // w (groups x ...; ld_other, other_group), or x for kGradWeights
  int64_t ld_other, other_group;
  void* out;
  int64_t ldo, out_group;
  Mx4Matrix a, b;             // kMx4: rows and weights
  float alpha;
  int act;                    // kGated
  float* slopes;              // [2][T][M], rows lds and the two slope_plane elements apart; or null
  int64_t lds, slope_plane;
};
// dpre[t, m] = dh[t, m] slopes[0][t, m], dpre[t, M + m] = dh[t, m] slopes[1][t, m]
// for the rows of the groups (offsets null: all T rows).
struct GatedGrad {
  int64_t T, M;
  int groups;
  const int32_t* offsets;
  int dtype;
  const void* dh;
  const float* slopes;
  int64_t lddh, lds, slope_plane;
  void* out;
  int64_t ldo;
  void* clear;  // T x K, rows ldc apart: zeros for rows in no group; or null
  int64_t K, ldc;
};
cudaError_t launch_gated_grad(const GatedGrad& q, int num_sms, cudaStream_t stream);
int take_gated_status(int* status);  // the stream is idle; bit 1: bad group offsets
cudaError_t launch_product(const Product& q, int num_sms, cudaStream_t stream);
void withhold_next_product(int pairs, int cta, int kblock, uint32_t timeout_us);  // test hook, see ozk.h
int take_product_status(int* status);  // the stream is idle; bit 0: a wait ran out, bit 1: bad group offsets


// A few 16-bit rows times 4-bit weights (w: groups equal groups of N rows,
// gated 2 N): y[t, n] = alpha sum_k x[t, k] w[g(t)][n, k], or act of it times
// that of row N + n.
struct Gemv {
  int64_t T, N, K;
  const int32_t* offsets;  // device, w.groups + 1; null: one group of T rows
  const void* x;
  int64_t ldx;
  int dtype;
  Mx4Matrix w;
  float alpha;
  bool gated;
  int act;
  void* y;
  int64_t ldy;
  int out_type;
};
cudaError_t launch_mx4_gemv(const Gemv& q, int num_sms, cudaStream_t stream);
int take_gemv_status(int* status);  // the stream is idle; bit 1: bad group offsets

}  // namespace ozk
