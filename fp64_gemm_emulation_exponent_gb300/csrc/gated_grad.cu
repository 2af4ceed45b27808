// The gradient of a gated product with respect to its two projections:
//   dpre[t, m] = dh[t, m] s0[t, m],   dpre[t, M + m] = dh[t, m] s1[t, m],
// s0 = dh/dgate = u act'(g) and s1 = dh/dup = act(g) as the forward product
// stored them in fp32, so no exponential is taken here and the activation is not
// known.  Each product is rounded to fp32 and to 16 bits.
//
// 14 bytes move for an element of dh: bound by HBM.  A warp takes a row's run of
// up to 512 columns with 16-byte accesses, the loads of two vectors ahead of
// the stores: 16384 x 4096 bf16 134 us, 7.0 TB/s.  Where the gradient of x follows, the kernel also
// clears its rows in no group, which the product leaves as they are.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "lowp.h"

namespace ozk {
namespace {

__device__ int g_gated_status;  // bit 1: bad group offsets

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 2;
constexpr int kRun = 32 * 8 * kUnroll;  // columns of a unit

struct GradParams {
  int64_t lddh, lds, plane, ldo;
  int T, M, groups, runs;  // runs: units of a row
  FastDiv div_runs;
  const int32_t* offsets;
  const uint16_t* dh;
  const float* slopes;
  uint16_t* out;
  uint16_t* clear;   // T x K, or null: rows in no group are set to zero
  int64_t ldc;
  int K;
};

// The rows of the groups: they follow one another from the first offset to the
// largest, cut to [0, T].
__device__ __forceinline__ int2 rows_of(const GradParams& p) {
  const int lane = threadIdx.x & 31;
  int most = 0;
  bool bad = false;
  for (int i = lane; i <= p.groups; i += 32) {
    const int at = p.offsets[i];
    most = max(most, at);
    if (blockIdx.x == 0) bad |= at < (i ? p.offsets[i - 1] : 0) || at > p.T;
  }
  most = min(static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, most)), p.T);
  if (blockIdx.x == 0 && __any_sync(0xFFFFFFFFu, bad) && threadIdx.x == 0) atomicOr(&g_gated_status, 2);
  return {min(max(p.offsets[0], 0), p.T), most};
}

// Both elements of a 16-bit pair times an fp32 factor each.
template <bool BF>
__device__ __forceinline__ uint32_t mul2(uint32_t d, float lo, float hi) {
  uint32_t r;
  if (BF) {
    lo *= __uint_as_float(d << 16);
    hi *= __uint_as_float(d & 0xFFFF0000u);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  } else {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&d));
    lo *= v.x;
    hi *= v.y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  }
  return r;
}
template <bool BF>
__device__ __forceinline__ uint4 mul8(const uint4& d, const uint4 (&s)[2]) {
  auto f = [](uint32_t v) { return __uint_as_float(v); };
  return make_uint4(mul2<BF>(d.x, f(s[0].x), f(s[0].y)), mul2<BF>(d.y, f(s[0].z), f(s[0].w)),
                    mul2<BF>(d.z, f(s[1].x), f(s[1].y)), mul2<BF>(d.w, f(s[1].z), f(s[1].w)));
}
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// Zeros into row `row` of what is to be cleared: the whole warp.
__device__ __forceinline__ void clear_row(const GradParams& p, int64_t row, int lane) {
  uint16_t* to = p.clear + row * p.ldc;
  const int head = min(p.K, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(to) & 15)) / 2 % 8));
  for (int c = lane; c < head; c += 32) to[c] = 0;
  const int vectors = (p.K - head) / 8;
  for (int v = lane; v < vectors; v += 32) *reinterpret_cast<uint4*>(to + head + 8 * v) = make_uint4(0u, 0u, 0u, 0u);
  for (int c = head + 8 * vectors + lane; c < p.K; c += 32) to[c] = 0;
}

// VEC: rows and halves of dpre that start on 16 bytes; else element by element.
template <bool BF, bool VEC>
__global__ void __launch_bounds__(kThreads) gated_grad_kernel(const GradParams p) {
  grid_dependency_sync();
  const int lane = threadIdx.x & 31;
  const int2 span = p.offsets ? rows_of(p) : make_int2(0, p.T);
  const int64_t units = static_cast<int64_t>(span.y - span.x) * p.runs;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kWarps) {
    int64_t row;
    if (u < (int64_t{1} << 31)) row = div_fast(static_cast<uint32_t>(u), p.div_runs);
    else row = u / p.runs;
    const int c0 = static_cast<int>(u - row * p.runs) * kRun;
    row += span.x;
    const uint16_t* dh = p.dh + row * p.lddh;
    const float *s0 = p.slopes + row * p.lds, *s1 = s0 + p.plane;
    uint16_t *o0 = p.out + row * p.ldo, *o1 = o0 + p.M;
    if (VEC) {
      uint4 d[kUnroll], a[kUnroll][2], b[kUnroll][2];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int c = c0 + (i * 32 + lane) * 8;
        if (c >= p.M) continue;
        d[i] = load16(dh + c);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          a[i][j] = load16(s0 + c + 4 * j);
          b[i][j] = load16(s1 + c + 4 * j);
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int c = c0 + (i * 32 + lane) * 8;
        if (c >= p.M) continue;
        *reinterpret_cast<uint4*>(o0 + c) = mul8<BF>(d[i], a[i]);
        *reinterpret_cast<uint4*>(o1 + c) = mul8<BF>(d[i], b[i]);
      }
    } else {
      const int end = min(c0 + kRun, p.M);
      for (int c = c0 + lane; c < end; c += 32) {
        const uint32_t d = dh[c];
        o0[c] = static_cast<uint16_t>(mul2<BF>(d, s0[c], 0.0f));
        o1[c] = static_cast<uint16_t>(mul2<BF>(d, s1[c], 0.0f));
      }
    }
  }
  if (p.clear == nullptr) return;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < span.x + (p.T - span.y); r += step)
    clear_row(p, r < span.x ? r : r - span.x + span.y, lane);
}

std::atomic<bool> g_any{false};

}  // namespace

cudaError_t launch_gated_grad(const GatedGrad& q, int num_sms, cudaStream_t stream) {
  g_any.store(true, std::memory_order_relaxed);
  GradParams p = {};
  p.lddh = q.lddh;
  p.lds = q.lds;
  p.plane = q.slope_plane;
  p.ldo = q.ldo;
  p.T = static_cast<int>(q.T);
  p.M = static_cast<int>(q.M);
  p.groups = q.groups;
  p.runs = static_cast<int>((q.M + kRun - 1) / kRun);
  p.div_runs = fast_div(p.runs);
  p.offsets = q.offsets;
  p.dh = static_cast<const uint16_t*>(q.dh);
  p.slopes = q.slopes;
  p.out = static_cast<uint16_t*>(q.out);
  p.clear = static_cast<uint16_t*>(q.clear);
  p.ldc = q.ldc;
  p.K = static_cast<int>(q.K);
  auto aligned = [](const void* a) { return reinterpret_cast<uintptr_t>(a) % 16 == 0; };
  const bool vec = aligned(q.dh) && aligned(q.slopes) && aligned(q.out) && q.M % 8 == 0 && (q.T == 1 || q.lddh % 8 == 0) &&
                   (q.T == 1 || q.lds % 4 == 0) && q.slope_plane % 4 == 0 && (q.T == 1 || q.ldo % 8 == 0);
  const int64_t units = q.T * std::max(p.runs, 1);  // rows that are cleared want warps too
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((units + kWarps - 1) / kWarps, 8 * num_sms)));
  const bool bf = q.dtype == OZK_BF16;
  auto kernel = bf ? (vec ? gated_grad_kernel<true, true> : gated_grad_kernel<true, false>)
                   : (vec ? gated_grad_kernel<false, true> : gated_grad_kernel<false, false>);
  return launch_dependent(kernel, grid, dim3(kThreads), 0, stream, p);
}

int take_gated_status(int* status) {
  *status = 0;
  if (!g_any.load(std::memory_order_relaxed)) return OZK_OK;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_gated_status, sizeof(int)) != cudaSuccess) return OZK_ERR_CUDA;
  if (v) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_gated_status, &zero, sizeof(int)) != cudaSuccess) return OZK_ERR_CUDA;
  }
  *status = v;
  return OZK_OK;
}

}  // namespace ozk
