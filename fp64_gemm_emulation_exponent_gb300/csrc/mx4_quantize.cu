// Microscaled 4-bit floating point: quantisation of rows and its inverse.
//
// A row is cut into blocks (16 elements for nvfp4, 32 for mxfp4); a block is
// stored as E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign) and one scale
// byte.  With x' = x * prescale rounded once to fp32 and amax = max |x'| over
// the block:
//   nvfp4  s = amax / 6 rounded to E4M3 (nearest even, at most 448);
//   mxfp4  s = 2^(floor(log2 amax) - 2), exponent limited to [-127, 127];
//   code = x' / s rounded to E2M1 (nearest, ties to the even code, at most 6).
// A block whose scale is 0 (amax = 0, or amax/6 below half of 2^-9) stands
// for zeros; one that holds an Inf or NaN gets the format's NaN scale.
//
// Storage: codes are kpad / 2 bytes a row (kpad = K rounded up to 64, element
// 2i in the low half of byte i, zeros past K).  Scale bytes are laid out as
// the tensor cores take them: 512-byte tiles of 128 rows x 4 blocks, row r of
// a tile at 16 (r % 32) + 4 (r / 32 % 4), tiles of one row block contiguous
// along K.  Group g, starting at row o_g, has its first row block at
// o_g / 128 + g: each group starts a tile of its own, the start follows from
// o_g alone, and o_g+1 / 128 + g + 1 is never below the end of group g.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "lowp.h"

namespace ozk {
namespace {

constexpr int kThreads = 256;
constexpr int kLaneElems = 16;                // elements a lane quantises at once
constexpr int kWarpElems = 32 * kLaneElems;   // of one row

struct Mx4Params {
  int64_t rows, K, ld;         // matrix and its leading dimension (elements)
  int64_t units;               // (row, 512-column chunk) pairs
  int kpad, kgroups, chunks;   // kgroups: scale words (4 blocks) per row
  FastDiv div_chunks;
  const int32_t* offsets;      // group starts (groups + 1), or null: groups of rows_per_group
  int groups;
  int64_t rows_per_group;
  float prescale;
  const void* x;
  void* out;                   // dequantise
  uint8_t* codes;
  uint8_t* scales;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __bfloat162float(v);
  else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
  else if constexpr (std::is_same<T, double>::value) return __double2float_rn(v);
  else return v;
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __float2bfloat16_rn(v);
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
  else if constexpr (std::is_same<T, double>::value) return static_cast<double>(v);
  else return v;
}

// Byte offset of the scale word (4 blocks) kg = 0 of `row`, or -1 for a row
// outside every group.  Groups that overlap or run backwards cannot take it
// out of the buffer: o_g <= row gives a row block of at most row / 128 + g.
__device__ __forceinline__ int64_t scale_row(const Mx4Params& p, int64_t row) {
  int64_t g, o;
  if (p.offsets == nullptr) {
    g = p.groups == 1 ? 0 : row / p.rows_per_group;
    o = g * p.rows_per_group;
  } else {
    int lo = 0, hi = p.groups;  // the last group that starts at or before the row
    while (lo + 1 < hi) {
      const int mid = (lo + hi) / 2;
      if (p.offsets[mid] <= row) lo = mid;
      else hi = mid;
    }
    g = lo;
    o = p.offsets[lo];
    if (o < 0 || o > row || row >= p.offsets[lo + 1]) return -1;
  }
  const int64_t r = row - o;
  return (o / 128 + g + r / 128) * p.kgroups * 512 + (r % 32) * 16 + (r / 32 % 4) * 4;
}

// 16 elements k0.. of a row as fp32, zeros past K.
template <typename T, bool VEC>
__device__ __forceinline__ void load16(const T* row, int64_t k0, int64_t K, float (&v)[kLaneElems]) {
  if (VEC && k0 + kLaneElems <= K) {
    constexpr int per = 16 / sizeof(T);
    uint4 raw[kLaneElems / per];
#pragma unroll
    for (int i = 0; i < kLaneElems / per; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(row + k0) + i);
    const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
    for (int i = 0; i < kLaneElems; ++i) v[i] = to_f32(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kLaneElems; ++i) v[i] = k0 + i < K ? to_f32(row[k0 + i]) : 0.0f;
  }
}

// Codes of eight values, the first in the low half of the low byte.
__device__ __forceinline__ uint32_t codes8(const float* q) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

// E4M3 byte of v >= 0 (nearest even, at most 448), and the value of a byte.
__device__ __forceinline__ uint32_t e4m3_of(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kThreads) mx4_quantize_kernel(const Mx4Params p) {
  grid_dependency_sync();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); u < p.units; u += warps) {
    const int64_t row = u / p.chunks;
    const int chunk = static_cast<int>(u - row * p.chunks);
    const int64_t at = scale_row(p, row);
    if (at < 0) continue;
    const int k0 = chunk * kWarpElems + lane * kLaneElems;
    float v[kLaneElems];
    load16<T, VEC>(static_cast<const T*>(p.x) + row * p.ld, k0, p.K, v);
    uint32_t top = 0;  // largest |x'| as bits: Inf and NaN compare above every finite value
#pragma unroll
    for (int i = 0; i < kLaneElems; ++i) {
      v[i] *= p.prescale;
      top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    if (FMT == OZK_MXFP4) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    const bool finite = top < 0x7F800000u;
    uint32_t byte, lo = 0, hi = 0;
    if (FMT == OZK_MXFP4) {
      const int e = static_cast<int>(top >> 23) - 2;
      byte = static_cast<uint32_t>(max(e, 0));
      const float inv = __uint_as_float((254u - byte) << 23);  // exact: 1 / s
#pragma unroll
      for (int i = 0; i < kLaneElems; ++i) v[i] *= inv;
    } else {
      byte = e4m3_of(__fdiv_rn(__uint_as_float(top), 6.0f));
      const float s = e4m3_value(byte);
      const float inv = byte ? __frcp_rn(s) : 0.0f;
      // x' / s correctly rounded (Markstein's residual step from the rounded
      // reciprocal): the ties of the E2M1 rounding, multiples t s with few
      // bits, come out exactly, and nothing else rounds onto them
#pragma unroll
      for (int i = 0; i < kLaneElems; ++i) {
        const float q = v[i] * inv;
        v[i] = fmaf(fmaf(-q, s, v[i]), inv, q);
      }
    }
    if (finite) {
      lo = codes8(v);
      hi = codes8(v + 8);
    } else {
      byte = FMT == OZK_MXFP4 ? 0xFFu : 0x7Fu;
    }
    if (k0 < p.kpad)
      *reinterpret_cast<uint2*>(p.codes + row * (p.kpad / 2) + k0 / 2) = make_uint2(lo, hi);
    // four scale bytes to a word: of 4 lanes (nvfp4), of lanes 0, 2, 4, 6 of 8 (mxfp4)
    constexpr int step = FMT == OZK_MXFP4 ? 2 : 1;
    uint32_t word = byte << (8 * ((lane / step) & 3));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, step);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * step);
    const int kg = k0 / (64 * step);
    if (lane % (4 * step) == 0 && kg < p.kgroups)
      *reinterpret_cast<uint32_t*>(p.scales + at + static_cast<int64_t>(kg) * 512) = word;
  }
}

// The values 16 codes stand for: the E2M1 value, exact in fp16, times the
// scale (at most 6 significant bits, exact in fp32; a NaN scale gives NaN).
template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kThreads) mx4_dequantize_kernel(const Mx4Params p) {
  grid_dependency_sync();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); u < p.units; u += warps) {
    const int64_t row = u / p.chunks;
    const int k0 = static_cast<int>(u - row * p.chunks) * kWarpElems + lane * kLaneElems;
    const int64_t at = scale_row(p, row);
    if (at < 0 || k0 >= p.K) continue;
    const uint2 c = *reinterpret_cast<const uint2*>(p.codes + row * (p.kpad / 2) + k0 / 2);
    constexpr int block = FMT == OZK_MXFP4 ? 32 : 16;
    const int b = k0 / block;
    const uint32_t byte = p.scales[at + static_cast<int64_t>(b / 4) * 512 + b % 4];
    float s;
    if (FMT == OZK_MXFP4)
      s = byte == 0xFFu ? __uint_as_float(0x7FC00000u) : byte ? __uint_as_float(byte << 23) : __uint_as_float(1u << 22);
    else
      s = e4m3_value(byte);
    T v[kLaneElems];
#pragma unroll
    for (int i = 0; i < kLaneElems / 2; ++i) {
      uint32_t h;
      const uint32_t two = ((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFFu;
      asm("{\n\t.reg .b8 b, z;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(two));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * i] = from_f32<T>(f.x * s);
      v[2 * i + 1] = from_f32<T>(f.y * s);
    }
    T* dst = static_cast<T*>(p.out) + row * p.ld + k0;
    if (VEC && k0 + kLaneElems <= p.K) {
#pragma unroll
      for (int i = 0; i < kLaneElems * static_cast<int>(sizeof(T)) / 16; ++i)
        reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(v)[i];
    } else {
#pragma unroll
      for (int i = 0; i < kLaneElems; ++i)
        if (k0 + i < p.K) dst[i] = v[i];
    }
  }
}

template <typename F>
auto pick_type(int dtype, F&& f) {
  switch (dtype) {
    case OZK_BF16: return f(__nv_bfloat16{});
    case OZK_F16: return f(__half{});
    case OZK_F64: return f(double{});
    default: return f(float{});
  }
}

size_t type_bytes(int dtype) { return dtype == OZK_F64 ? 8 : dtype == OZK_F32 ? 4 : 2; }

Mx4Params make_params(const Mx4Matrix& m, int64_t ld) {
  Mx4Params p = {};
  p.rows = m.rows;
  p.K = m.K;
  p.ld = ld;
  p.kpad = static_cast<int>(ozk_kpad(m.K));
  p.kgroups = mx4_kgroups(m.K, m.format);
  // enough 512-column chunks for the codes and the scale words (a word covers 64 or 128 columns)
  p.chunks = (p.kgroups * (m.format == OZK_MXFP4 ? 128 : 64) + kWarpElems - 1) / kWarpElems;
  p.units = m.rows * p.chunks;
  p.offsets = m.offsets;
  p.groups = m.groups;
  p.rows_per_group = m.groups > 0 ? std::max<int64_t>(m.rows / m.groups, 1) : 1;
  p.codes = m.codes;
  p.scales = m.scales;
  return p;
}

unsigned grid_of(int64_t units, int num_sms) {
  const int64_t blocks = (units + kThreads / 32 - 1) / (kThreads / 32);
  return static_cast<unsigned>(std::min<int64_t>(blocks, static_cast<int64_t>(num_sms) * 8));
}

bool vec_ok(const void* x, int64_t ld, int dtype) {
  return reinterpret_cast<uintptr_t>(x) % 16 == 0 && (static_cast<size_t>(ld) * type_bytes(dtype)) % 16 == 0;
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4Matrix& m, const void* x, int64_t ldx, int dtype, float prescale,
                                int num_sms, cudaStream_t stream) {
  Mx4Params p = make_params(m, ldx);
  p.x = x;
  p.prescale = prescale;
  const bool vec = vec_ok(x, ldx, dtype);
  return pick_type(dtype, [&](auto t) {
    using T = decltype(t);
    auto k = m.format == OZK_MXFP4 ? (vec ? mx4_quantize_kernel<T, OZK_MXFP4, true> : mx4_quantize_kernel<T, OZK_MXFP4, false>)
                                   : (vec ? mx4_quantize_kernel<T, OZK_NVFP4, true> : mx4_quantize_kernel<T, OZK_NVFP4, false>);
    return launch_dependent(k, dim3(grid_of(p.units, num_sms)), dim3(kThreads), 0, stream, p);
  });
}

cudaError_t launch_mx4_dequantize(const Mx4Matrix& m, void* out, int64_t ldo, int dtype, int num_sms,
                                  cudaStream_t stream) {
  Mx4Params p = make_params(m, ldo);
  p.out = out;
  const bool vec = vec_ok(out, ldo, dtype);
  return pick_type(dtype, [&](auto t) {
    using T = decltype(t);
    auto k = m.format == OZK_MXFP4
                 ? (vec ? mx4_dequantize_kernel<T, OZK_MXFP4, true> : mx4_dequantize_kernel<T, OZK_MXFP4, false>)
                 : (vec ? mx4_dequantize_kernel<T, OZK_NVFP4, true> : mx4_dequantize_kernel<T, OZK_NVFP4, false>);
    return launch_dependent(k, dim3(grid_of(p.units, num_sms)), dim3(kThreads), 0, stream, p);
  });
}

}  // namespace ozk
