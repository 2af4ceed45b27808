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
//
// Both ways are bound by HBM and, for 16-bit types, nearly as much by their
// instructions (about 150 per 512 elements and warp).  Measured on a GB300,
// 16384 x 8192: bf16 to NVFP4 58.6 us (5.9 TB/s; 51 at the measured 6.68), to
// MXFP4 56 us, fp32 88 us (6.9 TB/s), FP64 236 us (4.9 TB/s), back to bf16 59 us (5.9 TB/s), to FP64 225; rows that are only 4-byte
// aligned 81 us.  What counted: a lane's 32 bytes in one access
// (two of 16 touch every sector twice; dequantise 74 -> 59 us), the maximum two
// elements at a time and arithmetic on pairs, quotients without a division
// (66.5 -> 60.6 us with the loop unrolled), no search for a row's group where
// there are no offsets (-> 58.6).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "lowp.h"
#include "tc_ptx.cuh"

namespace ozk {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLaneElems = 16;                // elements a lane quantises at once
constexpr int kWarpElems = 32 * kLaneElems;   // columns a warp takes at once: a chunk of a row
constexpr int kMaxRun = 4;                    // chunks of one row a warp takes one after the other

struct Mx4Params {
  int64_t rows, K, ld;         // matrix and its leading dimension (elements)
  int64_t units;               // (row, run of chunks) pairs, a warp's work
  int kpad, kgroups, chunks;   // chunks of a row; kgroups: scale words (4 blocks) of a row
  int run, runs;               // chunks a unit takes; units of a row
  FastDiv div_runs;            // used while units < 2^31
  const int32_t* offsets;      // group starts (groups + 1), or null: groups of rows_per_group
  int groups;
  int64_t rows_per_group;
  float prescale;
  const void* x;
  void* out;                   // dequantise
  uint8_t* codes;
  uint8_t* scales;
};

// Row and first chunk of unit u.
__device__ __forceinline__ int64_t row_of(const Mx4Params& p, int64_t u, int* chunk) {
  if (p.units < (int64_t{1} << 31)) {
    const uint32_t row = div_fast(static_cast<uint32_t>(u), p.div_runs);
    *chunk = static_cast<int>(static_cast<uint32_t>(u) - row * static_cast<uint32_t>(p.runs)) * p.run;
    return row;
  }
  const int64_t row = u / p.runs;
  *chunk = static_cast<int>(u - row * p.runs) * p.run;
  return row;
}

// The groups' starts: up to kLaneGroups groups lie in the lanes of every warp,
// as they came; more in shared memory, cut so that they rise inside [0, rows].
// A product cuts bad offsets the same way, so codes, scales and products agree
// on the group of a row.  In lanes they cost no barrier and a row's search no
// memory: a row in 8 groups 2.3 us with every block checking them first, 1.8 so;
// 32 rows in 256 groups 2.7 us with a search in global memory, 2.4 so.
constexpr int kLaneGroups = 31;
struct Starts {
  int own;           // start of group `lane`, INT32_MAX past the last end
  bool raw;          // as it came, not yet cut
  const int* table;
};

template <bool RAGGED>
__device__ __forceinline__ Starts load_starts(const Mx4Params& p, int lane) {
  extern __shared__ int table[];
  if (!RAGGED) return {0, false, table};
  if (p.groups <= kLaneGroups) return {lane <= p.groups ? p.offsets[lane] : INT32_MAX, true, table};
  bool bad = false;
  for (int i = threadIdx.x; i <= p.groups; i += kThreads) {
    const int at = p.offsets[i], before = i ? p.offsets[i - 1] : 0;
    bad |= at < before || at > p.rows;
    table[i] = at;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      if (blockIdx.x == 0) atomicOr(&g_status, 2);
      int at = 0;
      for (int i = 0; i <= p.groups; ++i) table[i] = at = min(max(table[i], at), static_cast<int>(p.rows));
    }
    __syncthreads();
  }
  return {0, false, table};
}

// Cuts offsets that lie in lanes (the whole warp; at their first use, so that
// a row's elements are on their way before they are waited for), and reports
// bad ones, once a grid.
__device__ __forceinline__ void cut_starts(const Mx4Params& p, Starts& s, int lane) {
  s.raw = false;
  const int before = __shfl_up_sync(0xFFFFFFFFu, s.own, 1);
  const bool bad = lane <= p.groups && (s.own < (lane ? before : 0) || s.own > p.rows);
  if (!__any_sync(0xFFFFFFFFu, bad)) return;
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_status, 2);
  s.own = max(s.own, 0);
#pragma unroll
  for (int d = 1; d < 32; d *= 2) s.own = max(s.own, __shfl_up_sync(0xFFFFFFFFu, s.own, d));  // below d: their own
}

// Byte offset of the scale word (4 blocks) kg = 0 of `row`, or -1 for a row
// outside every group (the whole warp, on one row).
template <bool RAGGED>
__device__ __forceinline__ int64_t scale_row(const Mx4Params& p, Starts& s, int64_t row64, int lane) {
  const int row = static_cast<int>(row64);  // below 2^30
  int g = 0, o = 0;
  if (RAGGED && p.groups <= kLaneGroups) {
    if (s.raw) cut_starts(p, s, lane);
    g = __popc(__ballot_sync(0xFFFFFFFFu, s.own <= row)) - 1;  // a start past the rows is past this one
    if (g < 0 || g >= p.groups) return -1;
    o = __shfl_sync(0xFFFFFFFFu, s.own, g);
  } else if (RAGGED) {
    int lo = 0, hi = p.groups;  // the last group that starts at or before the row
    while (lo + 1 < hi) {
      const int mid = (lo + hi) / 2;
      if (s.table[mid] <= row) lo = mid;
      else hi = mid;
    }
    g = lo;
    o = s.table[lo];
    if (o > row || row >= s.table[lo + 1]) return -1;
  } else if (p.groups > 1) {
    const int per = static_cast<int>(p.rows_per_group);
    g = row / per;
    o = g * per;
  }
  const int r = row - o;
  return (static_cast<int64_t>((o >> 7) + g + (r >> 7)) * p.kgroups) * 512 + ((r & 31) << 4) + ((r >> 3) & 12);
}

// 16 elements of a row per lane, raw: lane l takes columns k0 + 16 l .. + 15,
// zeros past K.  Read as 32- or 16-byte words where base and row stride allow it;
// otherwise the warp reads its chunk in words of ALIGN bytes, neighbouring
// lanes neighbouring words, and turns it round in shared memory.
template <typename T>
struct Raw {
  static constexpr int kWords = kLaneElems * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
};

// Element i as fp32.
template <typename T>
__device__ __forceinline__ float element(const Raw<T>& r, int i) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    return __uint_as_float(i & 1 ? r.w[i / 2] & 0xFFFF0000u : r.w[i / 2] << 16);
  else if constexpr (std::is_same<T, __half>::value)
    return __half2float(__ushort_as_half(static_cast<unsigned short>(r.w[i / 2] >> (16 * (i & 1)))));
  else if constexpr (std::is_same<T, double>::value)
    return __double2float_rn(__hiloint2double(static_cast<int>(r.w[2 * i + 1]), static_cast<int>(r.w[2 * i])));
  else
    return __uint_as_float(r.w[i]);
}

// 32 bytes at once (32-byte aligned): a lane's whole sector in one access.
// Volatile and coherent, as are the other loads (plain ones, which no memory
// clobber lets over it): the kernel before this one may still be writing until
// the wait at the kernel's start is through.
__device__ __forceinline__ void load32(const void* src, uint32_t* d) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]), "=r"(d[7])
               : "l"(src));
}
__device__ __forceinline__ void store32(void* dst, const uint32_t* d) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(d[0]), "r"(d[1]), "r"(d[2]),
               "r"(d[3]), "r"(d[4]), "r"(d[5]), "r"(d[6]), "r"(d[7])
               : "memory");
}

// The word of a row that starts at element k (with sizeof(T) == 2: k and k + 1), zeros past K; word aligned.
template <typename T>
__device__ __forceinline__ uint32_t load_word(const T* row, int64_t k, int64_t K) {
  const uint16_t* h = reinterpret_cast<const uint16_t*>(row + k);
  return k + 1 < K ? *reinterpret_cast<const uint32_t*>(h) : k < K ? *h : 0u;
}

template <typename T, int ALIGN>
__device__ __forceinline__ void load_raw(const T* row, int k0, int64_t K, int lane, uint8_t* stage, Raw<T>& r) {
  constexpr int kWords = Raw<T>::kWords;
  if constexpr (ALIGN >= 16) {
    const int k = k0 + lane * kLaneElems;
    if (k + kLaneElems <= K) {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(row + k);
      if constexpr (ALIGN == 32) {
#pragma unroll
        for (int i = 0; i < kWords / 8; ++i) load32(src + 32 * i, r.w + 8 * i);
      } else {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const uint4 v = reinterpret_cast<const uint4*>(src)[i];
          r.w[4 * i] = v.x;
          r.w[4 * i + 1] = v.y;
          r.w[4 * i + 2] = v.z;
          r.w[4 * i + 3] = v.w;
        }
      }
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) r.w[i] = load_word(row, k + 2 * i, K);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        r.w[i] = k + i / (kWords / kLaneElems) < K ? reinterpret_cast<const uint32_t*>(row + k)[i] : 0u;
    }
  } else {
    if constexpr (ALIGN == 4 && sizeof(T) == 2) {
      uint32_t w[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = load_word(row, k0 + 2 * (32 * i + lane), K);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kWords; ++i) reinterpret_cast<uint32_t*>(stage)[32 * i + lane] = w[i];
    } else {
      T w[kLaneElems];
#pragma unroll
      for (int i = 0; i < kLaneElems; ++i) {
        const int64_t k = k0 + 32 * i + lane;
        w[i] = k < K ? row[k] : T(0.0f);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kLaneElems; ++i) reinterpret_cast<T*>(stage)[32 * i + lane] = w[i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(stage)[kWords / 4 * lane + i];
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
  }
}

// Largest magnitude of a lane's elements, times prescale, as fp32 bits: Inf
// and NaN compare above every finite value.  Rounding is monotone, so this is
// the largest |x'|.  16-bit types take the maximum of two elements at a time.
template <typename T>
__device__ __forceinline__ uint32_t top_of(const Raw<T>& r, float prescale) {
  float top;
  if constexpr (sizeof(T) == 2) {
    uint32_t m = r.w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < kLaneElems / 2; ++i) m = __vmaxu2(m, r.w[i] & 0x7FFF7FFFu);
    const uint32_t h = max(m & 0xFFFFu, m >> 16);
    if constexpr (std::is_same<T, __half>::value) top = __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
    else top = __uint_as_float(h << 16);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kLaneElems; ++i) m = max(m, __float_as_uint(element(r, i)) & 0x7FFFFFFFu);
    top = __uint_as_float(m);
  }
  return __float_as_uint(top * prescale) & 0x7FFFFFFFu;
}

template <typename T>
__device__ __forceinline__ void set_double(Raw<T>& r, int i, double v) {
  r.w[2 * i] = static_cast<uint32_t>(__double2loint(v));
  r.w[2 * i + 1] = static_cast<uint32_t>(__double2hiint(v));
}

// Elements 2 i and 2 i + 1 of a lane's 16, rounded to T.
template <typename T>
__device__ __forceinline__ void set_pair(Raw<T>& r, int i, float lo, float hi) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.w[i]) : "f"(hi), "f"(lo));
  } else if constexpr (std::is_same<T, __half>::value) {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r.w[i]) : "f"(hi), "f"(lo));
  } else if constexpr (std::is_same<T, double>::value) {
    set_double(r, 2 * i, lo);
    set_double(r, 2 * i + 1, hi);
  } else {
    r.w[2 * i] = __float_as_uint(lo);
    r.w[2 * i + 1] = __float_as_uint(hi);
  }
}
template <typename T>
__device__ __forceinline__ void store_element(T* dst, const Raw<T>& r, int i) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(r.w[i / 2] >> (16 * (i & 1)));
  } else {
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(T)) / 4; ++j)
      reinterpret_cast<uint32_t*>(dst)[j] = r.w[i * (static_cast<int>(sizeof(T)) / 4) + j];
  }
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Codes of eight values (four pairs), the first in the low half of the low byte.
__device__ __forceinline__ uint32_t codes8(const uint64_t* q) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .f32 l, h;\n\t"
      "mov.b64 {l, h}, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b0, h, l;\n\t"
      "mov.b64 {l, h}, %2;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, h, l;\n\t"
      "mov.b64 {l, h}, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 b2, h, l;\n\t"
      "mov.b64 {l, h}, %4;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, h, l;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "l"(q[0]), "l"(q[1]), "l"(q[2]), "l"(q[3]));
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

// v / s from an approximate reciprocal and one residual step (Markstein 1990):
// within a little over half an ulp.  What the rounding to few bits after it
// needs is that a tie, v = t s with t a boundary between codes (t s has at
// most 7 bits), comes out as t exactly, which the residual makes it, and that
// no other fp32 v does: its quotient is at least 2^-23 / m of t away, m < 2 the
// mantissa of t s, more than half an ulp of t by a margin of 2^-7 of it.
__device__ __forceinline__ float quotient(float v, float s, float inv) {
  const float q = v * inv;
  return fmaf(fmaf(-q, s, v), inv, q);
}
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// Quantises one lane's 16 elements at column k and stores codes and scales.
template <typename T, int FMT>
__device__ __forceinline__ void quantize16(const Mx4Params& p, const Raw<T>& r, int64_t row, int k, int64_t at, int lane) {
  uint32_t top = top_of(r, p.prescale);
  if (FMT == OZK_MXFP4) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  uint64_t v[kLaneElems / 2];
#pragma unroll
  for (int i = 0; i < kLaneElems / 2; ++i) v[i] = pack2(element(r, 2 * i), element(r, 2 * i + 1));
  if (p.prescale != 1.0f) {
    const uint64_t ps = pack2(p.prescale, p.prescale);
#pragma unroll
    for (int i = 0; i < kLaneElems / 2; ++i) v[i] = mul2(v[i], ps);
  }
  uint32_t byte, lo = 0, hi = 0;
  if (FMT == OZK_MXFP4) {
    byte = static_cast<uint32_t>(max(static_cast<int>(top >> 23) - 2, 0));
    const float f = __uint_as_float((254u - byte) << 23);
    const uint64_t inv = pack2(f, f);  // 1 / s, exact
#pragma unroll
    for (int i = 0; i < kLaneElems / 2; ++i) v[i] = mul2(v[i], inv);
  } else {
    byte = e4m3_of(quotient(__uint_as_float(top), 6.0f, 1.0f / 6.0f));
    const float s = e4m3_value(byte);
    const float f = byte ? reciprocal(s) : 0.0f;
    const uint64_t inv = pack2(f, f), neg = pack2(-s, -s);
#pragma unroll
    for (int i = 0; i < kLaneElems / 2; ++i) {
      const uint64_t q = mul2(v[i], inv);  // quotient(), two at a time
      v[i] = fma2(fma2(q, neg, v[i]), inv, q);
    }
  }
  if (top < 0x7F800000u) {
    lo = codes8(v);
    hi = codes8(v + 4);
  } else {
    byte = FMT == OZK_MXFP4 ? 0xFFu : 0x7Fu;
  }
  if (k < p.kpad) *reinterpret_cast<uint2*>(p.codes + row * (p.kpad / 2) + k / 2) = make_uint2(lo, hi);
  // four scale bytes to a word: of 4 lanes (nvfp4), of lanes 0, 2, 4, 6 of 8 (mxfp4)
  constexpr int step = FMT == OZK_MXFP4 ? 2 : 1;
  uint32_t word = byte << (8 * ((lane / step) & 3));
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, step);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * step);
  const int kg = k / (64 * step);
  if (lane % (4 * step) == 0 && kg < p.kgroups)
    *reinterpret_cast<uint32_t*>(p.scales + at + static_cast<int64_t>(kg) * 512) = word;
}

template <typename T, int FMT, int ALIGN, bool RAGGED>
__global__ void __launch_bounds__(kThreads, sizeof(T) > 4 ? 2 : 4) mx4_quantize_kernel(const Mx4Params p) {
  grid_dependency_sync();
  __shared__ alignas(16) uint8_t stages[ALIGN >= 16 ? 16 : kWarps * kWarpElems * sizeof(T)];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* stage = ALIGN >= 16 ? stages : stages + warp * kWarpElems * sizeof(T);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
  Starts starts = load_starts<RAGGED>(p, lane);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < p.units; u += warps) {
    int c;
    const int64_t row = row_of(p, u, &c);
    const T* src = static_cast<const T*>(p.x) + row * p.ld;
    const int c1 = min(c + p.run, p.chunks);
    Raw<T> r;
    load_raw<T, ALIGN>(src, c * kWarpElems, p.K, lane, stage, r);
    const int64_t at = scale_row<RAGGED>(p, starts, row, lane);
    if (at < 0) continue;
#pragma unroll 2
    for (;;) {  // the next chunk is on its way while this one is quantised
      Raw<T> next;
      if (c + 1 < c1) load_raw<T, ALIGN>(src, (c + 1) * kWarpElems, p.K, lane, stage, next);
      quantize16<T, FMT>(p, r, row, c * kWarpElems + lane * kLaneElems, at, lane);
      if (++c >= c1) break;
      r = next;
    }
  }
}

// The E2M1 values of codes 2 i and 2 i + 1 of a lane's 16.
__device__ __forceinline__ float2 code_pair(uint2 code, int i) {
  uint32_t h;
  const uint32_t two = ((i < 4 ? code.x : code.y) >> (8 * (i & 3))) & 0xFFu;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The values 16 codes stand for: the E2M1 value, exact in fp16, times the
// scale (at most 6 significant bits; a NaN scale gives NaN).  The product is
// exact in fp32 but for scales from 2^126, where it can pass fp32's range; for
// FP64, which holds it, such a product is done again in FP64 (for every scale it
// would take 281 us for 16384 x 8192, 226 so).
// Blocks of an SM: as many as the registers of a lane's 16 elements leave room for.
constexpr int dequantize_blocks(int size, int align) {
  return size > 4 ? 3 : size == 4 ? (align == 16 ? 5 : 4) : align == 32 ? 4 : align == 2 ? 5 : 6;
}

template <typename T, int FMT, int ALIGN, bool RAGGED>
__global__ void __launch_bounds__(kThreads, dequantize_blocks(sizeof(T), ALIGN)) mx4_dequantize_kernel(const Mx4Params p) {
  grid_dependency_sync();
  __shared__ alignas(16) uint8_t stages[ALIGN >= 16 ? 16 : kWarps * kWarpElems * sizeof(T)];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T* stage = reinterpret_cast<T*>(ALIGN >= 16 ? stages : stages + warp * kWarpElems * sizeof(T));
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
  Starts starts = load_starts<RAGGED>(p, lane);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < p.units; u += warps) {
    int c;
    const int64_t row = row_of(p, u, &c);
    const int64_t at = scale_row<RAGGED>(p, starts, row, lane);
    if (at < 0) continue;
    const int c1 = min(c + p.run, p.chunks);
    const uint8_t* codes = p.codes + row * (p.kpad / 2);
    T* dst = static_cast<T*>(p.out) + row * p.ld;
    uint2 run_codes[kMaxRun];  // all of the unit's loads at once
    uint32_t run_bytes[kMaxRun];
#pragma unroll
    for (int i = 0; i < kMaxRun; ++i) {
      const int k = (c + i) * kWarpElems + lane * kLaneElems;
      run_codes[i] = make_uint2(0, 0);
      run_bytes[i] = 0;
      if (c + i < c1 && k < p.K) {
        run_codes[i] = *reinterpret_cast<const uint2*>(codes + k / 2);
        const int b = k / (FMT == OZK_MXFP4 ? 32 : 16);
        run_bytes[i] = p.scales[at + static_cast<int64_t>(b / 4) * 512 + b % 4];
      }
    }
#pragma unroll
    for (int j = 0; j < kMaxRun; ++j, ++c) {
      if (c >= c1) break;
      const int k = c * kWarpElems + lane * kLaneElems;
      const uint2 code = run_codes[j];
      const uint32_t byte = run_bytes[j];
      float s;
      if (FMT == OZK_MXFP4)
        s = byte == 0xFFu ? __uint_as_float(0x7FC00000u) : byte ? __uint_as_float(byte << 23) : __uint_as_float(1u << 22);
      else
        s = e4m3_value(byte);
      Raw<T> r;
#pragma unroll
      for (int i = 0; i < kLaneElems / 2; ++i) {
        const float2 f = code_pair(code, i);
        set_pair(r, i, f.x * s, f.y * s);
      }
      if constexpr (sizeof(T) == 8 && FMT == OZK_MXFP4) {
        if (byte >= 253u && byte != 0xFFu) {
#pragma unroll
          for (int i = 0; i < kLaneElems / 2; ++i) {
            const float2 f = code_pair(code, i);
            set_double(r, 2 * i, static_cast<double>(f.x) * s);
            set_double(r, 2 * i + 1, static_cast<double>(f.y) * s);
          }
        }
      }
      constexpr int kWords = Raw<T>::kWords;
      if (ALIGN == 32 && k + kLaneElems <= p.K) {
#pragma unroll
        for (int i = 0; i < kWords / 8; ++i) store32(reinterpret_cast<uint8_t*>(dst + k) + 32 * i, r.w + 8 * i);
      } else if (ALIGN == 16 && k + kLaneElems <= p.K) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i)
          reinterpret_cast<uint4*>(dst + k)[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
      } else if (ALIGN >= 16) {
#pragma unroll
        for (int i = 0; i < kLaneElems; ++i)
          if (k + i < p.K) store_element(dst + k + i, r, i);
      } else {  // turned round in shared memory: neighbouring lanes write neighbouring words
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i)
          reinterpret_cast<uint4*>(stage)[kWords / 4 * lane + i] =
              make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
        __syncwarp();
        const int64_t k0 = static_cast<int64_t>(c) * kWarpElems;
        if constexpr (ALIGN == 4 && sizeof(T) == 2) {
#pragma unroll
          for (int i = 0; i < kLaneElems / 2; ++i) {
            const int64_t at2 = k0 + 2 * (32 * i + lane);
            const uint32_t w = reinterpret_cast<const uint32_t*>(stage)[32 * i + lane];
            if (at2 + 1 < p.K) reinterpret_cast<uint32_t*>(dst)[at2 / 2] = w;
            else if (at2 < p.K) *reinterpret_cast<uint16_t*>(dst + at2) = static_cast<uint16_t>(w);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kLaneElems; ++i)
            if (k0 + 32 * i + lane < p.K) dst[k0 + 32 * i + lane] = stage[32 * i + lane];
        }
      }
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

// Warps that keep the memory busy: units of one chunk until every SM has
// kFullWarps of them, then runs of up to kMaxRun chunks, which share the row's
// addressing and have the next chunk's loads in flight.
constexpr int kFullWarps = 48;

Mx4Params make_params(const Mx4Matrix& m, int64_t ld, int num_sms) {
  Mx4Params p = {};
  p.rows = m.rows;
  p.K = m.K;
  p.ld = ld;
  p.kpad = static_cast<int>(ozk_kpad(m.K));
  p.kgroups = mx4_kgroups(m.K, m.format);
  // enough chunks for the codes and the scale words (a word covers 64 or 128 columns)
  p.chunks = (p.kgroups * (m.format == OZK_MXFP4 ? 128 : 64) + kWarpElems - 1) / kWarpElems;
  const int64_t per_warp = m.rows * p.chunks / (static_cast<int64_t>(num_sms) * kFullWarps);
  p.run = static_cast<int>(std::min<int64_t>(std::min<int64_t>(kMaxRun, p.chunks), std::max<int64_t>(per_warp, 1)));
  p.runs = (p.chunks + p.run - 1) / p.run;
  p.units = m.rows * p.runs;
  p.div_runs = fast_div(p.runs);
  p.offsets = m.offsets;
  p.groups = m.groups;
  p.rows_per_group = std::max<int64_t>(m.rows / m.groups, 1);
  p.codes = m.codes;
  p.scales = m.scales;
  return p;
}

unsigned grid_of(int64_t units, int num_sms) {
  return static_cast<unsigned>(std::min<int64_t>((units + kWarps - 1) / kWarps, static_cast<int64_t>(num_sms) * 8));
}

size_t starts_bytes(const Mx4Matrix& m) {
  return m.offsets != nullptr && m.groups > kLaneGroups ? (static_cast<size_t>(m.groups) + 1) * sizeof(int) : 0;
}

// The widest word every row's first element is aligned to: 32, 16, 4 or 2 bytes.
int alignment(const void* x, int64_t ld, int dtype) {
  const size_t a = reinterpret_cast<uintptr_t>(x) | (static_cast<size_t>(ld) * type_bytes(dtype));
  return a % 32 == 0 ? 32 : a % 16 == 0 ? 16 : a % 4 == 0 ? 4 : 2;
}

// f(element type, format, alignment, ragged groups) with constants.  A matrix
// without offsets has kernels without the search for a row's group (1537 x 2090
// fp16 to MXFP4 3.70 us, 3.82 with it).
template <typename F>
cudaError_t dispatch(int dtype, int format, int align, bool ragged, F&& f) {
  return pick_type(dtype, [&](auto t) {
    using T = decltype(t);
    auto aligned = [&](auto fmt, auto a) {
      return ragged ? f(t, fmt, a, std::true_type{}) : f(t, fmt, a, std::false_type{});
    };
    auto with = [&](auto fmt) {
      if (align == 32) return aligned(fmt, std::integral_constant<int, 32>{});
      if (align == 16) return aligned(fmt, std::integral_constant<int, 16>{});
      if (align == 4 || sizeof(T) > 2) return aligned(fmt, std::integral_constant<int, 4>{});
      return aligned(fmt, std::integral_constant<int, sizeof(T) == 2 ? 2 : 4>{});
    };
    return format == OZK_MXFP4 ? with(std::integral_constant<int, OZK_MXFP4>{})
                               : with(std::integral_constant<int, OZK_NVFP4>{});
  });
}

std::atomic<bool> g_with_offsets{false};  // launched yet: without, there is no status to read

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4Matrix& m, const void* x, int64_t ldx, int dtype, float prescale,
                                int num_sms, cudaStream_t stream) {
  if (m.offsets != nullptr) g_with_offsets.store(true, std::memory_order_relaxed);
  Mx4Params p = make_params(m, ldx, num_sms);
  p.x = x;
  p.prescale = prescale;
  const bool groups = m.offsets != nullptr;
  return dispatch(dtype, m.format, alignment(x, ldx, dtype), groups, [&](auto t, auto fmt, auto align, auto ragged) {
    return launch_dependent(mx4_quantize_kernel<decltype(t), fmt.value, align.value, ragged.value>,
                            dim3(grid_of(p.units, num_sms)), dim3(kThreads), starts_bytes(m), stream, p);
  });
}

cudaError_t launch_mx4_dequantize(const Mx4Matrix& m, void* out, int64_t ldo, int dtype, int num_sms,
                                  cudaStream_t stream) {
  if (m.offsets != nullptr) g_with_offsets.store(true, std::memory_order_relaxed);
  Mx4Params p = make_params(m, ldo, num_sms);
  p.out = out;
  const bool groups = m.offsets != nullptr;
  return dispatch(dtype, m.format, alignment(out, ldo, dtype), groups, [&](auto t, auto fmt, auto align, auto ragged) {
    return launch_dependent(mx4_dequantize_kernel<decltype(t), fmt.value, align.value, ragged.value>,
                            dim3(grid_of(p.units, num_sms)), dim3(kThreads), starts_bytes(m), stream, p);
  });
}

int take_mx4_status(int* status) {
  *status = 0;
  return g_with_offsets.load(std::memory_order_relaxed) ? take_status(status) : OZK_OK;
}

}  // namespace ozk
