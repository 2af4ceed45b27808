// Products of a few 16-bit rows with microscaled 4-bit weights:
//   y[t, n] = alpha sum_k x[t, k] w[g(t)][n, k], and its gated form
//   h[t, n] = act(alpha sum_k x[t, k] w[g][n, k]) (alpha sum_k x[t, k] w[g][H + n, k]).
//
// What bounds them is reading the weights once: N K (1/2 + 1/block) bytes,
// 42 weights a cycle and SM at the measured 6.8 TB/s, so the work on a weight
// between memory and its product is kept below 4 x 512 weights in 48 cycles:
//   - E2M1 codes become fp16 pairs by one conversion a byte (64 lanes a cycle
//     and SM); as fp16 they are exact, and so are NVFP4 codes times their
//     E4M3 scale (6 significant bits).  MXFP4 scales reach past fp16, and
//     multiply the fp32 sums of their blocks.
//   - The products run on the tensor cores as m16n8k16 with the weights on the
//     16-row side, 8 rows of x on the other (mma.sync: 8 cycles of a quarter
//     of an SM for 256 weights; tcgen05 would want the converted weights
//     written back to shared memory first).
//   - Sums over K are free in order, so lane q of a row takes the 8 weights of
//     the 4 bytes that ldmatrix hands it out of 16 (32 weights), as terms 2 q,
//     2 q + 1, 2 q + 8, 2 q + 9 of two steps, and the rows of x are read in
//     the same order.
// Rows of bf16 x do not fit fp16 as they are.  A panel (some columns of a
// row) is scaled by a power of two that brings its largest element to
// [2^15, 2^16): exact for every element down to 2^-32 of the largest.  Where a
// panel holds smaller ones, they take part in a further run over the weights,
// scaled by 2^33 more, and so on (at most 8 runs); activations all but never
// have them.
//
// A block owns 16 R output rows of w (gated: 8 R of each projection) and all
// of K; its warps take the chunks of 128 columns in turn, each through a ring
// of its own in shared memory filled by asynchronous copies, and the warps'
// sums are added at the end in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <map>
#include <mutex>

#include "activation.cuh"
#include "lowp.h"

namespace ozk {
namespace {

__device__ int g_gemv_status;  // bit 1: bad group offsets

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 128;              // columns of a chunk: 64 bytes of codes a row
constexpr int kRange = 33;               // binades of a panel's elements that one run takes
constexpr int kMxShift = 22;             // MXFP4 sums are formed 2^-22 smaller: s 2^-22 stays below overflow

template <int FMT, int R, int NT>
struct Shape {
  static constexpr bool NV = FMT == OZK_NVFP4;
  static constexpr int WORDS = NV ? 2 : 1;                       // scale words of a row and chunk
  static constexpr int CODES = R * 1024;                         // bytes of a chunk
  static constexpr int STAGE = CODES + R * 16 * WORDS * 4;
  static constexpr int DEPTH = R == 4 ? 3 : 4;
  static constexpr int TOKENS = 8 * NT;
  static constexpr int PANEL = 4096 / NT;                        // columns of x that are staged at a time
  static constexpr int PITCH = PANEL * 2 + 64;                   // most bytes of a staged row: see pitch
  static constexpr int RING = kWarps * DEPTH * STAGE;
  static_assert(kWarps * R * NT * 4 * 32 * 4 <= RING, "the warps' sums take the ring's place");
  static_assert(PANEL % (kChunk * kWarps) == 0, "every warp has as many chunks of a panel");
};

struct GemvParams {
  int T, N, K, groups;     // N: output columns
  int w_rows;              // rows of w per group: N, gated 2 N
  int kpad, words;         // columns of the codes; scale words of a row
  const int32_t* offsets;  // null: one group of T rows
  const uint8_t* codes;
  const uint8_t* scales;
  const uint16_t* x;
  int64_t ldx;
  void* y;
  int64_t ldy;
  int out_type;
  float alpha;
  int act;                 // gated only
  bool vec;                // rows of x start on 16 bytes
  int pitch;               // bytes of a staged row of x: 64 more than a multiple of 128, so that rows alternate in banks
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// 16 or 4 bytes to shared memory, zeros where !valid.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Eight codes as four fp16 pairs, in order.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Byte `sel` of a word of E4M3 scales as an fp16 pair.
__device__ __forceinline__ uint32_t scale_half2(uint32_t word, uint32_t sel) {
  const uint32_t both = __byte_perm(word, 0, sel * 0x11u);
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(both)));
  return r;
}
// 2^(b - 127 - kMxShift) of byte `i` of a word of E8M0 scales; 255 is NaN.
__device__ __forceinline__ float scale_mx(uint32_t word, int i) {
  const uint32_t b = (word >> (8 * i)) & 0xFFu;
  // in two exact steps: 2^(b - 127) is subnormal for b = 0, and small ones stay exact down to 2^-149
  const float s = __uint_as_float(b == 255u ? 0x7FC00000u : b == 0u ? 0x00400000u : b << 23);
  return s * (1.0f / (1 << kMxShift));
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Group `rank` of those that have rows: its number, first row and rows; rows
// is 0 where there are fewer.  Offsets are cut to a rising sequence inside
// [0, T] by a running maximum, and reported by the caller where that changed
// any.  Every warp finds it by itself.
struct Found {
  int e, row0, rows;
  bool bad;
};
__device__ __forceinline__ Found find_group(const GemvParams& p, int rank) {
  const int lane = threadIdx.x & 31;
  Found f{0, 0, 0, false};
  int seen = 0, before = 0;  // groups with rows so far; the end of the last one looked at
  {
    const int first = p.offsets[0];
    before = min(max(first, 0), p.T);
    f.bad = before != first;
  }
  for (int b = 0; b < p.groups; b += 32) {
    const int e = b + lane;
    const bool in = e < p.groups;
    const int end = in ? p.offsets[e + 1] : 0;
    int cut = in ? min(max(end, 0), p.T) : 0;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, cut, d);
      if (lane >= d) cut = max(cut, v);
    }
    cut = max(cut, before);
    if (in && cut != end) f.bad = true;
    const int up = __shfl_up_sync(0xFFFFFFFFu, cut, 1);
    const int start = lane ? up : before;
    const bool has = in && cut > start;
    const uint32_t with = __ballot_sync(0xFFFFFFFFu, has);
    const uint32_t here = __ballot_sync(0xFFFFFFFFu, has && seen + __popc(with & ((1u << lane) - 1u)) == rank);
    if (here) {
      const int src = __ffs(here) - 1;
      f.e = b + src;
      f.row0 = __shfl_sync(0xFFFFFFFFu, start, src);
      f.rows = __shfl_sync(0xFFFFFFFFu, cut, src) - f.row0;
    }
    seen += __popc(with);
    before = __shfl_sync(0xFFFFFFFFu, cut, 31);
  }
  f.bad = __any_sync(0xFFFFFFFFu, f.bad);
  return f;
}

// Elements [k, k + 8) of a row of x as stored, zeros from K on.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int k, int K, bool vec) {
  if (vec && k + 8 <= K) {
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(row + k) : "memory");
    return v;
  }
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = k + i < K ? row[k + i] : 0u;
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

__device__ __forceinline__ float pow2f(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// v 2^e for e beyond the exponents of one factor.
__device__ __forceinline__ float scaled(float v, int e) {
  const int half = e / 2;
  return v * pow2f(half) * pow2f(e - half);
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int FMT, int R, int NT, bool GATED, bool BF>
__global__ void __launch_bounds__(kThreads) gemv_kernel(const GemvParams p) {
  using S = Shape<FMT, R, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_max[S::TOKENS], s_min[S::TOKENS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_sync();

  int e = 0, row0 = 0, rows = p.T;
  if (p.offsets) {
    const Found f = find_group(p, blockIdx.y);
    if (f.bad && blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) atomicOr(&g_gemv_status, 2);
    e = f.e;
    row0 = f.row0;
    rows = f.rows;
    if (rows == 0) return;
  }

  // This block's rows of w: row r of tile i, rows past the last one doubled.
  constexpr int kOut = GATED ? 8 : 16;  // output columns of a tile
  const int n0 = blockIdx.x * (kOut * R);
  auto w_row = [&](int i, int r) {
    const int n = min(n0 + kOut * i + (GATED ? r & 7 : r), p.N - 1);
    return GATED && r >= 8 ? p.N + n : n;
  };
  const int64_t group_row = static_cast<int64_t>(e) * p.w_rows;
  const uint8_t* codes = p.codes + group_row * (p.kpad / 2);
  const uint8_t* scales = p.scales + (group_row / 128 + e) * p.words * 512;

  const uint32_t ring = smem_addr(smem) + static_cast<uint32_t>(warp * S::DEPTH * S::STAGE);
  const uint32_t xs = smem_addr(smem) + S::RING;
  const int chunks = (p.kpad + kChunk - 1) / kChunk;

  // The rows that this lane copies: 4 lanes a row of 64 bytes, 8 rows at a time.
  const uint8_t* src[2 * R];
  uint32_t dst[2 * R];
#pragma unroll
  for (int j = 0; j < 2 * R; ++j) {
    const int r = (j & 1) * 8 + (lane >> 2), piece = lane & 3;
    src[j] = codes + static_cast<int64_t>(w_row(j >> 1, r)) * (p.kpad / 2) + piece * 16;
    dst[j] = static_cast<uint32_t>((j >> 1) * 1024 + r * 64 + ((piece ^ (r >> 1 & 3)) * 16));
  }
  constexpr int kScaleCopies = (R * 16 * S::WORDS + 31) / 32;
  const uint8_t* ssrc[kScaleCopies];
#pragma unroll
  for (int j = 0; j < kScaleCopies; ++j) {  // word (lane + 32 j) of a chunk: [word][tile][row]
    const int i = lane + 32 * j, word = i / (16 * R), tile = i / 16 % R, row = w_row(tile, i % 16);
    ssrc[j] = scales + (static_cast<int64_t>(row / 128) * p.words + word) * 512 + row % 32 * 16 + row / 32 % 4 * 4;
  }
  auto fetch = [&](int chunk, int slot) {
    const uint32_t at = ring + static_cast<uint32_t>(slot * S::STAGE);
    const bool in = chunk * kChunk + (lane & 3) * 32 < p.kpad;
    const int64_t off = in ? static_cast<int64_t>(chunk) * (kChunk / 2) : 0;
#pragma unroll
    for (int j = 0; j < 2 * R; ++j) copy16(at + dst[j], in ? src[j] + off : codes, in);
#pragma unroll
    for (int j = 0; j < kScaleCopies; ++j) {
      const int i = lane + 32 * j, word = i / (16 * R);
      const bool sin = chunk * S::WORDS + word < p.words;
      if (i < R * 16 * S::WORDS)
        copy4(at + S::CODES + i * 4, sin ? ssrc[j] + static_cast<int64_t>(chunk) * S::WORDS * 512 : scales, sin);
    }
  };

  for (int t0 = 0; t0 < rows; t0 += S::TOKENS) {
    const int tokens = min(S::TOKENS, rows - t0);
    const uint16_t* x = p.x + (static_cast<int64_t>(row0) + t0) * p.ldx;
    float tot[R][NT][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) tot[i][n][c] = 0.0f;

    bool more = false;  // elements are left for a further run
    int run = 0;
    do {
      more = false;
      int next = warp;  // chunk that is fetched next
#pragma unroll
      for (int s = 0; s < S::DEPTH - 1; ++s) {
        if (next < chunks) fetch(next, s);
        copy_commit();
        next += kWarps;
      }
      int slot = 0;
      int chunk = warp;
      for (int k0 = 0; k0 < p.kpad; k0 += S::PANEL) {
        // ---- the panel of x, as fp16
        __syncthreads();  // the last panel (or the sums before) is done with
        const int vectors = min(S::PANEL, (p.kpad - k0 + kChunk - 1) / kChunk * kChunk) / 8;
        if (BF && tid < S::TOKENS) {
          s_max[tid] = 0u;
          s_min[tid] = 0xFFFFu;
        }
        if (BF) __syncthreads();
        for (int t = 0; t < tokens; ++t) {
          uint32_t hi = 0u, lo = 0xFFFFFFFFu;
          for (int v = tid; v < vectors; v += kThreads) {
            const uint4 w = load8(x + t * p.ldx, k0 + 8 * v, p.K, p.vec);
            sts128(xs + static_cast<uint32_t>(t * p.pitch + 16 * v), w);
            if (BF) {
              const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t m = a[i] & 0x7FFF7FFFu;
                hi = __vmaxu2(hi, m);
                lo = __vminu2(lo, (m + 0x7FFF7FFFu) ^ 0x80008000u);  // m - 1, zeros last
              }
            }
          }
          if (BF) {
            hi = __reduce_max_sync(0xFFFFFFFFu, max(hi & 0xFFFFu, hi >> 16));
            lo = __reduce_min_sync(0xFFFFFFFFu, min(lo & 0xFFFFu, lo >> 16));
            if (lane == 0) {
              atomicMax(&s_max[t], hi);
              atomicMin(&s_min[t], lo);
            }
          }
        }
        __syncthreads();
        if (BF) {
          for (int t = 0; t < tokens; ++t) {
            // exponent of the largest element; this run takes those from `top` down to `bottom` (bit patterns)
            const int E = max(static_cast<int>(s_max[t] >> 7), 1) - kRange * run;
            const uint32_t top = E < 1 ? 0u : static_cast<uint32_t>(E + 1) << 7;  // below 1: all of them are through
            const uint32_t bottom = E - (kRange - 1) <= 1 ? 0u : static_cast<uint32_t>(E - (kRange - 1)) << 7;
            const uint32_t least = s_min[t] + 1u;  // the smallest but zero; 0x10000: none
            const bool all = run == 0 && least >= bottom;
            if (least < bottom) more = true;
            const int shift = 142 - max(E, 1);
            const float f1 = pow2f(shift / 2), f2 = pow2f(shift - shift / 2);
            for (int v = tid; v < vectors; v += kThreads) {
              const uint32_t at = xs + static_cast<uint32_t>(t * p.pitch + 16 * v);
              const uint4 w = lds128(at);
              uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t u = a[i] << 16, h = a[i] & 0xFFFF0000u;
                if (!all) {
                  const uint32_t ml = a[i] & 0x7FFFu, mh = a[i] >> 16 & 0x7FFFu;
                  if (ml < bottom || ml >= top) u = 0u;
                  if (mh < bottom || mh >= top) h = 0u;
                }
                a[i] = pack_half2(__uint_as_float(u) * f1 * f2, __uint_as_float(h) * f1 * f2);
              }
              sts128(at, make_uint4(a[0], a[1], a[2], a[3]));
            }
          }
          __syncthreads();
        }

        // ---- this warp's chunks of the panel
        float acc[R][NT][4];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][n][c] = 0.0f;
#pragma unroll 1
        for (; chunk < chunks && chunk * kChunk < k0 + S::PANEL; chunk += kWarps) {
          copy_wait<S::DEPTH - 2>();
          __syncwarp();
          // the slot that was used before this one is free
          if (next < chunks) fetch(next, slot == 0 ? S::DEPTH - 1 : slot - 1);
          copy_commit();
          next += kWarps;
          const uint32_t at = ring + static_cast<uint32_t>(slot * S::STAGE);
          const uint32_t xat = xs + static_cast<uint32_t>((lane >> 2) * p.pitch + (chunk * kChunk - k0) * 2 + (lane & 3) * 16);
          uint32_t sc[R][2][S::WORDS];
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int w = 0; w < S::WORDS; ++w)
                sc[i][half][w] = lds32(at + S::CODES + static_cast<uint32_t>((w * R + i) * 16 + half * 8 + (lane >> 2)) * 4);
#pragma unroll
          for (int s = 0; s < 4; s += 2) {
            uint4 xb[2][NT];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int n = 0; n < NT; ++n)
                xb[j][n] = 8 * n + (lane >> 2) < tokens ? lds128(xat + static_cast<uint32_t>(8 * n * p.pitch + (s + j) * 64))
                                                        : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const int r = (lane & 7) + (lane & 8);
              uint32_t w[4];
              ldmatrix4(at + static_cast<uint32_t>(i * 1024 + r * 64 + (((s + (lane >> 4)) ^ (r >> 1 & 3)) * 16)), w);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint32_t lo[4], hi[4];
                decode8(w[2 * j], lo);
                decode8(w[2 * j + 1], hi);
                if (S::NV) {
                  const uint32_t sel = 2u * ((s + j) & 1) + ((lane >> 1) & 1u);
                  const uint32_t sl = scale_half2(sc[i][0][(s + j) >> 1 & (S::WORDS - 1)], sel);
                  const uint32_t sh = scale_half2(sc[i][1][(s + j) >> 1 & (S::WORDS - 1)], sel);
#pragma unroll
                  for (int c = 0; c < 4; ++c) {
                    lo[c] = mul_half2(lo[c], sl);
                    hi[c] = mul_half2(hi[c], sh);
                  }
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    mma16816(acc[i][n], lo[0], hi[0], lo[1], hi[1], xb[j][n].x, xb[j][n].y);
                    mma16816(acc[i][n], lo[2], hi[2], lo[3], hi[3], xb[j][n].z, xb[j][n].w);
                  }
                } else {
                  const float sl = scale_mx(sc[i][0][0], s + j), sh = scale_mx(sc[i][1][0], s + j);
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma16816(c, lo[0], hi[0], lo[1], hi[1], xb[j][n].x, xb[j][n].y);
                    mma16816(c, lo[2], hi[2], lo[3], hi[3], xb[j][n].z, xb[j][n].w);
                    acc[i][n][0] = fmaf(c[0], sl, acc[i][n][0]);
                    acc[i][n][1] = fmaf(c[1], sl, acc[i][n][1]);
                    acc[i][n][2] = fmaf(c[2], sh, acc[i][n][2]);
                    acc[i][n][3] = fmaf(c[3], sh, acc[i][n][3]);
                  }
                }
              }
            }
          }
          slot = slot + 1 == S::DEPTH ? 0 : slot + 1;
        }
        // ---- into the sums, without the panel's scale
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int t = 8 * n + 2 * (lane & 3) + c;
            int back = S::NV ? 0 : kMxShift;
            if (BF && t < tokens) back += max(max(static_cast<int>(s_max[t] >> 7), 1) - kRange * run, 1) - 142;
#pragma unroll
            for (int i = 0; i < R; ++i) {
              tot[i][n][c] += scaled(acc[i][n][c], back);
              tot[i][n][c + 2] += scaled(acc[i][n][c + 2], back);
            }
          }
      }
      copy_wait<0>();
      ++run;
    } while (BF && __syncthreads_or(more));

    // ---- the warps' sums, in order; all copies are in, and no warp reads the ring any more
    __syncthreads();
    float* part = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) part[((warp * R + i) * NT + n) * 128 + c * 32 + lane] = tot[i][n][c];
    __syncthreads();
    auto sum = [&](int i, int n, int c, int l) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += part[((w * R + i) * NT + n) * 128 + c * 32 + l];
      return v;
    };
    for (int o = tid; o < R * NT * (GATED ? 64 : 128); o += kThreads) {
      // a value of lane l = 4 row + token / 2: c = token % 2, + 2 for the second eight rows of the tile
      const int col = o % kOut, t = o / kOut % 8, n = o / kOut / 8 % NT, i = o / kOut / 8 / NT;
      const int l = (col & 7) * 4 + (t >> 1), c = t & 1;
      const int token = 8 * n + t, out = n0 + kOut * i + col;
      if (token >= tokens || out >= p.N) continue;
      float v = p.alpha * sum(i, n, GATED ? c : c + 2 * (col >> 3), l);
      if (GATED) v = act_value(v, p.act) * (p.alpha * sum(i, n, c + 2, l));
      const int64_t at = (static_cast<int64_t>(row0) + t0 + token) * p.ldy + out;
      if (p.out_type == OZK_F32) static_cast<float*>(p.y)[at] = v;
      else if (p.out_type == OZK_F16) static_cast<__half*>(p.y)[at] = __float2half_rn(v);
      else static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
    }
    __syncthreads();  // the ring is filled again
  }
}

// Once per device and kernel: the shared-memory opt-in.
cudaError_t allow_smem(const void* kernel, int bytes) {
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, cudaError_t> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  auto it = done.find({dev, kernel});
  if (it == done.end())
    it = done.emplace(std::make_pair(dev, kernel), cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)).first;
  return it->second;
}

template <int FMT, int R, int NT, bool GATED, bool BF>
cudaError_t launch(GemvParams p, cudaStream_t stream) {
  using S = Shape<FMT, R, NT>;
  auto kernel = gemv_kernel<FMT, R, NT, GATED, BF>;
  constexpr int kMost = S::RING + S::TOKENS * S::PITCH;
  static_assert(kMost + 8 * S::TOKENS <= 232448, "shared memory");
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kMost);
  if (e != cudaSuccess) return e;
  const int per = (GATED ? 8 : 16) * R;
  const dim3 grid((p.N + per - 1) / per, p.offsets ? std::min(p.groups, p.T) : 1);
  p.pitch = std::min(S::PANEL, (p.kpad + kChunk - 1) / kChunk * kChunk) * 2 + 64;
  const size_t smem = S::RING + static_cast<size_t>(std::min(p.T, S::TOKENS)) * p.pitch;
  return launch_dependent(kernel, grid, dim3(kThreads), smem, stream, p);
}

template <int FMT, bool GATED, bool BF>
cudaError_t choose(const GemvParams& p, int num_sms, cudaStream_t stream) {
  const int active = p.offsets ? std::min(p.groups, p.T) : 1;
  const int rows = (p.T + active - 1) / active;  // of a group, as their mean: the offsets are on the device
  const int64_t tiles = static_cast<int64_t>((p.N + (GATED ? 7 : 15)) / (GATED ? 8 : 16)) * active;
  if (rows <= 8) {
    if (tiles >= 16 * num_sms) return launch<FMT, 4, 1, GATED, BF>(p, stream);
    if (tiles >= 4 * num_sms) return launch<FMT, 2, 1, GATED, BF>(p, stream);
    return launch<FMT, 1, 1, GATED, BF>(p, stream);
  }
  if (rows <= 16) return tiles >= 3 * num_sms ? launch<FMT, 4, 2, GATED, BF>(p, stream) : launch<FMT, 1, 2, GATED, BF>(p, stream);
  return tiles >= 2 * num_sms ? launch<FMT, 2, 4, GATED, BF>(p, stream) : launch<FMT, 1, 4, GATED, BF>(p, stream);
}

std::atomic<bool> g_any{false};

}  // namespace

cudaError_t launch_mx4_gemv(const Gemv& q, int num_sms, cudaStream_t stream) {
  g_any.store(true, std::memory_order_relaxed);
  GemvParams p = {};
  p.T = static_cast<int>(q.T);
  p.N = static_cast<int>(q.N);
  p.K = static_cast<int>(q.K);
  p.groups = q.w.groups;
  p.w_rows = static_cast<int>(q.w.rows / q.w.groups);
  p.kpad = static_cast<int>(ozk_kpad(q.K));
  p.words = mx4_kgroups(q.K, q.w.format);
  p.offsets = q.offsets;
  p.codes = q.w.codes;
  p.scales = q.w.scales;
  p.x = static_cast<const uint16_t*>(q.x);
  p.ldx = q.ldx;
  p.y = q.y;
  p.ldy = q.ldy;
  p.out_type = q.out_type;
  p.alpha = q.K ? q.alpha : 1.0f;
  p.act = q.act;
  p.vec = reinterpret_cast<uintptr_t>(q.x) % 16 == 0 && (q.ldx % 8 == 0 || q.T == 1);
  const bool bf = q.dtype == OZK_BF16, gated = q.gated;
#define OZK_GEMV(FMT)                                                                                              \
  (gated ? (bf ? choose<FMT, true, true>(p, num_sms, stream) : choose<FMT, true, false>(p, num_sms, stream))       \
         : (bf ? choose<FMT, false, true>(p, num_sms, stream) : choose<FMT, false, false>(p, num_sms, stream)))
  return q.w.format == OZK_MXFP4 ? OZK_GEMV(OZK_MXFP4) : OZK_GEMV(OZK_NVFP4);
#undef OZK_GEMV
}

int take_gemv_status(int* status) {
  *status = 0;
  if (!g_any.load(std::memory_order_relaxed)) return OZK_OK;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_gemv_status, sizeof(int)) != cudaSuccess) return OZK_ERR_CUDA;
  if (v) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_gemv_status, &zero, sizeof(int)) != cudaSuccess) return OZK_ERR_CUDA;
  }
  *status = v;
  return OZK_OK;
}

}  // namespace ozk
