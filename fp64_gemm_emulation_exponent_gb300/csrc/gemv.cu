// Products of a few 16-bit rows with microscaled 4-bit weights:
//   y[t, n] = alpha sum_k x[t, k] w[g(t)][n, k], and its gated form
//   h[t, n] = act(alpha sum_k x[t, k] w[g][n, k]) (alpha sum_k x[t, k] w[g][H + n, k]).
//
// The floor is reading the weights once: N K (1/2 + 1/block) bytes, 42 weights
// a cycle and SM at the measured 6.8 TB/s, or a quarter of an SM's 512 weights
// (a unit: 32 columns of 16 rows) in 48 cycles.  The work on a weight between
// memory and its product decides how near the kernel comes:
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
// bf16 rows do not fit fp16 as they are.  A warp scales each row by a power of
// two that brings the largest element of the first chunk it takes to [2^9,
// 2^10): exact as fp16 for every element from 2^-26 to 2^6 of that one.  Every
// chunk is checked for it; where one does not fit, the sums are put away and
// the scale starts again from that chunk, and elements that are too small even
// so take part in further passes over the chunk, 27 binades at a time.  Those
// passes cost what they compute.  Rows that are gelu(g) u take no longer than
// normal ones with g of a standard deviation of 1, but with 2 or 4 (gelu(-6) is
// 2^-27, and a chunk has such) two to four times as long; us, normal / 2 / 4: 1 x
// 8192 x 4096 6.8 / 13.1 / 21.4, 8 x 8192 x 8192 12.1 / 26.2 / 34.4, 16 x 8192 x
// 8192 15.9 / 49.1 / 63.2.  After silu at most a half longer.  fp16 rows need
// neither check nor passes: 5.7, 10.0 and 12.6.
//
// A block owns 16 R output rows of w (gated: 8 R of each projection) and all
// of K; its warps take the chunks of 128 or 256 columns in turn, each through a
// ring of its own in shared memory (codes, scales and x) filled by asynchronous
// copies, no barrier between them, and the warps' sums are added at the end in
// a fixed order.
//
// Measured on a GB300 (us in replayed graphs, weights from HBM; floor at 6.79
// TB/s): 8192 x 4096 NVFP4, 1 row 6.8, 8 rows 7.6, 16 rows 9.6 (2.8, and some 2
// of a launch); 8192 x 8192 10.8, 11.9, 15.8 (5.6); 1024 x 4096 3.2, 4.0, 5.4;
// 32 rows over 32 experts, 4096 -> 2048 MXFP4, 20.7 (10.6).  No unit is full: HBM
// 24-42%, issue slots 38-51% (36 instructions a unit with one row and many
// columns, 18.5 of them the conversions, scales and products themselves), tensor
// pipe 13-24%.  What is left is latency on 2 to 3.3 warps a scheduler, the start
// (2 of 5.4 us pass before a warp's first chunk is in), and blocks that are two on
// some SMs and one on others (a sixth).  Without the products the loop runs at
// 82% of HBM's rate.
// The steps (16 x 8192 x 8192 / 1 x 8192 x 4096, us): x staged as fp16 for the
// whole block, panel by panel 58.8 / 10.7; rings and conversion per warp 24.3 /
// 11.9; chunks of 256 columns, blocks of two tiles 21.3 / 7.8; copies without
// tests 18.3 / 7.6; the path of wide chunks out of line, scale words of all tiles in
// one copy 17.9 / 7.8; 8 warps of 255 registers 16.6; the first chunk's prefetch
// 15.7 / 6.8.
// What did not help: rows of x converted by all lanes together where a tile has
// three or fewer (a fifth fewer instructions, 5% slower: a longer way from the
// copy to the products), more warps a block at the price of registers (30% slower
// with 16 rows), three blocks an SM, prefetching further ahead, whole ranges of
// columns to L2 for grouped rows (13% slower).
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

constexpr int kTop = 9;         // exponent that the largest element of a row is scaled to
constexpr int kHead = 6;        // binades above it that fp16 has room for
constexpr int kBelow = 26;      // binades below it that stay exact: down to 2^-17, 7 bits above fp16's last

// W: warps. NT: tiles of 8 rows of x; 0: one or two rows, which the lanes convert together.
template <int FMT, int R, int NT, int W>
struct Shape {
  static constexpr bool NV = FMT == OZK_NVFP4;
  static constexpr bool FEW = NT == 0;
  static constexpr int TILES = FEW ? 1 : NT;
  static constexpr int TOKENS = FEW ? 2 : 8 * NT;
  static constexpr int ROWS = FEW ? 2 : NT;       // rows of x that a lane keeps a scale for
  static constexpr int CHUNK = FEW ? 256 : 128;   // columns of a chunk
  static constexpr int ROW = CHUNK / 2;           // bytes of codes of a row
  static constexpr int PIECES = ROW / 16;
  static constexpr int WORDS = CHUNK / (NV ? 64 : 128);  // scale words of a row
  static constexpr int CODES = R * 16 * ROW;
  static constexpr int SCALES = (R * 16 * WORDS * 4 + 255) / 256 * 256;
  static constexpr int XROW = CHUNK * 2;          // bytes of a row of x
  static constexpr int DEPTH = FEW && R == 1 ? 3 : 2;
  static constexpr int STAGE = CODES + SCALES;
  static constexpr int SUMS = R * TILES * 512;    // bytes of a warp's sums, at its end in the ring's place
  // Chunks of x that a warp has room for: with two, the next one's rows come while one is multiplied.
  static constexpr int XCHUNKS = NT == 1 ? 2 : 1;
  // A warp's part of shared memory: its ring, and rows of x.
  static constexpr int RING = (DEPTH * STAGE + 511) / 512 * 512;
  static constexpr int part(int tokens) { return RING + XCHUNKS * tokens * XROW; }
  static_assert(XCHUNKS == 1 || DEPTH == 2, "codes and x take turns alike");
  static constexpr int bytes(int tokens) { return W * part(tokens); }
  static_assert(SUMS <= RING, "the sums take the ring's place");
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
  bool side;               // the scale words of a block's tiles lie side by side
  int tokens;              // rows of x that a stage has room for
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// 4, 8 or 16 bytes to shared memory.
template <int BYTES>
__device__ __forceinline__ void copy(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
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
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&v)[N]) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(addr) : "memory");
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr) : "memory");
  } else {
    static_assert(N == 4, "one, two or four words");
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
  }
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
// Both halves of a times the low or the high half of b.
template <bool HIGH>
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 s = *reinterpret_cast<__half2*>(&b), v = __hmul2(*reinterpret_cast<__half2*>(&a), HIGH ? __high2half2(s) : __low2half2(s));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two E4M3 bytes as an fp16 pair; two E8M0 bytes as a bf16 pair (2^-127 is one of its subnormals, 255 is NaN).
__device__ __forceinline__ uint32_t e4m3_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ uint32_t e8m0_bf162(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
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

// Elements [k, k + 8) of a row of x as stored, zeros from K on, at any alignment.
__device__ __forceinline__ uint4 load16(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load8(const uint16_t* row, int k, int K, bool vec) {
  if (vec && k + 8 <= K) return load16(row + k);
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
  const int half = e >> 1;
  return v * pow2f(half) * pow2f(e - half);
}
// ---- bf16 pairs as fp16 pairs
// Largest and smallest magnitudes of some elements, in both halves: m + 0x7FFF
// a half makes zeros 0x7FFF and others 0x8000 + (m - 1), so that the unsigned
// maximum and the signed minimum leave zeros out.
struct Range {
  uint32_t hi = 0x7FFF7FFFu, lo = 0x7FFF7FFFu;
  __device__ __forceinline__ void add(uint32_t a, uint32_t b) {
    a = (a & 0x7FFF7FFFu) + 0x7FFF7FFFu;
    b = (b & 0x7FFF7FFFu) + 0x7FFF7FFFu;
    hi = __vimax3_u16x2(hi, a, b);
    lo = __vimin3_s16x2(lo, a, b);
  }
  __device__ __forceinline__ void add(const uint4& v) {
    add(v.x, v.y);
    add(v.z, v.w);
  }
  // Over all lanes of the warp.
  __device__ __forceinline__ void warp_wide() {
    hi = __reduce_max_sync(0xFFFFFFFFu, max(hi & 0xFFFFu, hi >> 16)) * 0x10001u;
    const int least = __reduce_min_sync(0xFFFFFFFFu, min(static_cast<int>(static_cast<int16_t>(lo & 0xFFFFu)), static_cast<int>(lo) >> 16));
    lo = (static_cast<uint32_t>(least) & 0xFFFFu) * 0x10001u;
  }
  // What hi and lo are when all but zeros have exponents from E - kBelow to E + kHead.
  static __device__ __forceinline__ Range within(int E) {
    const uint32_t most = static_cast<uint32_t>(min((E + kHead + 1) << 7, 0x8000)) + 0x7FFEu;
    const int least = E - kBelow <= 1 ? -0x8000 : ((E - kBelow) << 7) - 0x8001;
    return {most * 0x10001u, (static_cast<uint32_t>(least) & 0xFFFFu) * 0x10001u};
  }
  __device__ __forceinline__ bool inside(const Range& r) const {
    return __vmaxu2(hi, r.hi) == r.hi && __vmins2(lo, r.lo) == r.lo;
  }
  // Biased exponents of the largest and the smallest but zero (0 as 1); without any element: none.
  __device__ __forceinline__ bool any() const { return (hi & 0x80008000u) != 0u; }
  __device__ __forceinline__ int top() const {
    const uint32_t m = max(hi & 0xFFFFu, hi >> 16);
    return max(static_cast<int>((m - 0x7FFFu) >> 7), 1);
  }
  __device__ __forceinline__ int bottom() const {
    const int a = static_cast<int16_t>(lo & 0xFFFFu), b = static_cast<int16_t>(lo >> 16);
    return max((min(a, b) + 0x8001) >> 7, 1);
  }
};
__device__ __forceinline__ uint32_t to_half2(uint32_t pair, uint32_t factor) {
  uint32_t v, r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(pair), "r"(factor));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(v & 0xFFFF0000u)), "f"(__uint_as_float(v << 16)));
  return r;
}
// The scale 2^shift(E) for a largest exponent E, as a bf16 pair.
__device__ __forceinline__ int shift_of(int E) { return min(kTop + 127 - E, 127); }
__device__ __forceinline__ uint32_t factor_of(int E) { return static_cast<uint32_t>((shift_of(E) + 127) << 7) * 0x10001u; }
// Those of a pair with exponents from E down to E - kBelow, zeros for the others.
__device__ __forceinline__ uint32_t only(uint32_t pair, int E) {
  const uint32_t top = E < 1 ? 0u : static_cast<uint32_t>(E + 1) << 7;
  const uint32_t bottom = E - kBelow <= 1 ? 0u : static_cast<uint32_t>(E - kBelow) << 7;
  const uint32_t l = pair & 0x7FFFu, h = pair >> 16 & 0x7FFFu;
  if (l < bottom || l >= top) pair &= 0xFFFF0000u;
  if (h < bottom || h >= top) pair &= 0x0000FFFFu;
  return pair;
}
__device__ __forceinline__ uint4 only(uint4 v, int E) {
  return make_uint4(only(v.x, E), only(v.y, E), only(v.z, E), only(v.w, E));
}
__device__ __forceinline__ uint4 to_half2(uint4 v, uint32_t factor) {
  return make_uint4(to_half2(v.x, factor), to_half2(v.y, factor), to_half2(v.z, factor), to_half2(v.w, factor));
}

// Where 16-byte pieces lie: of a row of codes of a tile, and of a row of x.
template <typename S>
__device__ __forceinline__ uint32_t code_piece(int r, int piece) {
  return static_cast<uint32_t>(r * S::ROW + ((piece ^ (S::FEW ? r & 7 : r >> 1 & 3)) * 16));
}
template <typename S>
__device__ __forceinline__ uint32_t x_piece(int t, int piece) {
  return static_cast<uint32_t>(t * S::XROW + ((piece ^ (t & 1) * 4) * 16));
}

// acc += the products of a chunk's weights (stage at `at`) with its rows of x
// (at `xat`; convert makes fp16 of eight elements of this lane's row of tile
// n).  Lanes of rows that are not there read the last one; their sums are
// nobody's.
template <typename S, int R, typename F>
__device__ __forceinline__ void multiply(uint32_t at, uint32_t xat, int tokens, int pairs, float (&acc)[R][S::TILES][4], F convert) {
  constexpr int TILES = S::TILES;
  const int lane = threadIdx.x & 31;
  const uint32_t wat = at + code_piece<S>(lane & 15, lane >> 4);
  const uint32_t sat = at + S::CODES + static_cast<uint32_t>((lane >> 2) * (4 * R));
  uint32_t xrow[TILES];
#pragma unroll
  for (int n = 0; n < TILES; ++n) xrow[n] = xat + x_piece<S>(min(8 * n + (lane >> 2), tokens - 1), lane & 3);
#pragma unroll
  for (int s = 0; s < S::CHUNK / 64; ++s) {  // 64 columns: two segments of 32
    if (s >= pairs) break;                   // the last chunk
    uint4 xb[2][TILES];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int n = 0; n < TILES; ++n) xb[j][n] = convert(lds128(xrow[n] ^ static_cast<uint32_t>((2 * s + j) * 64)), n);
    uint32_t scl[R], sch[R];  // of rows lane / 4 and lane / 4 + 8 of the tiles
    lds_words(sat + (S::NV ? s : s >> 1) * (64 * R), scl);
    lds_words(sat + (S::NV ? s : s >> 1) * (64 * R) + 32 * R, sch);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      uint32_t w[4];
      ldmatrix4((wat ^ static_cast<uint32_t>(s * 32)) + i * 16 * S::ROW, w);
      uint32_t sl = scl[i], sh = sch[i];
      if (S::NV) {  // of a word's four blocks of 16 the lane's own: one in each segment
        const uint32_t pick = lane & 2 ? 0x31u : 0x20u;
        sl = e4m3_half2(__byte_perm(sl, 0, pick));
        sh = e4m3_half2(__byte_perm(sh, 0, pick));
      } else {
        sl = e8m0_bf162(s & 1 ? sl >> 16 : sl);
        sh = e8m0_bf162(s & 1 ? sh >> 16 : sh);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t lo[4], hi[4];
        decode8(w[2 * j], lo);
        decode8(w[2 * j + 1], hi);
        if (S::NV) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            lo[c] = j ? mul_half2<true>(lo[c], sl) : mul_half2<false>(lo[c], sl);
            hi[c] = j ? mul_half2<true>(hi[c], sh) : mul_half2<false>(hi[c], sh);
          }
#pragma unroll
          for (int n = 0; n < TILES; ++n) {
            mma16816(acc[i][n], lo[0], hi[0], lo[1], hi[1], xb[j][n].x, xb[j][n].y);
            mma16816(acc[i][n], lo[2], hi[2], lo[3], hi[3], xb[j][n].z, xb[j][n].w);
          }
        } else {
          const float fl = __uint_as_float(j ? sl & 0xFFFF0000u : sl << 16);
          const float fh = __uint_as_float(j ? sh & 0xFFFF0000u : sh << 16);
#pragma unroll
          for (int n = 0; n < TILES; ++n) {
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma16816(c, lo[0], hi[0], lo[1], hi[1], xb[j][n].x, xb[j][n].y);
            mma16816(c, lo[2], hi[2], lo[3], hi[3], xb[j][n].z, xb[j][n].w);
            acc[i][n][0] = fmaf(c[0], fl, acc[i][n][0]);
            acc[i][n][1] = fmaf(c[1], fl, acc[i][n][1]);
            acc[i][n][2] = fmaf(c[2], fh, acc[i][n][2]);
            acc[i][n][3] = fmaf(c[3], fh, acc[i][n][3]);
          }
        }
      }
    }
  }
}

// Calls f(i, n, c, 2^back) for every sum of this lane (tile i, rows of x 8 n + 2 (lane % 4) + c % 2), where E is the
// exponent that the scale of this lane's row (lane / 4) of tile n was made for.
template <int R, int TILES, typename F>
__device__ __forceinline__ void unscaled(const int (&E)[TILES], F f) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < TILES; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int back = __shfl_sync(0xFFFFFFFFu, -shift_of(E[n]), (2 * (lane & 3) + c) * 4);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        f(i, n, c, back);
        f(i, n, c + 2, back);
      }
    }
}

// A chunk whose rows of x (as they came, at `xat`) hold elements too small for
// their largest one's scale: one run over its weights for every kBelow + 1
// binades, added to `away`.  E and low: exponents of the largest and the
// smallest element of this lane's row of every tile.  Out of line, so that the
// loop that calls it keeps its registers: what it costs is said above.
template <typename S, int R>
__device__ __noinline__ void multiply_wide(uint32_t at, uint32_t xat, int tokens, int pairs, const int (&E)[S::TILES],
                                           const int (&low)[S::TILES], float* away) {
  constexpr int TILES = S::TILES;
  int top[TILES];
#pragma unroll
  for (int n = 0; n < TILES; ++n) top[n] = E[n];
  for (;;) {
    float acc[R][TILES][4] = {};
    multiply<S, R>(at, xat, tokens, pairs, acc, [&](uint4 v, int n) { return to_half2(only(v, top[n]), factor_of(top[n])); });
    unscaled<R>(top, [&](int i, int n, int c, int back) { away[(i * TILES + n) * 4 + c] += scaled(acc[i][n][c], back); });
    bool left = false;
#pragma unroll
    for (int n = 0; n < TILES; ++n) {
      left = left || low[n] < top[n] - kBelow;
      top[n] -= kBelow + 1;
    }
    if (!__any_sync(0xFFFFFFFFu, left)) return;
  }
}

// Blocks of an SM that registers are kept for: 16 warps of 128 registers, but for
// 16 rows on four tiles 8 warps of 255 (16 x 8192 x 4096 NVFP4 11.7 us with 16
// warps a block, 9.6 so; before the prefetch 10.3, and 10.9 with two blocks of 8).
constexpr int blocks_of(int R, int NT, int W) { return (NT == 0 && R == 1 ? 24 : R == 4 && NT == 2 ? 8 : 16) / W; }

template <int FMT, int R, int NT, int W, bool GATED, bool BF>
__global__ void __launch_bounds__(32 * W, blocks_of(R, NT, W)) gemv_kernel(const GemvParams p) {
  using S = Shape<FMT, R, NT, W>;
  constexpr int TILES = S::TILES;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // This block's output columns: tile i has kOut of them, 32 from the next
  // tile's, so that the scale words of all tiles lie side by side.
  constexpr int kOut = GATED ? 8 : 16, kSub = 32 / kOut;
  const uint32_t N = static_cast<uint32_t>(p.N), n0 = blockIdx.x / kSub * (32 * R) + blockIdx.x % kSub * kOut;
  if (n0 >= N) return;
  auto w_row = [&](uint32_t r) {  // of row r of the tiles
    const uint32_t n = n0 + r / 16 * 32 + (GATED ? r & 7 : r & 15);
    return GATED && (r & 8) ? N + n : n;
  };
  auto in_range = [&](uint32_t r) { return n0 + r / 16 * 32 + (GATED ? r & 7 : r & 15) < N; };
  const uint32_t pitch = static_cast<uint32_t>(p.kpad) / 2;  // bytes of a row of codes

  // Every warp's first chunk is on its way to L2 while the kernel before still
  // runs: a hint that reads nothing, so what that kernel writes is not missed
  // (1 x 8192 x 4096 NVFP4 7.8 us without, 6.9 so, 7.4 with two chunks).
  if (!p.offsets && warp * S::ROW < static_cast<int>(pitch)) {
#pragma unroll
    for (uint32_t r = lane; r < 16 * R; r += 32)
      if (in_range(r))
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.codes + static_cast<uint64_t>(w_row(r)) * pitch + warp * S::ROW));
  }
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

  const uint8_t *codes = p.codes, *scales = p.scales;
  const uint32_t block_bytes = static_cast<uint32_t>(p.words) * 512;  // of the scales of 128 rows
  if (e) {
    const uint32_t group_row = static_cast<uint32_t>(e) * static_cast<uint32_t>(p.w_rows);  // below 2^30
    codes += static_cast<uint64_t>(group_row) * pitch;
    scales += static_cast<uint64_t>(group_row / 128 + e) * block_bytes;
  }

  // A warp's ring of codes and scale words, and one or two chunks' rows of x (FEW:
  // as fp16; else as they came).  16-byte pieces are swapped within a row so that
  // the rows that are read together lie in different banks.
  const uint32_t part_bytes = static_cast<uint32_t>(S::part(p.tokens));
  const uint32_t ring = smem_addr(smem) + static_cast<uint32_t>(warp) * part_bytes;
  const uint32_t xat0 = ring + S::RING;
  const int chunks = (p.kpad + S::CHUNK - 1) / S::CHUNK;
  // What this lane copies of a chunk: piece `lane % PIECES` of every
  // 32 / PIECES-th of the tiles' rows, and scale words.  Rows past the last one
  // are left out: what lies in their place reaches only sums that are not
  // written.
  constexpr int kCopies = R * 16 * S::PIECES / 32, kStep = 32 / S::PIECES;
  const int r0 = lane / S::PIECES;
  const uint8_t* src = codes + static_cast<uint64_t>(n0 + r0) * pitch + lane % S::PIECES * 16;
  const uint64_t up = GATED ? static_cast<uint64_t>(N) * pitch : 0;  // from a row to that of the other projection
  const bool all_rows = n0 + 32 * (R - 1) + kOut <= N;
  const uint32_t dst = code_piece<S>(r0, lane % S::PIECES);
  // Scale words (lane + 32 j) of a chunk, each of all tiles: [word][row of a tile][tile]
  constexpr int kScaleCopies = (16 * S::WORDS + 31) / 32;
  auto scale_at = [&](uint32_t row) {
    return scales + static_cast<uint64_t>(row / 128) * block_bytes + (row % 32 * 16 + row / 32 % 4 * 4 + lane / 16 * 512);
  };
  const uint8_t* ssrc = scale_at(w_row(lane & 15));

  for (int t0 = 0; t0 < rows; t0 += S::TOKENS) {
    const int tokens = min(S::TOKENS, rows - t0);
    const uint16_t* x = p.x + (static_cast<int64_t>(row0) + t0) * p.ldx;
    auto fetch = [&](int chunk, int slot) {
      const uint32_t at = ring + static_cast<uint32_t>(slot * S::STAGE);
      const uint8_t* from = src + static_cast<uint32_t>(chunk) * S::ROW;
      const uint32_t sfrom = static_cast<uint32_t>(chunk) * (S::WORDS * 512);  // below the 2^25 bytes of a row block
      auto code = [&](int j) {
        // rows 8 apart (where FEW, 4: pieces differ by one bit) have their pieces in the same places
        const uint32_t to = S::FEW && (j & 1) ? dst ^ 64u : dst;
        constexpr int kPer = 16 / kStep;  // copies of a tile
        const uint32_t row = j / kPer * 32 + (GATED ? j % (kPer / 2) : j % kPer) * kStep;
        copy<16>(at + to + j * kStep * S::ROW, (GATED && j % kPer >= kPer / 2 ? from + up : from) + static_cast<uint64_t>(row) * pitch);
      };
      auto scale = [&](int j) {
        const uint32_t to = at + S::CODES + (lane + 32 * j) * (4 * R);
        if (p.side) {
          copy<4 * R>(to, ssrc + sfrom + j * 1024);
        } else {
#pragma unroll 1
          for (int i = 0; i < R; ++i)
            if (in_range(16 * i + (lane & 15)))
              copy<4>(to + 4 * i, scale_at(w_row(16 * i + (lane & 15))) + sfrom + j * 1024);
        }
      };
      if (all_rows && (chunk + 1) * S::CHUNK <= p.kpad) {
#pragma unroll
        for (int j = 0; j < kCopies; ++j) code(j);
#pragma unroll
        for (int j = 0; j < kScaleCopies; ++j)
          if (S::WORDS > 1 || lane < 16) scale(j);
      } else {  // the rows, columns and words that are there
        const bool in = chunk * S::CHUNK + lane % S::PIECES * 32 < p.kpad;
#pragma unroll
        for (int j = 0; j < kCopies; ++j)
          if (in && in_range(r0 + kStep * j)) code(j);
#pragma unroll
        for (int j = 0; j < kScaleCopies; ++j)
          if ((S::WORDS > 1 || lane < 16) && in_range(lane & 15) && chunk * S::WORDS + lane / 16 + 2 * j < p.words) scale(j);
      }
    };
    // The chunk's rows of x: to shared memory, or FEW this lane's eight elements of every row.
    uint4 xr[2];
    auto fetch_x = [&](int chunk, int slot) {
      const bool whole = p.vec && (chunk + 1) * S::CHUNK <= p.K;
      if (S::FEW) {
        const int k = chunk * S::CHUNK + lane * 8;
        const uint16_t* row = x + k;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t >= tokens) break;
          xr[t] = whole ? load16(row) : load8(row - k, k, p.K, p.vec);
          row += p.ldx;
        }
        return;
      }
      const int k = chunk * S::CHUNK + (lane & 15) * 8;
      const uint32_t to = xat0 + static_cast<uint32_t>(slot * p.tokens * S::XROW) + x_piece<S>(lane >> 4, lane & 15);
      const uint16_t* row = x + (lane >> 4) * p.ldx + k;
      if (whole) {
#pragma unroll
        for (int i = 0; i < S::TOKENS / 2; ++i)
          if (2 * i + (lane >> 4) < tokens) copy<16>(to + i * 2 * S::XROW, row + i * 2 * p.ldx);
      } else {
#pragma unroll 1
        for (int i = 0; 2 * i + (lane >> 4) < tokens; ++i) sts128(to + i * 2 * S::XROW, load8(row + i * 2 * p.ldx - k, k, p.K, p.vec));
      }
    };
    float acc[R][TILES][4];
    auto clear = [&]() {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int n = 0; n < TILES; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i][n][c] = 0.0f;
    };
    clear();
    // The largest exponent that a row's scale is made for, the scale 2^shift(E), and what fits it: FEW, of row t; else of
    // this lane's row (lane / 4) of tile n.
    int E[S::ROWS];
    uint32_t factor[S::ROWS];
    Range limit[S::ROWS];
#pragma unroll
    for (int n = 0; n < S::ROWS; ++n) E[n] = 0, factor[n] = 0u, limit[n] = {0u, 0u};  // nothing fits
    auto row_values = [&](const int (&of)[S::ROWS], int (&own)[TILES]) {  // those of this lane's rows
#pragma unroll
      for (int n = 0; n < TILES; ++n) own[n] = S::FEW ? of[(lane >> 2) ? S::ROWS - 1 : 0] : of[n];
    };
    bool kept = false;          // sums of an earlier scale have been put away
    float away[R * TILES * 4];  // in local memory: used where a scale starts again
    // The sums without their scale to `to`, with what was put away.
    auto put = [&](auto&& to) {
      int own[TILES];
      row_values(E, own);
      unscaled<R>(own, [&](int i, int n, int c, int back) {
        const int at = (i * TILES + n) * 4 + c;
        const float v = BF ? scaled(acc[i][n][c], back) : acc[i][n][c];
        to(at, kept ? v + away[at] : v);
      });
    };

    int next = warp;  // chunk that is fetched next
#pragma unroll
    for (int s = 0; s < S::DEPTH - 1; ++s) {
      if (next < chunks) fetch(next, s);
      if (S::XCHUNKS == 2 && next < chunks) fetch_x(next, s);
      copy_commit();
      next += W;
    }
    if (S::XCHUNKS == 1 && warp < chunks) fetch_x(warp, 0);
    if (S::XCHUNKS == 1 && !S::FEW) copy_commit();
    int slot = 0;
#pragma unroll 1
    for (int chunk = warp; chunk < chunks; chunk += W) {
      __syncwarp();  // the slot that was used before this one is free
      const int spare = slot == 0 ? S::DEPTH - 1 : slot - 1;
      if (next < chunks) {
        fetch(next, spare);
        if (S::XCHUNKS == 2) fetch_x(next, spare);
      }
      copy_commit();
      copy_wait<S::DEPTH - 1>();  // all but the latest are in, x among them
      __syncwarp();
      next += W;
      const uint32_t xat = xat0 + (S::XCHUNKS == 2 ? static_cast<uint32_t>(slot * p.tokens * S::XROW) : 0u);
      const uint32_t at = ring + static_cast<uint32_t>(slot * S::STAGE);

      // ---- do this chunk's rows fit their scales?
      bool part = false;               // some do not, whatever the scale
      int low[S::ROWS];                // a row's smallest exponent
      if (BF) {
        Range range[S::ROWS];
        bool fits = true;
#pragma unroll
        for (int n = 0; n < S::ROWS; ++n) {
          if (S::FEW) {
            if (n >= tokens) break;
            range[n].add(xr[n]);
          } else {
            const uint32_t row = xat + x_piece<S>(min(8 * n + (lane >> 2), tokens - 1), lane & 3);
#pragma unroll
            for (int s = 0; s < S::CHUNK / 32; ++s) range[n].add(lds128(row ^ static_cast<uint32_t>(s * 64)));
          }
          fits = fits && range[n].inside(limit[n]);
        }
        if (!__all_sync(0xFFFFFFFFu, fits)) {
          if (chunk != warp) {
            put([&](int i, float v) { away[i] = v; });
            kept = true;
            clear();
          }
          bool small = false;
#pragma unroll
          for (int n = 0; n < S::ROWS; ++n) {
            if (S::FEW) {
              if (n < tokens) range[n].warp_wide();
            } else {
#pragma unroll
              for (int d = 1; d < 4; d *= 2) {
                range[n].hi = __vmaxu2(range[n].hi, __shfl_xor_sync(0xFFFFFFFFu, range[n].hi, d));
                range[n].lo = __vmins2(range[n].lo, __shfl_xor_sync(0xFFFFFFFFu, range[n].lo, d));
              }
            }
            E[n] = range[n].any() ? range[n].top() : 1;
            low[n] = range[n].any() ? range[n].bottom() : 256;
            factor[n] = factor_of(E[n]);
            limit[n] = Range::within(E[n]);
            small = small || low[n] < E[n] - kBelow;
          }
          part = __any_sync(0xFFFFFFFFu, small);
        }
      }
      const int pairs = min(S::CHUNK, p.kpad - chunk * S::CHUNK) / 64;
      if (S::FEW) {  // this chunk's rows, converted, to shared memory
        __syncwarp();
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (t < tokens) sts128(xat + x_piece<S>(t, lane), BF && !part ? to_half2(xr[t], factor[t]) : xr[t]);
        __syncwarp();
        if (chunk + W < chunks) fetch_x(chunk + W, 0);
      }
      if (!BF || !part) {
        multiply<S, R>(at, xat, tokens, pairs, acc, [&](uint4 v, int n) { return BF && !S::FEW ? to_half2(v, factor[n]) : v; });
      } else {
        if (!kept) {
#pragma unroll
          for (int i = 0; i < R * TILES * 4; ++i) away[i] = 0.0f;
          kept = true;
        }
        int top[TILES], least[TILES];
        row_values(E, top);
        row_values(low, least);
        multiply_wide<S, R>(at, xat, tokens, pairs, top, least, away);
      }
      if (S::XCHUNKS == 1 && !S::FEW) {
        __syncwarp();
        if (chunk + W < chunks) fetch_x(chunk + W, 0);
        copy_commit();
      }
      slot = slot + 1 == S::DEPTH ? 0 : slot + 1;
    }
    copy_wait<0>();
    __syncwarp();
    {
      float* mine = reinterpret_cast<float*>(smem + static_cast<size_t>(warp) * part_bytes) + lane;
      put([&](int i, float v) { mine[i * 32] = v; });
    }

    // ---- the warps' sums, in order
    __syncthreads();
    auto sum = [&](int i, int n, int c, int l) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w)
        v += reinterpret_cast<const float*>(smem + static_cast<size_t>(w) * part_bytes)[((i * TILES + n) * 4 + c) * 32 + l];
      return v;
    };
    constexpr int kRows = S::FEW ? 2 : 8;  // rows of x of a tile that can be there
    for (int o = tid; o < R * TILES * kRows * kOut; o += 32 * W) {
      // a value of lane l = 4 row + token / 2: c = token % 2, + 2 for the second eight rows of the tile
      const int col = o % kOut, t = o / kOut % kRows, n = o / (kOut * kRows) % TILES, i = o / (kOut * kRows * TILES);
      const int l = (col & 7) * 4 + (t >> 1), c = t & 1;
      const int token = 8 * n + t, out = static_cast<int>(n0) + 32 * i + col;
      if (token >= tokens || out >= p.N) continue;
      float v = p.alpha * sum(i, n, GATED ? c : c + 2 * (col >> 3), l);
      if (GATED) v = act_value(v, p.act) * (p.alpha * sum(i, n, c + 2, l));
      const int64_t to = (static_cast<int64_t>(row0) + t0 + token) * p.ldy + out;
      if (p.out_type == OZK_F32) static_cast<float*>(p.y)[to] = v;
      else if (p.out_type == OZK_F16) static_cast<__half*>(p.y)[to] = __float2half_rn(v);
      else static_cast<__nv_bfloat16*>(p.y)[to] = __float2bfloat16_rn(v);
    }
    if (t0 + S::TOKENS < rows) __syncthreads();  // the rings are filled again
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

template <int FMT, int R, int NT, int W, bool GATED, bool BF>
cudaError_t launch(GemvParams p, cudaStream_t stream) {
  using S = Shape<FMT, R, NT, W>;
  auto kernel = gemv_kernel<FMT, R, NT, W, GATED, BF>;
  static_assert(S::bytes(S::TOKENS) <= 232448, "shared memory");
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), S::bytes(S::TOKENS));
  if (e != cudaSuccess) return e;
  const int sub = GATED ? 4 : 2;  // blocks that share 32 R columns
  const dim3 grid((p.N + 32 * R - 1) / (32 * R) * sub, p.offsets ? std::min(p.groups, p.T) : 1);
  p.tokens = std::min(p.T, S::TOKENS);
  p.side = !GATED || p.N % (32 * R) == 0;
  return launch_dependent(kernel, grid, dim3(32 * W), S::bytes(p.tokens), stream, p);
}

// The block's form by the rows of x and the tiles of 16 rows of w.  More tiles
// a block (R) spread the conversion of x over more weights, more warps (W) the
// columns over more of the SM; what serves best is some 2048 warps in all with
// up to two rows, and blocks for nearly every SM with more.  Of all forms at 20
// sizes of 1 to 16 rows the one taken was the best or within 2% of it.  NVFP4, us,
// the form taken and the best other: 1 x 16384 x 4096 10.8 and 12.3 (8 warps); 1 x 8192 x
// 8192 10.8 and 11.8 (4 warps); 1 x 4096 x 16384 10.7 and 12.3 (8 warps); 1 x 1024
// x 4096 3.2 and 3.8 (two tiles).  8 x 16384 x 4096 11.9 and 11.8 (8 warps); 8 x
// 8192 x 8192 11.9 and 12.3 (8 warps); 8 x 4096 x 16384 13.3 and 15.2 (8 warps); 8 x
// 1024 x 4096 4.0 and 4.7 (two tiles).  32 rows over 32 experts 21.0 and 22.2 (8
// warps).  16 x 8192 x 8192 15.8 and 18.9 (two tiles); 16 x 4096 x 16384 18.4 and 20.8
// (8 warps); 16 x 1024 x 4096 5.4 and 6.5 (two tiles).  Tiles of 32 rows of x took
// longer than two runs of 16 (45 and 33 us at 8192 x 8192, in an earlier form).
template <int FMT, bool GATED, bool BF>
cudaError_t choose(const GemvParams& p, int num_sms, cudaStream_t stream) {
  const int active = p.offsets ? std::min(p.groups, p.T) : 1;
  const int rows = (p.T + active - 1) / active;  // of a group, as their mean: the offsets are on the device
  const int64_t tiles = static_cast<int64_t>((p.N + (GATED ? 7 : 15)) / (GATED ? 8 : 16)) * active;
  if (p.T <= 2) {  // no group has more
    if (tiles >= 6 * num_sms) return launch<FMT, 2, 0, 4, GATED, BF>(p, stream);
    if (tiles >= 3 * num_sms) return launch<FMT, 2, 0, 8, GATED, BF>(p, stream);
    if (tiles >= num_sms) return launch<FMT, 2, 0, 16, GATED, BF>(p, stream);
    return launch<FMT, 1, 0, 8, GATED, BF>(p, stream);
  }
  if (rows <= 8) {
    if (tiles >= 6 * num_sms) return launch<FMT, 4, 1, 4, GATED, BF>(p, stream);
    if (tiles >= 3 * num_sms) return launch<FMT, 4, 1, 16, GATED, BF>(p, stream);
    if (tiles >= num_sms) return launch<FMT, 2, 1, 16, GATED, BF>(p, stream);
    return launch<FMT, 1, 1, 8, GATED, BF>(p, stream);
  }
  if (tiles >= 3 * num_sms) return launch<FMT, 4, 2, 8, GATED, BF>(p, stream);
  if (tiles >= num_sms) return launch<FMT, 2, 2, 16, GATED, BF>(p, stream);
  return launch<FMT, 1, 2, 8, GATED, BF>(p, stream);
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
