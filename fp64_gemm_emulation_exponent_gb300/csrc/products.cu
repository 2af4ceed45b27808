// Low-precision products on the tensor cores: rows grouped by expert with
// 16-bit operands (forward and both gradients), and microscaled 4-bit
// operands (one group or many).
//
// One tile is kTileRows (or, on a CTA pair, twice that) output columns by up
// to BN output rows of one group.  The operand with few rows of its own (the
// grouped rows) takes the N side of tcgen05.mma and the weights the M side:
// N may be any multiple of 16, so a group of three rows costs the tensor
// cores and the copies three rows' worth, not a tile's, and the weights,
// which bound small calls, stream through whole.
//   forward, 4-bit   out[t, m] = sum_k x[t, k] w[e][m, k]     both K-major
//   gradient of x    out[t, m] = sum_k dy[t, k] w[e][k, m]    w M-major
//   gradient of w    out[e][n, m] = sum_t dy[t, n] x[t, m]    both MN-major,
//                    the group's rows are the reduction
// The MN-major operands are read as they lie (tcgen05's transposed operand
// form), nothing is transposed in memory.
//
// Roles of a CTA (12 warps): warps 0 and 3 issue the TMA loads, warp 1 the
// MMAs, warp 2 (gradient of w) clears the rows past a group's end in its last
// block, warps 4..11 the epilogue.  Every mbarrier wait is bounded; a wait
// that runs out latches the fault and stops the roles of the CTA and its peer;
// once all have stopped, the copies in flight are waited for, each on the
// barrier that it was issued on, and the kernel returns.
//
// Measured on a GB300 (CUDA events around graph replays; rates against the
// measured 1852 TFLOP/s bf16 and 6.68 TB/s):
//   8 groups of 2048 rows, 4096 x 4096, bf16: 288 us forward, 287 us dx, 278 us
//     dw, 1.91-1.98 PFLOP/s, bound by the MMAs (516 cycles a stage of 512)
//   8192^3 NVFP4: 150-154 us, 7.2 PFLOP/s, 0.97 of four times the bf16 rate; a stage
//     of 38 KB an SM takes 525 cycles to arrive, its MMAs 512
//   8192 rows over 16 groups, 4096 -> 2048, bf16: 97 us, 1.42 PFLOP/s; the
//     weights are read for two tiles of rows only, HBM and MMAs about even
//   1 x 8192 x 4096 NVFP4: 5.9 us, 2.1 of them a launch with nothing to do; one
//     SM takes in 64-74 bytes a cycle, and the 64 tiles are on 64 SMs
// What did not help: prefetching the next tile's operands into L2 by TMA (10-20%
// slower: the copies' requests are what is short) or the weights' lines by an
// idle warp 16 stages ahead (no change; 40 ahead 18% slower), scale tiles multicast in
// the pair, a cluster of two or four CTAs along the terms of a small call (the
// cluster's launch and barriers cost 1.9 us, the split saves 1.7), weights on
// the N side in tiles of 64.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <map>
#include <mutex>

#include "lowp.h"
#include "tc_ptx.cuh"

namespace ozk {
namespace {

constexpr int kTileRows = 128;   // M side of one CTA: TMEM lanes
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr uint32_t kRowBytes = 128;                       // K bytes of a stage: one swizzle row
constexpr uint32_t kABytes = kTileRows * kRowBytes;       // 16 KB
constexpr uint32_t kScaleTile = 512;                      // 128 rows x 4 scale bytes
constexpr uint64_t kStageNs = 4000;  // what a stage may take, for the limits of the waits (0.3 us is usual)
constexpr int kSuper = 16;       // tiles of the M side that run together (L2 reuse)

constexpr int kTableInts = 4 * (kMaxGroups + 1);  // group table: see Group
constexpr int kSortGroups = 256;                // up to so many groups are put in order

// Formats of an instance.  k16: 16-bit operands; the 4-bit ones differ in the
// MMA's kind and in how many blocks a step of 64 takes (4 scale bytes, or 2).
enum Format { kNv = OZK_NVFP4, kMx = OZK_MXFP4, k16 = 2 };

template <ProductOp OP, int FMT, int BN_, bool PAIR_>
struct Config {
  static constexpr bool PAIR = PAIR_;
  static constexpr int BN = BN_;
  static constexpr bool MX = OP == kMx4;
  // operands read across K: the weights of the gradient of x, both of the gradient of w
  static constexpr bool A_MN = OP == kGradRows || OP == kGradWeights;
  static constexpr bool B_MN = OP == kGradWeights;
  static constexpr int CTAS = PAIR ? 2 : 1;               // CTAs a tile is laid across
  static constexpr int BLOCK_K = MX ? 256 : 64;          // K elements of a stage
  static constexpr int MMA_K = MX ? 64 : 16;             // of one MMA: 32 bytes
  static constexpr int B_ROWS = BN / CTAS;               // N rows a CTA stages
  // grouped rows (gradient of w: columns of dy, one slab) of one copy
  static constexpr int BOX = OP == kGradWeights || BN >= 256 ? 64 : 32;
  static constexpr uint32_t B_BYTES = B_ROWS * kRowBytes;
  static constexpr uint32_t BOX_BYTES = BOX * kRowBytes;
  static constexpr int KG = FMT == kNv ? 4 : 2;          // scale words of a stage
  static constexpr int NB = (BN + 127) / 128;            // 128-row scale tiles of the N side
  static constexpr uint32_t SFA_BYTES = MX ? KG * kScaleTile : 0;
  static constexpr uint32_t SFB_BYTES = MX ? NB * KG * kScaleTile : 0;
  static constexpr uint32_t STAGE = kABytes + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int STAGES = MX ? 5 : 6;
  // Two accumulators and the scales in 512 TMEM columns: with 256-column
  // accumulators beside scales the two share their last and first columns
  // (48 or 24).  The epilogue takes those first, and the next tile's MMAs
  // start once it has, while it works on the rest.
  static constexpr uint32_t SF_COLS = MX ? KG * 4 + KG * 4 * NB : 0;
  static constexpr bool SHARED = 2 * BN + SF_COLS > 512;
  static constexpr uint32_t TMEM = 2 * BN + SF_COLS <= 256 ? 256 : 512;
  static constexpr uint32_t ACC1 = SHARED ? TMEM - SF_COLS - BN : BN;  // first column of the second accumulator
  static constexpr uint32_t SF_BASE = TMEM - SF_COLS;
  static_assert(!SHARED || (BN == 256 && ACC1 >= 192), "the shared columns lie in two blocks of 32 of each accumulator");
  // full, empty, tail and peer tail per stage (the tails: gradient of w);
  // accumulator full and empty; drain
  static constexpr int BARS = (OP == kGradWeights ? 4 : 2) * STAGES + 5;
  static constexpr uint32_t OUT_STAGE = 8192;  // of each side of the epilogue: 32 rows of 128 16-bit columns
  static constexpr uint32_t CTRL = 384;  // barriers, TMEM address, abort flag; from 256 on the loaders' last issues
  static constexpr uint32_t FIXED = 1024 + STAGES * STAGE + 2 * OUT_STAGE + CTRL;
  static_assert(8 * BARS + 8 <= 256 && 256 + 2 * 8 * STAGES <= CTRL, "control words");
  static_assert(FIXED + 4 * kTableInts <= 232448, "shared memory");
  static_assert(BN % 32 == 0 && B_ROWS % BOX == 0, "copies of whole boxes fill a stage exactly");
};

struct ProductParams {
  int T, M, N, K;
  int groups, tiles_m, tiles_n;  // tiles_n: of a group (gradient of w only)
  FastDiv div_tail;              // tiles_m mod kSuper
  bool sort;                     // groups by falling cost of a tile
  const int32_t* offsets;
  void* out;
  int out_type;
  int64_t ldo, out_group;
  float alpha;
  bool vec;        // 16-byte stores: a 16-bit output whose rows are 16-byte aligned
  uint64_t timeout_ns;  // limit of a pipeline wait: what a whole tile's stages may take, and 2 s
  int withhold_kb, withhold_cta;  // the stage that test runs withhold (of that CTA's first tile), or -1
  uint32_t idesc;  // types, majorness, M; N is filled in per tile
};

// One lane of a converged warp.  The compiler then knows that a single thread
// runs the branch, and takes tcgen05's warp-uniform operands from it directly.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// A value that is the same in every lane, made so for the compiler: loops and
// addresses built on it then run on the warp's uniform registers, which TMA
// and MMA instructions take their operands from.  Inside a one-thread branch
// every operand is moved over for every instruction (a loaded stage 380 cycles
// of the loader, 336 so).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

__device__ __forceinline__ bool mbar_test_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Arrival on a barrier of the pair that passes on no memory of this thread's
// (accumulators handed back: their reads are complete).  A release at cluster
// scope waits until the thread's global stores are performed, the previous
// block's among them: 1600 cycles between a tile's last MMA and the next one's
// first.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// Shared-memory matrix descriptors, 128-byte swizzle, version 1.  K-major:
// rows of 128 bytes of K, 8-row groups 1024 bytes apart.  MN-major: slabs of
// 64 rows-or-columns (128 bytes) by 64 of K; 8 of K are 1024 bytes (the
// stride offset), the next 64 rows-or-columns a slab of 8 KB away (the
// leading offset).
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  constexpr uint64_t lead = MN ? 8192 >> 4 : 1;
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (lead << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// Of one 512-byte scale tile: 32 rows of 16 bytes, 8-row groups 128 bytes apart, no swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (static_cast<uint64_t>(128 >> 4) << 32) |
         (1ull << 46);
}

// One scale tile into four TMEM columns, the same in every lane quadrant.
// Copies and MMAs issued by one thread run in the order they were issued.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  if (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

#define OZK_MMA_SCALED(GROUP, KIND)                                                                              \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                 \
               "tcgen05.mma." GROUP "." KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                  \
               "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)                                          \
               : "memory")
template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, uint32_t acc) {
  if (FMT == kNv) {
    if (PAIR) OZK_MMA_SCALED("cta_group::2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
    else OZK_MMA_SCALED("cta_group::1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
  } else {
    if (PAIR) OZK_MMA_SCALED("cta_group::2", "kind::mxf4.block_scale.scale_vec::2X");
    else OZK_MMA_SCALED("cta_group::1", "kind::mxf4.block_scale.scale_vec::2X");
  }
}
#undef OZK_MMA_SCALED

// ---------------------------------------------------------------------------
// The schedule
// ---------------------------------------------------------------------------
// Group table in shared memory, in the order the groups' tiles run: first
// tile, first row, rows, and number of each group; after the last the number
// of tiles.
struct Group {
  int first, row0, rows, e;
};
static_assert(sizeof(Group) == 16, "one shared-memory load");

// Output rows of a tile of a group with `total` of them: equal tiles, not full
// ones and a rest.  A tile's MMAs and copies take time in proportion to its
// rows, and equal ones fill the SMs evenly.  4-bit rows keep whole tiles, as
// their scale tiles lie.
template <typename C, ProductOp OP>
__device__ __forceinline__ int tile_rows(int total) {
  if (C::MX) return C::BN;
  const unsigned n = static_cast<unsigned>(total), tiles = (n + C::BN - 1) / C::BN;
  const unsigned rows = tiles <= 1 ? n : (n + tiles - 1) / tiles;
  return static_cast<int>((rows + 31) / 32 * 32);
}

// Fills the table (all threads).  Where any offset lies outside [0, T] or runs
// backwards, that is latched as a fault and the groups are cut to a rising
// sequence inside [0, T]: every access stays inside the operands, no row
// belongs to two groups, and the tiles' count stays the one the host allowed
// for.  Where tiles run in several waves, the
// groups run by falling cost of a tile (its rows; for the gradient of w, the
// rows it sums), so that the last wave, which not every CTA gets a tile of, is
// that of the cheapest tiles.
template <typename C, ProductOp OP>
__device__ __forceinline__ void build_groups(const ProductParams& p, Group* g) {
  const int tid = threadIdx.x, lane = tid & 31;
  auto offset = [&](int e) { return p.offsets ? p.offsets[e] : e ? p.T : 0; };
  bool bad = false;
  auto group_at = [&](int e, int from) {  // `from`: the end of the group before it, where offsets are bad
    const int first = offset(e), end = offset(e + 1);
    const int lo = min(max(first, from), p.T), hi = min(max(end, lo), p.T);
    bad |= lo != first || hi != end;
    return Group{0, lo, hi - lo, e};
  };
  auto tiles_of = [&](int rows) {
    return (OP == kGradWeights ? p.tiles_n : static_cast<int>((static_cast<unsigned>(rows) + C::BN - 1) / C::BN)) * p.tiles_m;
  };
  if (p.groups == 1) {
    if (tid == 0) {
      g[0] = group_at(0, 0);
      g[1].first = tiles_of(g[0].rows);
      if (bad) atomicOr(&g_status, 2);
    }
    return;
  }
  for (int e = tid; e < p.groups; e += kThreads) g[e] = group_at(e, 0);
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      atomicOr(&g_status, 2);
      int from = 0;
      for (int e = 0; e < p.groups; ++e) {
        g[e] = group_at(e, from);
        from = g[e].row0 + g[e].rows;
      }
    }
    __syncthreads();
  }
  if (p.sort) {  // at most kSortGroups groups: one thread each
    int place = 0;
    Group mine = {};
    auto cost = [&](int rows) { return OP == kGradWeights ? rows : tile_rows<C, OP>(rows); };
    if (tid < p.groups) {
      mine = g[tid];
      const int own = cost(mine.rows);
      for (int e = 0; e < p.groups; ++e) {
        const int other = cost(g[e].rows);
        place += other > own || (other == own && e < tid);
      }
    }
    __syncthreads();
    if (tid < p.groups) g[place] = mine;
    __syncthreads();
  }
  if (tid < 32) {
    int carry = 0;
    for (int b = 0; b < p.groups; b += 32) {
      const int at = b + lane;
      const int tiles = at < p.groups ? tiles_of(g[at].rows) : 0;
      int sum = tiles;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += v;
      }
      if (at < p.groups) g[at].first = carry + sum - tiles;
      carry += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) g[p.groups].first = carry;
  }
}

// The tiles of one CTA (pair) `me` of `all`: one of each wave, up the CTAs and
// down again in turn, which evens out costs that fall along the schedule.
// -1 past the last tile.
struct Walk {
  int me, all, tiles;
  __device__ __forceinline__ int at(int wave) const {
    const int u = wave * all + (wave & 1 ? all - 1 - me : me);
    return u < tiles ? u : -1;
  }
};

struct Tile {  // the same in every lane
  int e, row0;     // group and its first row
  int m0, n0;      // first output column; first output row within the group
  int n;           // output rows of the tile
  int half;        // N rows of each CTA (all of them on a single CTA), MMA N = CTAS * half
  int k, blocks;   // terms, and stages they take
};

// Tile u of the schedule; `at` is its group's place in the table.  Within a
// group the tiles run in super rows of kSuper tile columns of the output,
// row by row: what runs together shares a few operands' tiles in L2.
template <typename C, ProductOp OP>
__device__ __forceinline__ Tile tile_at(const ProductParams& p, const Group* g, int u, int& at) {
  while (u >= uniform(g[at + 1].first)) ++at;  // u only grows
  const int4 v = *reinterpret_cast<const int4*>(g + at);
  const Group group{uniform(v.x), uniform(v.y), uniform(v.z), uniform(v.w)};
  Tile t;
  t.e = group.e;
  t.row0 = group.row0;
  const unsigned total_n = static_cast<unsigned>(OP == kGradWeights ? p.N : group.rows);
  const unsigned tn = (total_n + C::BN - 1) / C::BN;
  unsigned r = static_cast<unsigned>(u - group.first), m = 0, n;
  if (p.tiles_m > kSuper) {  // several super rows
    const unsigned super = r / kSuper / tn;
    r -= super * kSuper * tn;
    m = super * kSuper;
  }
  if (p.tiles_m - m >= kSuper) {
    n = r / kSuper;
    m += r % kSuper;
  } else {  // the last, tiles_m mod kSuper wide
    n = div_fast(r, p.div_tail);
    m += r - n * (static_cast<unsigned>(p.tiles_m) % kSuper);
  }
  t.m0 = static_cast<int>(m) * (kTileRows * C::CTAS);
  const int step = tile_rows<C, OP>(static_cast<int>(total_n));
  t.n0 = static_cast<int>(n) * step;
  t.n = min(step, static_cast<int>(total_n) - t.n0);
  t.half = C::PAIR ? (t.n + 31) / 32 * 16 : (t.n + 15) / 16 * 16;
  t.k = OP == kGradWeights ? group.rows : p.K;
  t.blocks = (t.k + C::BLOCK_K - 1) / C::BLOCK_K;
  return t;
}

// The gradient of w reduces over a group's rows: where the last MMA step
// (16 rows) reaches past the group's end, the rows after it belong to the
// next group and must not enter the sum, whatever they hold.
template <ProductOp OP>
__device__ __forceinline__ bool has_tail(const Tile& t) {
  return OP == kGradWeights && t.k % 16 != 0;
}

// ---------------------------------------------------------------------------
// Epilogue: 32 accumulator columns (output rows n0 .. n0 + 31) of 32 TMEM
// lanes (consecutive output columns).
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ T out_of(float v) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __float2bfloat16_rn(v);
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
  else return v;
}

template <typename T>
__device__ __forceinline__ void store_block(T* out, int64_t ldo, int rows, bool in_m, const uint32_t (&v)[32], float alpha) {
  if (!in_m) return;
  if (rows >= 32) {
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      *out = out_of<T>(__uint_as_float(v[c]) * alpha);
      out += ldo;
    }
  } else {
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (c < rows) out[c * ldo] = out_of<T>(__uint_as_float(v[c]) * alpha);
  }
}

// The same block of a 16-bit output with rows that start on 16 bytes.  A lane
// of TMEM is an output column, so a thread that reads its lane holds values
// that lie a whole row apart in the output; stored from there they take 32
// two-byte stores.  Read in the 16 x 256-bit form, four lanes share an
// accumulator row, pairs of output rows pack into a register, and stmatrix
// writes the 8 x 8 pieces transposed.  The four warps that hold the tile's 128
// output columns of these rows put them together in shared memory (two halves
// of 64 columns, 128-byte rows, swizzled), and whole blocks that end on 16
// bytes leave by TMA stores, full lines that no warp waits for: stored by the warps, in rows of 64
// bytes, a block took 535 cycles of its 820 (8192^2 x 1024 NVFP4 37.1 -> 35.3
// us, 8192^3 151.7 -> 149.7; a token's product 0.1 us slower).
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_rows(uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15]),
                 "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7]),
                 "+r"(b[8]), "+r"(b[9]), "+r"(b[10]), "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]), "+r"(b[15])
               :
               : "memory");
}
template <typename T>
__device__ __forceinline__ uint32_t pack16(uint32_t lo, uint32_t hi, float alpha) {
  uint32_t r;
  const float l = __uint_as_float(lo) * alpha, h = __uint_as_float(hi) * alpha;
  if constexpr (std::is_same<T, __half>::value) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(h), "f"(l));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(h), "f"(l));
  return r;
}
// This warp's 32 x 32 values into the block of its four warps (quad: which
// quarter of the 128 columns).
constexpr uint32_t kOutHalf = 32 * 128;  // 64 columns of 32 rows
__device__ __forceinline__ uint32_t out_piece(int n, int chunk) {  // 16-byte piece `chunk` (0..15) of row n
  return static_cast<uint32_t>((chunk >> 3) * static_cast<int>(kOutHalf) + n * 128 + (((chunk & 7) ^ (n & 7)) * 16));
}
template <typename T>
__device__ __forceinline__ void stage_block(uint32_t block, int quad, int lane, const uint32_t (&lo)[16],
                                            const uint32_t (&hi)[16], float alpha) {
  // lane l gives the address of row l % 8 of piece l / 8: output rows 8 (2 q + l / 16) .. and columns 16 half + 8 (l / 8 % 2) ..
  const int piece = lane >> 3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t(&v)[16] = half ? hi : lo;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t addr = block + out_piece(8 * (2 * q + (piece >> 1)) + (lane & 7), 4 * quad + 2 * half + (piece & 1));
      asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                   "r"(pack16<T>(v[8 * q], v[8 * q + 1], alpha)), "r"(pack16<T>(v[8 * q + 2], v[8 * q + 3], alpha)),
                   "r"(pack16<T>(v[8 * q + 4], v[8 * q + 5], alpha)), "r"(pack16<T>(v[8 * q + 6], v[8 * q + 7], alpha))
                   : "memory");
    }
  }
}
// `rows` rows and `cols` columns of a block by ordinary stores (a group's or
// the matrix's edge, where a whole box would reach past it): this warp's 8 rows.
__device__ __forceinline__ void store_edge(uint16_t* out, int64_t ldo, int rows, int cols, uint32_t block, int quad, int lane) {
  const int chunk = lane & 15;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = 8 * quad + 2 * i + (lane >> 4);
    if (n >= rows || 8 * chunk >= cols) continue;
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(block + out_piece(n, chunk))
                 : "memory");
    uint16_t* dst = out + n * ldo + 8 * chunk;
    if (8 * chunk + 8 <= cols) {
      *reinterpret_cast<uint4*>(dst) = w;
    } else {
      const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (8 * chunk + j < cols) dst[j] = static_cast<uint16_t>(e[j / 2] >> (16 * (j & 1)));
    }
  }
}

// ---------------------------------------------------------------------------
// The abort path
// ---------------------------------------------------------------------------
// A loader's last issue of a stage's copies: its number (from 1; 0: none), the
// bytes of this CTA, and for a group's last block, which arrives on the tail
// barrier, bit 31 and the parity of that barrier's phase in bit 30.  Lane s of
// each loader warp holds that of stage s until the roles end, so that a stage
// costs the loaders no store.
struct alignas(8) Issue {
  uint32_t number, word;
};
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Waits (each wait bounded) until every copy issued into this CTA's stages is
// in; one thread, once every role of the CTA and its peer has stopped.  A
// stage's earlier uses are over, or it would not have been issued again.  On a
// pair the copies of both CTAs arrive on the leader's barrier, armed by the
// leader for both: where only one of the two issued the stage's last use, the
// leader stands in for the other.
__device__ __forceinline__ Issue later(const Issue& a, const Issue& b) { return a.number > b.number ? a : b; }
template <typename C>
__device__ __forceinline__ void drain_copies(const Issue* issues, uint32_t full0, uint32_t tail0, bool leader) {
  for (int s = 0; s < C::STAGES; ++s) {
    const Issue own = later(issues[s], issues[C::STAGES + s]);
    const bool tail = own.word >> 31;
    if (tail) mbar_wait_drain(tail0 + 8 * s, (own.word >> 30) & 1u);
    bool full = own.number != 0 && !tail;
    uint32_t number = own.number;
    if (C::PAIR) {
      if (!leader) continue;
      const uint32_t remote = cluster_addr(smem_u32(issues + s), 1), other = remote + 8 * C::STAGES;
      const Issue peer = later({ld_shared_cluster(remote), ld_shared_cluster(remote + 4)},
                               {ld_shared_cluster(other), ld_shared_cluster(other + 4)});
      if (peer.number > own.number) {
        full = !(peer.word >> 31);
        number = peer.number;
        if (full) mbar_expect_tx(full0 + 8 * s, peer.word & 0xFFFFFu);
      } else if (peer.number < own.number && full) {
        mbar_complete_tx(full0 + 8 * s, own.word & 0xFFFFFu);
      }
    }
    if (full) mbar_wait_drain(full0 + 8 * s, ((number - 1) / C::STAGES) & 1u);
  }
}

// Barriers of the four epilogue warps of a side, and their agreement on a
// wait's outcome (each wait is bounded, so all four get here).
__device__ __forceinline__ void side_sync(int side) {
  asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(1 + side) : "memory");
}
__device__ __forceinline__ bool side_all(int side, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + side), "r"(static_cast<uint32_t>(ok))
      : "memory");
  return r != 0;
}

template <ProductOp OP, int FMT, int BN, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmR,
                   const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSR,
                   const __grid_constant__ CUtensorMap tmO, const ProductParams p) {
  using C = Config<OP, FMT, BN, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t sA = smem_u32(smem);
  const uint32_t sB = sA + C::STAGES * kABytes;
  const uint32_t sSA = sB + C::STAGES * C::B_BYTES;
  const uint32_t sSB = sSA + C::STAGES * C::SFA_BYTES;
  uint8_t* out_stage = smem + C::STAGES * C::STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(out_stage + 2 * C::OUT_STAGE);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Issue* issues = reinterpret_cast<Issue*>(reinterpret_cast<uint8_t*>(bars) + 256);
  Group* g = reinterpret_cast<Group*>(reinterpret_cast<uint8_t*>(bars) + C::CTRL);

  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0;               // in a pair
  const bool leader = rank == 0;
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * C::STAGES;
  const uint32_t accf0 = empty0 + 8 * C::STAGES;
  const uint32_t acce0 = accf0 + 16;
  const uint32_t drain = acce0 + 16;
  const uint32_t tail0 = drain + 8;               // this CTA's part of a group's last block is in
  const uint32_t peer0 = tail0 + 8 * C::STAGES;   // leader: the peer has cleared its part

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
      if (OP == kGradWeights) {
        mbar_init(tail0 + 8 * s, 1);
        mbar_init(peer0 + 8 * s, 1);
      }
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, C::CTAS * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmR);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), C::TMEM);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), C::TMEM);
      tmem_relinquish();
    }
  }
  // The set-up above touches nothing that the kernel before this one writes,
  // and without offsets neither does the table; loads and stores do.
  if (p.offsets) grid_dependency_sync();
  build_groups<C, OP>(p, g);
  tc_fence_before();
  __syncthreads();
  if (C::CTAS > 1) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = static_cast<uint32_t>(uniform(static_cast<int>(*reinterpret_cast<volatile uint32_t*>(tmem_slot))));
  const Walk walk{static_cast<int>(blockIdx.x) / C::CTAS, static_cast<int>(gridDim.x) / C::CTAS,
                  uniform(g[p.groups].first)};

  if (warp == 0 || warp == 3) {
    // ------------------------------ TMA producers ------------------------------
    // Two warps fill the stages in turn: filling one takes a warp about 330
    // cycles (waits, barrier, two to four copies), more than a stage of a
    // small tile takes to arrive or to be used.
    int stage = 0, e = 0, issued = 0;
    const int turn = warp == 3;
    uint32_t phase = 0, tails = 0;
    Issue last = {0, 0};  // of stage `lane`
    int withheld = static_cast<int>(blockIdx.x) == p.withhold_cta ? p.withhold_kb : -1;  // block of the first tile
    bool ok = true, waited = p.offsets != nullptr;
    for (int wave = 0, u; ok && (u = walk.at(wave)) >= 0; ++wave) {
      const Tile t = tile_at<C, OP>(p, g, u, e);
      const int m0 = t.m0 + static_cast<int>(rank) * kTileRows;
      const int n0 = t.n0 + static_cast<int>(rank) * t.half;
      const int boxes = (t.half + C::BOX - 1) / C::BOX;
      const uint32_t bytes = kABytes + static_cast<uint32_t>(boxes) * C::BOX_BYTES + C::SFA_BYTES + C::SFB_BYTES;
      for (int kb = 0; kb < t.blocks; ++kb) {
        const bool mine = (issued & 1) == turn;
        if (mine && !warp_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.timeout_ns)) {
          ok = false;
          break;
        }
        if (!waited) grid_dependency_sync();  // the first tile is laid out by now
        waited = true;
        const bool clear = has_tail<OP>(t) && kb == t.blocks - 1;
        const bool issue = mine && kb != withheld;
        if (issue && elect_one()) {
          uint32_t bar = full0 + 8 * stage;
          if (clear) {  // warp 2 passes the stage on once it has cleared the rows
            bar = tail0 + 8 * stage;
            mbar_expect_tx(bar, bytes);
          } else if (!PAIR) {
            mbar_expect_tx(bar, bytes);
          } else {
            if (leader) mbar_expect_tx(bar, 2 * bytes);
            bar = cluster_addr(bar, 0);
          }
          auto load2 = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1) {
            if (PAIR) tma_load_2d_pair(dst, map, c0, c1, clear ? cluster_addr(bar, rank) : bar);
            else tma_load_2d(dst, map, c0, c1, bar);
          };
          auto load3 = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2) {
            if (PAIR) tma_load_3d_pair(dst, map, c0, c1, c2, bar);
            else tma_load_3d(dst, map, c0, c1, c2, bar);
          };
          const uint32_t a = sA + stage * kABytes, b = sB + stage * C::B_BYTES;
          const int k0 = kb * C::BLOCK_K;
          if constexpr (OP == kForward) load3(a, &tmW, k0, m0, t.e);
          if constexpr (OP == kMx4) load3(a, &tmW, k0 / 2, m0, t.e);
          if constexpr (OP == kGradRows) {
            load3(a, &tmW, m0, k0, t.e);
            load3(a + kABytes / 2, &tmW, m0 + 64, k0, t.e);
          }
          if constexpr (OP == kGradWeights) {
            load2(a, &tmW, m0, t.row0 + k0);
            load2(a + kABytes / 2, &tmW, m0 + 64, t.row0 + k0);
          }
          for (int j = 0; j < boxes; ++j) {
            if constexpr (OP == kGradWeights) load2(b + j * C::BOX_BYTES, &tmR, n0 + C::BOX * j, t.row0 + k0);
            else load2(b + j * C::BOX_BYTES, &tmR, C::MX ? k0 / 2 : k0, t.row0 + n0 + C::BOX * j);
          }
          if constexpr (C::MX) {
            // scale tiles: of these weight rows, and of the tile's rows (on a pair both CTAs take all of them)
            const int wrow = static_cast<int>(static_cast<int64_t>(t.e) * p.M / 128);
            load3(sSA + stage * C::SFA_BYTES, &tmSW, 0, kb * C::KG, wrow + t.e + m0 / 128);
            load3(sSB + stage * C::SFB_BYTES, &tmSR, 0, kb * C::KG, t.row0 / 128 + t.e + t.n0 / 128);
          }
        }
        if (issue && lane == stage)
          last = {static_cast<uint32_t>(issued) + 1u, bytes | (clear ? 0x80000000u | ((tails >> stage) & 1u) << 30 : 0u)};
        if (clear) tails ^= 1u << stage;
        ++issued;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      withheld = -1;
    }
    if (lane < C::STAGES) issues[turn * C::STAGES + lane] = last;
    __syncwarp();
  } else if (warp == 1 && leader) {
    // ------------------------------ MMA issuer ------------------------------
    // first TMEM column of a stage's scale word: of the M side, and of the N side
    auto sfa_of = [&](int word) { return tmem_base + C::SF_BASE + 4u * word; };
    auto sfb_of = [&](int word) { return tmem_base + C::SF_BASE + 4u * C::KG + 4u * C::NB * word; };
    if (!p.offsets) grid_dependency_sync();  // reads nothing, but its waits are for this kernel's copies alone
    int stage = 0, e = 0, ab = 0;
    uint32_t phase = 0, aphase = 0;
    bool ok = true, first = true;
    for (int wave = 0, u; ok && (u = walk.at(wave)) >= 0; ++wave) {
      const Tile t = tile_at<C, OP>(p, g, u, e);
      if (t.blocks == 0) continue;
      // free: this accumulator's previous tile (two ago) is out; or, with
      // shared columns, the tile before this one is out of them
      if (C::SHARED ? (!first && !warp_wait(acce0 + 8 * (ab ^ 1), ab ? aphase : aphase ^ 1u, abort_flag, p.timeout_ns))
                    : !warp_wait(acce0 + 8 * ab, aphase ^ 1u, abort_flag, p.timeout_ns))
        break;
      first = false;
      tc_fence_after();
      const uint32_t d = tmem_base + (ab ? C::ACC1 : 0u);
      const uint32_t idesc = p.idesc | (static_cast<uint32_t>(t.half * C::CTAS >> 3) << 17);
      for (int kb = 0; kb < t.blocks; ++kb) {
        if (!warp_wait(full0 + 8 * stage, phase, abort_flag, p.timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t da = operand_desc<C::A_MN>(sA + stage * kABytes);
        const uint64_t db = operand_desc<C::B_MN>(sB + stage * C::B_BYTES);
        const int steps = min(4, (t.k - kb * C::BLOCK_K + C::MMA_K - 1) / C::MMA_K);
        if (elect_one()) {
          if constexpr (C::MX) {
#pragma unroll
            for (int i = 0; i < C::KG; ++i) {
              copy_scales<PAIR>(sfa_of(i), scale_desc(sSA + stage * C::SFA_BYTES + i * kScaleTile));
#pragma unroll
              for (int r = 0; r < C::NB; ++r)
                copy_scales<PAIR>(sfb_of(i) + 4 * r,
                                  scale_desc(sSB + stage * C::SFB_BYTES + (r * C::KG + i) * kScaleTile));
            }
          }
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if (s >= steps) continue;
            const uint32_t acc = (kb > 0 || s > 0) ? 1u : 0u;
            if constexpr (C::MX) {
              const int word = FMT == kNv ? s : s / 2;             // scale word of the step
              const uint32_t id = FMT == kNv ? 0u : 2u * (s & 1);  // its first byte
              mma_scaled<FMT, PAIR>(d, da + 2ull * s, db + 2ull * s, idesc | (id << 4) | (id << 29), sfa_of(word),
                                    sfb_of(word), acc);
            } else {
              // 32 bytes of K, or 16 rows of 128 bytes
              constexpr uint64_t step_a = C::A_MN ? (16 * kRowBytes) >> 4 : 2;
              constexpr uint64_t step_b = C::B_MN ? (16 * kRowBytes) >> 4 : 2;
              if (PAIR) mma_f16_pair(d, da + step_a * s, db + step_b * s, idesc, acc);
              else mma_f16(d, da + step_a * s, db + step_b * s, idesc, acc);
            }
          }
          if (PAIR) mma_commit_both(empty0 + 8 * stage);
          else mma_commit(empty0 + 8 * stage);
        }
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elect_one()) {
        if (PAIR) mma_commit_both(accf0 + 8 * ab);
        else mma_commit(accf0 + 8 * ab);
      }
      ab ^= 1;
      if (ab == 0) aphase ^= 1u;
    }
    if (elect_one()) {
      if (PAIR) mma_commit_local(drain);
      else mma_commit(drain);
      mbar_wait_drain(drain, 0);
    }
    __syncwarp();
  } else if (warp == 2 && OP == kGradWeights) {
    // ------------------------------ tails ------------------------------
    int e = 0;
    unsigned pos = 0;     // stages the producer has filled before this tile
    unsigned waited = 0;  // of them, before the last tile with a tail
    uint32_t tails = 0;
    for (int wave = 0, u; (u = walk.at(wave)) >= 0; ++wave) {
      const Tile t = tile_at<C, OP>(p, g, u, e);
      if (t.blocks > 0 && has_tail<OP>(t)) {
        const int stage = static_cast<int>((pos + t.blocks - 1) % C::STAGES);
        // this warp is ahead of the others by the tiles without a tail since the last one
        const uint64_t limit = p.timeout_ns + kStageNs * (pos + static_cast<unsigned>(t.blocks) - waited);
        if (!warp_wait(tail0 + 8 * stage, (tails >> stage) & 1u, abort_flag, limit)) break;
        waited = pos + static_cast<unsigned>(t.blocks);
        tails ^= 1u << stage;
        const int r0 = t.k % 64;                 // first row past the group's end; the MMAs stop at the next 16
        const int r1 = (r0 + 15) / 16 * 16;
        const int slabs_b = (t.half + 63) / 64;
        const int chunks = (r1 - r0) * 8;        // 16-byte pieces of one slab
        for (int i = lane; i < chunks * (2 + slabs_b); i += 32) {
          const int slab = i / chunks, at = (r0 * 128) + (i - slab * chunks) * 16;
          const uint32_t base = slab < 2 ? sA + stage * kABytes + slab * 8192
                                         : sB + stage * C::B_BYTES + (slab - 2) * 8192;
          st_shared_v4(base + static_cast<uint32_t>(at), 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        // the leader passes the stage on once the peer's part is cleared too
        if (PAIR && leader) {
          if (!warp_wait(peer0 + 8 * stage, ((tails >> stage) & 1u) ^ 1u, abort_flag, p.timeout_ns)) break;
          mbar_test_cluster(peer0 + 8 * stage, ((tails >> stage) & 1u) ^ 1u);  // acquire at cluster scope
        }
        if (lane == 0) {
          if (PAIR && !leader) mbar_arrive_cluster(cluster_addr(peer0 + 8 * stage, 0));
          else mbar_arrive(full0 + 8 * stage);
        }
      }
      pos += static_cast<unsigned>(t.blocks);
    }
  } else if (warp >= 4) {
    // ------------------------------ epilogue ------------------------------
    if (!p.offsets) grid_dependency_sync();
    const int quad = warp & 3, side = (warp - 4) >> 2;  // TMEM lanes 32 quad..; every other block of 32 columns
    const uint32_t block = smem_u32(out_stage) + static_cast<uint32_t>(side) * C::OUT_STAGE;
    int e = 0, ab = 0;
    uint32_t aphase = 0;
    for (int wave = 0, u; (u = walk.at(wave)) >= 0; ++wave) {
      const Tile t = tile_at<C, OP>(p, g, u, e);
      const int64_t m = t.m0 + static_cast<int>(rank) * kTileRows + quad * 32 + lane;
      const bool in_m = m < p.M;
      int64_t at = m;
      if (OP == kGradWeights) at += t.e * p.out_group + static_cast<int64_t>(t.n0) * p.ldo;
      else at += (static_cast<int64_t>(t.row0) + t.n0) * p.ldo;
      const bool has = t.blocks > 0;
      if (has) {
        if (!side_all(side, warp_wait(accf0 + 8 * ab, aphase, abort_flag, p.timeout_ns))) break;
        tc_fence_after();
      }
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + (ab ? C::ACC1 : 0u);
      // blocks of 32 columns, alternating between the two warps of a lane
      // quadrant; of accumulator 0 with shared columns the last two first
      constexpr int kBlocks = (BN + 63) / 64;
      bool held = has;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_remote(cluster_addr(acce0 + 8 * ab, 0));
          else mbar_arrive(acce0 + 8 * ab);
        }
        held = false;
      };
#pragma unroll 1
      for (int i = 0; i < kBlocks; ++i) {
        const int c = 64 * (C::SHARED && ab == 0 ? (i + kBlocks - 1) % kBlocks : i) + 32 * side;
        const int rows = t.n - c;
        const int64_t o = at + c * p.ldo;
        if (p.vec) {
          uint32_t lo[16], hi[16];
          if (rows > 0) {
            if (has) {
              tmem_ld_rows(taddr + static_cast<uint32_t>(c), lo);
              tmem_ld_rows(taddr + static_cast<uint32_t>(c) + (16u << 16), hi);
              tmem_wait_rows(lo, hi);
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) lo[j] = hi[j] = 0u;
            }
          }
          if (held && (C::SHARED || i == kBlocks - 1)) release();
          if (rows <= 0) continue;
          const int m0 = t.m0 + static_cast<int>(rank) * kTileRows;
          const bool issuer = quad == 0 && elect_one();
          if (issuer) bulk_wait_read();  // the block's last stores have read it
          side_sync(side);
          if (p.out_type == OZK_F16) stage_block<__half>(block, quad, lane, lo, hi, p.alpha);
          else stage_block<__nv_bfloat16>(block, quad, lane, lo, hi, p.alpha);
          fence_proxy_async_smem();
          side_sync(side);
          // A bulk store leaves out columns past M in whole 16-byte pieces alone: what lies in the piece that M
          // ends in would be overwritten.
          const int cols = p.M - m0;
          if (rows >= 32 && (cols >= kTileRows || cols % 8 == 0)) {
            const int n = OP == kGradWeights ? t.n0 + c : t.row0 + t.n0 + c;
            if (issuer) {
              if (m0 < p.M) tma_store_3d(&tmO, block, m0, n, OP == kGradWeights ? t.e : 0);
              if (m0 + 64 < p.M) tma_store_3d(&tmO, block + kOutHalf, m0 + 64, n, OP == kGradWeights ? t.e : 0);
            }
          } else {
            store_edge(static_cast<uint16_t*>(p.out) + o - (m - m0), p.ldo, min(rows, 32), cols, block, quad, lane);
          }
          continue;
        }
        uint32_t v[32];
        if (rows > 0) {
          if (has) {
            tmem_ld32(taddr + static_cast<uint32_t>(c), v);
            tmem_wait_ld(v);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
          }
        }
        if (held && (C::SHARED || i == kBlocks - 1)) release();
        if (rows <= 0) continue;
        if (p.out_type == OZK_F32) store_block(static_cast<float*>(p.out) + o, p.ldo, rows, in_m, v, p.alpha);
        else if (p.out_type == OZK_F16) store_block(static_cast<__half*>(p.out) + o, p.ldo, rows, in_m, v, p.alpha);
        else store_block(static_cast<__nv_bfloat16*>(p.out) + o, p.ldo, rows, in_m, v, p.alpha);
      }
      if (has) {
        ab ^= 1;
        if (ab == 0) aphase ^= 1u;
      }
    }
    // the stores in flight finish before the CTA's shared memory goes
    if (p.vec && quad == 0) {
      if (elect_one()) bulk_wait_all();
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (C::CTAS > 1) {
    if (threadIdx.x == 0 && *abort_flag)  // the peer stops too, its own limit aside
      st_shared_cluster(cluster_addr(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u), 1u);
    __syncwarp();
    cluster_sync();
  }
  if (*abort_flag) {  // of either CTA of a pair; nothing is issued any more
    if (threadIdx.x == 0) drain_copies<C>(issues, full0, tail0, leader);
    __syncthreads();
    if (C::CTAS > 1) cluster_sync();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem_base, C::TMEM);
    else tmem_dealloc(tmem_base, C::TMEM);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
bool make_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const int64_t* dims,
              const int64_t* strides, const uint32_t* box, bool swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t d[3], s[2];
  cuuint32_t b[3];
  const cuuint32_t step[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = static_cast<cuuint64_t>(std::max<int64_t>(dims[i], 1));
    b[i] = box[i];
    if (i) s[i - 1] = static_cast<cuuint64_t>(strides[i - 1]);
  }
  return enc(map, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), d, s, b, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Once per device and kernel: the shared-memory opt-in, and the number of
// clusters that fit the GPU at once.
cudaError_t setup(const void* kernel, size_t smem, int cluster, int* resident) {
  struct Setup {
    cudaError_t err;
    int resident;
  };
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, Setup> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  auto it = done.find({dev, kernel});
  if (it == done.end()) {
    Setup s{cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)), 0};
    if (s.err == cudaSuccess && cluster > 1) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
      cfg.blockDim = dim3(kThreads);
      cfg.gridDim = dim3(static_cast<unsigned>(cluster));
      cfg.dynamicSmemBytes = smem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      s.err = cudaOccupancyMaxActiveClusters(&s.resident, kernel, &cfg);
      if (s.err == cudaSuccess && s.resident < 1) s.err = cudaErrorInvalidConfiguration;
    }
    it = done.emplace(std::make_pair(dev, kernel), s).first;
  }
  *resident = it->second.resident;
  return it->second.err;
}

// What ozk_withhold_next_product asked of this host thread's next product.
struct Withhold {
  int pairs, cta, kblock;
  uint32_t timeout_us;  // 0: nothing asked
};
thread_local Withhold g_withhold = {};

template <ProductOp OP, int FMT, int BN, bool PAIR>
cudaError_t launch(const Product& q, int num_sms, cudaStream_t stream) {
  using C = Config<OP, FMT, BN, PAIR>;
  ProductParams p = {};
  p.T = static_cast<int>(q.T);
  p.M = static_cast<int>(q.M);
  p.N = static_cast<int>(q.N);
  p.K = static_cast<int>(q.K);
  p.groups = q.groups;
  p.offsets = q.offsets;
  p.out = q.out;
  p.out_type = q.out_type;
  p.ldo = q.ldo;
  p.out_group = q.out_group;
  p.alpha = q.K ? q.alpha : 1.0f;  // a sum of no terms is zero, whatever alpha
  p.vec = q.out_type != OZK_F32 && reinterpret_cast<uintptr_t>(q.out) % 16 == 0 && q.ldo % 8 == 0 &&
          (OP != kGradWeights || q.groups == 1 || q.out_group % 8 == 0);
  const int64_t terms = OP == kGradWeights ? q.T : q.K;
  p.timeout_ns = kTimeoutNs + kStageNs * static_cast<uint64_t>(terms / C::BLOCK_K);
  p.withhold_kb = -1;
  if (g_withhold.timeout_us != 0) {
    p.timeout_ns = 1000ull * g_withhold.timeout_us;
    p.withhold_kb = g_withhold.kblock;
    p.withhold_cta = g_withhold.cta;
    g_withhold.timeout_us = 0;
  }
  p.tiles_m = static_cast<int>((q.M + (kTileRows * C::CTAS) - 1) / (kTileRows * C::CTAS));
  p.tiles_n = static_cast<int>((q.N + C::BN - 1) / C::BN);
  p.div_tail = fast_div(p.tiles_m % kSuper);
  // D fp32; types; MN-major operands; M of the MMA
  p.idesc = static_cast<uint32_t>(kTileRows * C::CTAS >> 4) << 24;
  if (C::MX) p.idesc |= (1u << 7) | (1u << 10) | (FMT == kMx ? 1u << 23 : 0u);
  else
    p.idesc |= (1u << 4) | (q.dtype == OZK_BF16 ? (1u << 7) | (1u << 10) : 0u) | (C::A_MN ? 1u << 15 : 0u) |
               (C::B_MN ? 1u << 16 : 0u);

  CUtensorMap tmW, tmR, tmSW, tmSR, tmO;
  std::memset(&tmW, 0, sizeof tmW);
  std::memset(&tmR, 0, sizeof tmR);
  std::memset(&tmSW, 0, sizeof tmSW);
  std::memset(&tmSR, 0, sizeof tmSR);
  std::memset(&tmO, 0, sizeof tmO);
  const bool loads = q.T > 0 && q.K != 0;  // otherwise no tile has a term, and nothing is read
  if (loads && !C::MX) {
    const CUtensorMapDataType type = q.dtype == OZK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const int64_t inner_rows = OP == kGradWeights ? q.N : q.K;
    const int64_t dims_b[2] = {inner_rows, q.T}, strides_b[1] = {2 * q.ld_rows};
    const uint32_t box_b[2] = {64, static_cast<uint32_t>(C::BOX)};
    if (!make_map(&tmR, type, 2, q.rows, dims_b, strides_b, box_b, true)) return cudaErrorInvalidValue;
    bool ok;
    if (OP == kGradWeights) {
      const int64_t dims[2] = {q.M, q.T}, strides[1] = {2 * q.ld_other};
      const uint32_t box[2] = {64, 64};
      ok = make_map(&tmW, type, 2, q.other, dims, strides, box, true);
    } else {
      const int64_t dims[3] = {OP == kForward ? q.K : q.M, OP == kForward ? q.M : q.K, q.groups};
      const int64_t strides[2] = {2 * q.ld_other, 2 * q.other_group};
      const uint32_t box[3] = {64, OP == kForward ? 128u : 64u, 1};
      ok = make_map(&tmW, type, 3, q.other, dims, strides, box, true);
    }
    if (!ok) return cudaErrorInvalidValue;
  }
  if (loads && C::MX) {
    const int64_t half = ozk_kpad(q.K) / 2, kg = mx4_kgroups(q.K, FMT);
    const int64_t dims_a[3] = {half, q.M, q.groups}, strides_a[2] = {half, half * q.M};
    const uint32_t box_a[3] = {kRowBytes, 128u, 1};
    const int64_t dims_b[2] = {half, q.T}, strides_b[1] = {half};
    const uint32_t box_b[2] = {kRowBytes, static_cast<uint32_t>(C::BOX)};
    const int64_t strides_s[2] = {kScaleTile, kScaleTile * kg};
    const int64_t dims_sa[3] = {kScaleTile / 4, kg, mx4_row_blocks(q.b.rows, q.b.groups)};
    const int64_t dims_sb[3] = {kScaleTile / 4, kg, mx4_row_blocks(q.T, q.groups)};
    const uint32_t box_sa[3] = {kScaleTile / 4, C::KG, 1};
    const uint32_t box_sb[3] = {kScaleTile / 4, C::KG, C::NB};
    if (!make_map(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, q.b.codes, dims_a, strides_a, box_a, true) ||
        !make_map(&tmR, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q.a.codes, dims_b, strides_b, box_b, true) ||
        !make_map(&tmSW, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, q.b.scales, dims_sa, strides_s, box_sa, false) ||
        !make_map(&tmSR, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, q.a.scales, dims_sb, strides_s, box_sb, false))
      return cudaErrorInvalidValue;
  }
  if (p.vec) {
    const int64_t dims[3] = {q.M, OP == kGradWeights ? q.N : q.T, OP == kGradWeights ? q.groups : 1};
    const int64_t strides[2] = {2 * q.ldo, OP == kGradWeights && q.groups > 1 ? 2 * q.out_group : 2 * q.ldo * dims[1]};
    const uint32_t box[3] = {64, 32, 1};
    if (!make_map(&tmO, q.out_type == OZK_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q.out,
                  dims, strides, box, true))
      return cudaErrorInvalidValue;
  }
  auto kernel = product_kernel<OP, FMT, BN, PAIR>;
  const size_t table = (static_cast<size_t>(q.groups) + 1) * sizeof(Group);
  int resident = 0;
  cudaError_t e = setup(reinterpret_cast<const void*>(kernel),
                        C::FIXED + kTableInts * sizeof(int), C::CTAS, &resident);
  if (e != cudaSuccess) return e;
  // no more CTAs than there can be tiles; how many there are only the offsets say
  int64_t tiles = p.tiles_m;
  if (OP == kGradWeights) tiles *= static_cast<int64_t>(p.tiles_n) * q.groups;
  else tiles *= std::min<int64_t>(q.T, q.T / C::BN + q.groups);
  if (tiles == 0) return cudaSuccess;
  int64_t slots = C::CTAS > 1 ? std::min(num_sms / C::CTAS, resident) : num_sms;
  p.sort = tiles > slots && q.groups > 1 && q.groups <= kSortGroups;
  slots = std::min(slots, tiles);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(slots * C::CTAS));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::FIXED + table;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see grid_dependency_sync
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (C::CTAS > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {C::CTAS, 1, 1};
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, tmW, tmR, tmSW, tmSR, tmO, p);
}

// The form of the tiles, by modelled time: waves of tiles times (stages of a
// tile x cycles of a stage + a tile's fixed cycles), for a CTA pair's tile of
// 256 columns by up to 256 rows and for one CTA's of 128 by up to 128; a
// launch of pairs starts 2000 cycles later.  Rows per group are taken as
// their mean (the offsets are on the device).  The constants are measured: a
// stage takes about 330 cycles (4-bit 400) to issue however few its rows; with
// full tiles a pair's takes the 540 (550) of its MMAs and copies, a CTA's the
// 450 (510) that 32 (36) KB take from L2 with every SM loading.  Over 48
// sizes of all the operations, up to 8192 rows in 1 to 32 groups, the choice
// takes as long as the better of the two (within 0.2%), pairs alone 15% longer,
// single CTAs alone 5%, and more where it counts (pairs and single): 8192^3
// NVFP4 154 and 234 us; 16 groups of 512 rows, 4096 -> 2048 bf16, 92 and 108;
// but 1000 x 1537 x 2090 MXFP4 to fp32 8.2 and 6.2, and 32 rows in 32 groups,
// 4096 -> 2048 NVFP4, 30.0 and 28.5.
template <ProductOp OP, int FMT>
cudaError_t choose(const Product& q, int num_sms, cudaStream_t stream) {
  const bool mx = OP == kMx4, sum_rows = OP == kGradWeights;
  const double t = static_cast<double>(std::max<int64_t>(q.T, 1));
  const double groups = sum_rows ? q.groups : std::min(static_cast<double>(q.groups), t);
  const double rows = std::max(sum_rows ? static_cast<double>(q.N) : t / groups, 1.0);
  const double stages = std::ceil((sum_rows ? t / groups : static_cast<double>(q.K)) / (mx ? 256 : 64));
  auto cost = [&](int bn, int cols, int slots, double per_row, double fixed, double launch) {
    const double per_group = std::ceil(rows / bn);
    const double waves = std::ceil(groups * per_group * std::ceil(static_cast<double>(q.M) / cols) / slots);
    return waves * (stages * std::max(mx ? 400.0 : 330.0, per_row * rows / per_group) + fixed) + launch;
  };
  const double pair = cost(256, 256, num_sms / 2, mx ? 2.15 : 2.1, 3000, 2000);
  const double single = cost(128, 128, num_sms, mx ? 4.0 : 3.5, 2000, 0);
  const bool pairs = g_withhold.timeout_us ? g_withhold.pairs != 0 : pair < single;
  return pairs ? launch<OP, FMT, 256, true>(q, num_sms, stream)
               : launch<OP, FMT, 128, false>(q, num_sms, stream);
}

}  // namespace

static std::atomic<bool> g_any{false};  // a product was launched: without one there is no status to read

cudaError_t launch_product(const Product& q, int num_sms, cudaStream_t stream) {
  g_any.store(true, std::memory_order_relaxed);
  switch (q.op) {
    case kForward: return choose<kForward, k16>(q, num_sms, stream);
    case kGradRows: return choose<kGradRows, k16>(q, num_sms, stream);
    case kGradWeights: return choose<kGradWeights, k16>(q, num_sms, stream);
    default:
      return q.a.format == OZK_MXFP4 ? choose<kMx4, kMx>(q, num_sms, stream) : choose<kMx4, kNv>(q, num_sms, stream);
  }
}

int take_product_status(int* status) {
  *status = 0;
  return g_any.load(std::memory_order_relaxed) ? take_status(status) : OZK_OK;
}

void withhold_next_product(int pairs, int cta, int kblock, uint32_t timeout_us) {
  g_withhold = {pairs, cta, kblock, timeout_us};
}

}  // namespace ozk
