// sv_attention_mma.cu -- attention of drafted tokens over the paged cache on
// the 5th-generation tensor cores.
//
// The N nodes of a sequence and the G query heads of one cache head make R =
// N G rows that read the same keys and values.  An item is (sequence, cache
// head, up to 256 of these rows); its cached tokens are cut into tiles of
// 128, and all tiles of all items, in order, are dealt out evenly over one
// block per SM (an item counts as three tiles more, about what a segment costs
// besides its tiles), so that ragged lengths balance and a single long sequence
// uses every SM.  A block's share is a run of segments (a range of one item's
// tiles).  A segment that covers its item writes the result; any other leaves
// (maximum, sum, unnormalised output) in scratch, and a second grid joins
// them (at most two for each block, so the traffic is small).
//
// Per tile S = Q K^T (128 rows x 128 tokens) and O += P V, both by
// tcgen05.mma from shared memory filled by TMA (P from tensor memory, where
// it overlies S).  Two softmax warpgroups work in turn, each with its own S
// and O in tensor memory: with more than 128 rows each takes one half of them,
// else they take alternate tiles or, for 8-bit pools with more than 64 rows,
// each half of every tile's tokens (merged at the segment's end).
// The MMA warp issues S of one while the other computes its exponentials.
// A thread owns one row, so a row's maximum and sum need no shuffles.  The
// running maximum is only raised when a score exceeds it by 2^8: O is then
// rescaled in tensor memory; until then weights up to 2^8 (2^15 in float16) are
// exact enough in 16 bits, and the division by the sum at the end makes up for it.
//
// Weights enter the second product in the values' 16-bit type (float16: the
// largest near 2^7, so that 2^-32 of it is half of the smallest step).  8-bit pools
// go into the products as they are, by the 8-bit instructions: queries are
// scaled by a power of two a row and written as a sum of two (bfloat16) or
// three (16-bit floats) 8-bit terms of 4 significant bits each, exact but for
// elements so small that the step of the smallest codes, 2^-9, counts: half of
// it, with the largest element at 2^7 or more, is 2^-17 of that one.
// Weights need range as well as bits: behind a token that takes most of the
// weight, a long context's many small ones make up the rest of the sum.  They
// are sums of three (bfloat16) or four e5m2 terms of 3 significant bits each,
// the last one rounded, which is 2^-9 or 2^-12 of a weight at most; the largest
// is near 2^13 and the smallest step 2^-16, so that the absolute error stays
// below 2^-28 of the largest weight and scale.  (Two or three e4m3 terms, whose
// smallest step is 2^-9 under 2^6, took 143 us instead of 166 for the long
// chains below, calls in one graph, and lost such contexts: a tenth of the
// result at 4000 tokens.)
// An 8-bit product of n terms costs n/2 of a 16-bit one, and K and V
// cross shared memory once, without a widened copy (widening them to 16 bits
// first, by four warps, bound the kernel by shared memory: 2450 cycles a tile
// of 128 tokens instead of the 1425 that its 32 KB take from memory).  K's
// scales multiply S; V's multiply the weights, which a power of two a row that
// follows the largest scale the row sees keeps in the 8-bit range.
//
// What it takes and what bounds it (8 cache heads of 128; calls back to back):
//   64 trees of 26 nodes, 32 query heads, 700 to 4096 tokens, 16 bits: 143 us,
//     4.6 TB/s of K and V: memory, and the blocks' ends (106 to 124 us) and
//     the joining grid (7 us) behind it;
//   2 chains of 5, 64 query heads, 125,000 tokens, 8 bits: 191 us, 2.8 TB/s:
//     the turns of the products (1280 cycles a tile) and the softmax, 2600
//     cycles a tile in all;
//   8 trees of 64, 64 query heads, 3750 tokens, 16 bits: 85 us, 0.69 PFLOP/s:
//     the same turns (twice 1024 cycles of 3800 a tile), and joining (11 us).
// The plain form of sv_attention.cu takes 23.7, 59 and 20 ms for them.
#include <cuda.h>

#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "sv_cache_device.cuh"

namespace sv {
namespace {

constexpr int kTile = 128;        // tokens a tile, rows a half item
constexpr int kMaxCtas = 148;     // scratch is sized for this many blocks
constexpr int kMaxStages = 8;
constexpr int kScaleRing = kMaxStages;  // most tiles whose scales are held (8-bit pools)
// A segment's queries, last tile and result cost about as much as three tiles
// (64 trees of 26 nodes: the blocks' ends lay between 103 and 133 us without
// them in the split); they count where a block has several tiles.
constexpr int kExtra = 3;
constexpr int kJoinThreads = 512;
// 16-bit weights: log2 of the largest, and of what a weight may exceed it by.
// 16-bit floats reach 2^15, and below 2^-14 lose bits: with the largest near 1
// a weight under 2^-25 of it was zero.
constexpr float kBaseF16 = 7.0f, kLazy = 8.0f;
// 8-bit weights: the largest is near 2^13, and at most 2^15.5 < 57344.
constexpr float kBase8 = 13.0f, kLazy8 = 15.5f;
// log2 of the common factor that V's scales put on them.  Beyond these the
// weights without it (which are summed in 32 bits) would leave that type's
// range: scales above 2^109 cost the smallest weights, 2^-30 of the largest
// and more as the scales grow, and scales below 2^-94 the low bits.
constexpr int kLeastScale = -94, kMostScale = 121;

// Work split shared by the two grids.  An item counts as its tiles and `extra`
// more at its front, for what a segment costs besides its tiles; of all these
// units block c of n takes [start(c), start(c + 1)), the first blocks one more
// than the others.  A boundary among an item's extra units is one before it.
struct Split {
  long long each;
  int n, more, extra;
  __device__ __forceinline__ long long start(int c) const { return each * c + min(c, more); }
};

// Scratch: what each block found, for the joining grid, then the partial results.
constexpr size_t kPlanBytes = 16384;
__host__ __device__ inline size_t slot_floats(int DP) { return static_cast<size_t>(kTile) * (DP + 2); }

}  // namespace

struct MmaParams {
  AttnParams a;
  int R;        // rows of a (sequence, cache head)
  int halves;   // row tiles of 128
  int pairs;    // items of a (sequence, cache head)
  int box;      // tokens a TMA box: the largest power of two up to 128 that divides a page
  int head_first;  // the tensor maps' second axis is the head, not the place
  int stages;   // TMA ring entries
  int qtiles;   // row tiles of an item: 1 or 2
  int qrows;    // rows a Q tile has room for (a multiple of 8; the product reads 128, the rest is never used)
  int qbufs;    // Q buffers: 2, or 1 where two row tiles leave no room
  int scale_bytes;  // one scale array of a tile (8-bit pools)
  int scale_log;    // log2 of the tiles whose scales are held: 3, or 2 with up to 4 ring entries.  The ring
                    // may be `stages` entries ahead, and a tile's scales are needed until the
                    // product of the queries with the keys two tiles on: 2^scale_log >= stages / 2 + 2
  int negate;   // the scale is negative: Q is negated instead
  int zero;     // the scale is zero: Q is zero and the scale 1
  int qbox;     // nodes of a query box (the tensor map's); 0: plain loads
  int split;    // copies of the rows in the 128 lanes, each with a share of a tile's columns
  UDiv div_G;   // / a.G
  UDiv div_one, div_two;  // / rows of the only row tile, / 256 (the joining grid)
};

namespace {

__device__ __forceinline__ long long tokens_of(const AttnParams& a, int b, int& nodes, long long& len) {
  nodes = a.count ? min(max(__ldg(a.count + b), 0), a.N) : a.N;
  len = max(0, __ldg(a.cache_len + b));
  const long long cap = min(static_cast<long long>(a.c.max_pages) * a.c.page_size, 0x7fffffffll);
  const long long end = len + nodes;
  return nodes == 0 ? 0 : end < cap ? end : cap;
}
__device__ __forceinline__ int tiles_of(const AttnParams& a, int b) {
  int nodes;
  long long len;
  const long long t = (tokens_of(a, b, nodes, len) + kTile - 1) / kTile;
  return t < 1 ? 1 : static_cast<int>(t);
}

// The split, and where block c's share starts, by the first 256 threads of a
// block; all of them take part in the barriers.  b < 0: block c has none.
struct Found {
  Split split;
  int b, h, pr, into;  // sequence, cache head, pair of row tiles, units of that item before the share
  int tiles;         // of an item of that sequence
};
__device__ __forceinline__ void find_share(const AttnParams& a, int pairs, int blocks, int c, long long* sums, Found* f) {
  const int tid = threadIdx.x;
  const int per = (a.B + 255) / 256, per_b = a.c.heads * pairs;
  long long mine = 0;
  if (tid < 256) {
#pragma unroll 1
    for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) mine += static_cast<long long>(tiles_of(a, b)) * per_b;
    sums[tid] = mine;
  }
  __syncthreads();
  if (tid < 32) {
    long long s[8], run = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = run;
      run += sums[tid * 8 + i];
    }
    long long incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (tid >= o) incl += up;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[tid * 8 + i] = incl - run + s[i];
    if (tid == 31) {
      f->split.n = static_cast<int>(min(static_cast<long long>(blocks), incl));
      f->split.extra = incl >= 4ll * f->split.n ? kExtra : 0;
      const long long units = incl + static_cast<long long>(f->split.extra) * a.B * per_b;
      f->split.each = units / f->split.n;
      f->split.more = static_cast<int>(units - f->split.each * f->split.n);
      f->b = -1;
    }
  }
  __syncthreads();
  const int extra = f->split.extra;
  const long long x = c < f->split.n ? f->split.start(c) : -1;
  const int seqs = min(a.B - tid * per, per);  // this thread's sequences
  const long long first = sums[tid & 255] + static_cast<long long>(extra) * per_b * tid * per;
  if (tid < 256 && seqs > 0 && x >= first && x < first + mine + static_cast<long long>(extra) * per_b * seqs) {
    long long rem = x - first;
    int b = tid * per, t = tiles_of(a, b);
#pragma unroll 1
    while (rem >= static_cast<long long>(t + extra) * per_b) {
      rem -= static_cast<long long>(t + extra) * per_b;
      t = tiles_of(a, ++b);
    }
    const int item = static_cast<int>(rem / (t + extra));
    f->into = static_cast<int>(rem - static_cast<long long>(item) * (t + extra));
    f->h = item / pairs;
    f->pr = item - f->h * pairs;
    f->tiles = t;
    f->b = b;
  }
  __syncthreads();
}

// A block's segments in order, as every role walks them.
struct Walk {
  long long left;  // units of the share not yet walked, from this segment's item on
  int extra;
  int b, h, pr;    // sequence, cache head, pair of row tiles
  int tiles;       // of an item of b
  int t0, t1;      // this segment's tiles
  int nodes;
  long long len, total;
  bool first;
  __device__ __forceinline__ void load(const AttnParams& a) {
    total = tokens_of(a, b, nodes, len);
    const long long t = (total + kTile - 1) / kTile;
    tiles = t < 1 ? 1 : static_cast<int>(t);
  }
  // False: the share has no tile.
  __device__ __forceinline__ bool begin(const AttnParams& a, const Found& f, long long share) {
    extra = f.split.extra;
    b = f.b, h = f.h, pr = f.pr;
    first = true;
    load(a);
    left = share + f.into;
    t0 = max(0, f.into - extra);
    t1 = static_cast<int>(min(static_cast<long long>(tiles), left - extra));
    return t1 > t0;
  }
  __device__ __forceinline__ bool next(const AttnParams& a, int pairs) {
    left -= tiles + extra;
    if (left <= extra) return false;
    first = false;
    t0 = 0;
    if (++pr == pairs) {
      pr = 0;
      if (++h == a.c.heads) {
        h = 0;
        ++b;
        load(a);
      }
    }
    t1 = static_cast<int>(min(static_cast<long long>(tiles), left - extra));
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
  // Rows of the item, and whether it has two row tiles.
  __device__ __forceinline__ int row0() const { return pr * 2 * kTile; }
};

// ------------------------------------------------------------- PTX wrappers

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
      "%5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// Shared-memory operand with 128-byte swizzle: rows of 128 bytes, groups of 8
// rows 1024 bytes apart; for an operand whose rows run along K (V), `lbo` is
// the distance to the next 64 columns.  The low word of its descriptor; the
// high word is the same for all.
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t lbo) {
  return (addr & 0x3ffffu) >> 4 | (lbo >> 4) << 16;
}
constexpr uint32_t kOperandHigh = 1024u >> 4 | 1u << 14 | 2u << 29;
// f32 accumulator, M = 128; V is read transposed (its columns are the fast
// axis).  Types of A and B: 16 bits f16 0, bf16 1 (both the same); 8 bits
// e4m3 0, e5m2 1.
__host__ __device__ constexpr uint32_t mma_shape(uint32_t a_type, uint32_t b_type, int n, bool b_transposed) {
  return 1u << 4 | a_type << 7 | b_type << 10 | (b_transposed ? 1u << 16 : 0u) | static_cast<uint32_t>(n / 8) << 17 |
         8u << 24;
}
#define SV_MMA(KIND, A, MOVE_A)                                                                                \
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t" MOVE_A                  \
               "mov.b64 y, {%2, %5};\n\t"                                                                     \
               "tcgen05.mma.cta_group::1.kind::" KIND " [%0], " A ", y, %3, p;\n\t}" ::"r"(d),                 \
               "r"(a), "r"(b), "r"(shape), "r"(static_cast<uint32_t>(add)), "n"(kOperandHigh)                  \
               : "memory")
// D (+)= A B: A from shared (ss, by its low word) or tensor memory (ts).
template <bool E4>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, bool add) {
  if (E4)
    SV_MMA("f8f6f4", "x", "mov.b64 x, {%1, %5};\n\t");
  else
    SV_MMA("f16", "x", "mov.b64 x, {%1, %5};\n\t");
}
template <bool E4>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, bool add) {
  if (E4)
    SV_MMA("f8f6f4", "[%1]", "");
  else
    SV_MMA("f16", "[%1]", "");
}
#undef SV_MMA
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}
// Arrives on `bar` once every MMA this thread has issued is complete.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 columns of this warp's lanes; 16 or 8 back.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Two weights in the values' 16-bit type.
template <typename M>
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack_weights<__nv_bfloat16>(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <>
__device__ __forceinline__ uint32_t pack_weights<__half>(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// A value's leading 4 or 3 significant bits (towards zero): an e4m3 or e5m2
// value, where its exponent allows.
__device__ __forceinline__ float leading4(float x) { return __uint_as_float(__float_as_uint(x) & 0xfff00000u); }
__device__ __forceinline__ float leading3(float x) { return __uint_as_float(__float_as_uint(x) & 0xffe00000u); }
// Two e5m2 codes, rounded to nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t e5m2_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E5M2);
}

// Whether any element of a word is an infinity or a NaN.
template <typename T, bool E4>
__device__ __forceinline__ bool odd_word(uint32_t w) {
  if (E4) return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u;
  constexpr uint32_t e = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
  return (w & e) == e || (w >> 16 & e) == e;
}

struct Control {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t scale_full[kScaleRing];
  uint64_t s_full[2], p_ready[2][2], pv_done[2], o_done, q_full[2], q_empty[2], q_tma, drained;
  uint32_t tmem;
  int abort;
  int stop;              // abort, as the softmax warpgroups agreed on it
  int bad[2];            // a page of the segment is missing (by Q buffer)
  unsigned int odd[2][2];  // drafted tokens whose values hold an infinity or a NaN (by segment)
  int parent[2][64];
  float qscale[2][2 * kTile];
  float2 ml[2][kTile];
  alignas(16) float ones[4 * kTile];  // (as scales are laid out, in boxes of 8 to 128 tokens)
  long long sums[256];
  Found found;
};

// Bounded wait; once one has run out, every wait of the block returns at once
// and the roles run to their ends on whatever is there.
__device__ __noinline__ void wait_long(Control* s, uint64_t* bar, uint32_t parity, Ctrl* ctrl) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return;
  const unsigned long long t0 = global_ns();
#pragma unroll 1
  for (unsigned int spin = 1;; ++spin) {
    if (mbar_try_wait(bar, parity)) return;
    if ((spin & 63u) == 0u) {
      if (*reinterpret_cast<volatile int*>(&s->abort)) return;
      if (global_ns() - t0 > kWaitLimitNs) {
        *reinterpret_cast<volatile int*>(&s->abort) = 1;
        raise_flag(ctrl, kFlagTimeout);
        return;
      }
    }
  }
}
__device__ __forceinline__ void wait(Control* s, uint64_t* bar, uint32_t parity, Ctrl* ctrl) {
  if (!mbar_try_wait(bar, parity)) wait_long(s, bar, parity, ctrl);
}
__device__ __forceinline__ bool gave_up(const Control* s) { return *reinterpret_cast<const volatile int*>(&s->abort) != 0; }

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Largest score of a row's whole tile.  Both passes over a tile read a chunk
// ahead of the arithmetic.
__device__ __forceinline__ float tile_max(uint32_t s_addr) {
  float top[2] = {-INFINITY, -INFINITY};
  uint32_t v[2][16];
  tmem_ld16(s_addr, v[0]);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    tmem_wait_ld();
    if (c < 7) tmem_ld16(s_addr + (c + 1) * 16, v[(c + 1) & 1]);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const uint32_t* w = &v[c & 1][i];
      top[0] = fmax3(top[0], __uint_as_float(w[0]), __uint_as_float(w[1]));
      top[1] = fmax3(top[1], __uint_as_float(w[2]), __uint_as_float(w[3]));
    }
  }
  return fmaxf(top[0], top[1]);
}

// Tells `bar` that this warp's part of a hand-over is in tensor memory.
__device__ __forceinline__ void hand_over(uint64_t* bar) {
  tmem_wait_st();
  tmem_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// 2^x of two on the FMA pipe, with the special function unit's zero for masked
// scores and its NaN, both of which the polynomial does not know.
__device__ __forceinline__ void fma_ex2(float& a, float& b) {
  float p, q, za, zb;
  unpack2(ex2_poly_x2(a, b), p, q);
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(za) : "f"(a));
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(zb) : "f"(b));
  a = a > -126.0f ? p : za;
  b = b > -126.0f ? q : zb;
}

// Weights 2^(s c2 - shift) of 16 columns in the values' type, and their sums.
template <typename M>
__device__ __forceinline__ void weigh16(const uint32_t (&v)[16], unsigned long long c22, unsigned long long sh2,
                                        unsigned long long (&sum)[2], uint32_t (&out)[8]) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    unsigned long long x = fma2(pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), c22, sh2);
    unsigned long long y = fma2(pack2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), c22, sh2);
    float f[4];
    unpack2(x, f[0], f[1]);
    unpack2(y, f[2], f[3]);
    f[0] = ex2f(f[0]);
    f[1] = ex2f(f[1]);
    x = pack2(f[0], f[1]);
    if (i & 4) {
      fma_ex2(f[2], f[3]);  // a quarter of them
    } else {
      f[2] = ex2f(f[2]);
      f[3] = ex2f(f[3]);
    }
    y = pack2(f[2], f[3]);
    sum[0] = add2(sum[0], x);
    sum[1] = add2(sum[1], y);
    out[i >> 1] = pack_weights<M>(f[0], f[1]);
    out[(i >> 1) + 1] = pack_weights<M>(f[2], f[3]);
  }
}
__device__ __forceinline__ float total2(const unsigned long long (&sum)[2]) {
  float a, b, d, e;
  unpack2(sum[0], a, b);
  unpack2(sum[1], d, e);
  return (a + b) + (d + e);
}

// A row's whole tile into tensor memory over the scores; returns the sum.
// `half` is told when the first half of 128 columns is there.
template <typename M>
__device__ __forceinline__ float tile_weights(uint32_t s_addr, float c2, float shift, uint64_t* half) {
  const unsigned long long c22 = splat2(c2), sh2 = splat2(-shift);
  unsigned long long sum[2] = {0ull, 0ull};
  uint32_t v[2][16];
  tmem_ld16(s_addr, v[0]);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t out[8];
    tmem_wait_ld();
    if (c < 7) tmem_ld16(s_addr + (c + 1) * 16, v[(c + 1) & 1]);
    weigh16<M>(v[c & 1], c22, sh2, sum, out);
    tmem_st8(s_addr + c * 8, out);
    if (c == 3) hand_over(half);
  }
  return total2(sum);
}

// ---- the same for 8-bit pools.  A tile's scales lie in boxes of u = 8, 16 or
// 32 tokens, 32 floats apart.
struct Scales {
  const float *k, *v;
  int low, mul;  // u - 1, 32 / u
  __device__ __forceinline__ int at(int col) const { return (col & ~low) * mul + (col & low); }
};
// v *= K's scales of 16 columns from `col`.
__device__ __forceinline__ void scale_chunk(uint32_t (&v)[16], const Scales& sc, int col) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(sc.k + sc.at(col + (i & 8)) + (i & 4));
    float f[4];
    unpack2(mul2(pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), k.x), f[0], f[1]);
    unpack2(mul2(pack2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), k.y), f[2], f[3]);
#pragma unroll
    for (int z = 0; z < 4; ++z) v[i + z] = __float_as_uint(f[z]);
  }
}
__device__ __forceinline__ void max_chunk(const uint32_t (&v)[16], float (&top)[2]) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    top[0] = fmax3(top[0], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
    top[1] = fmax3(top[1], __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
  }
}
// Weights take the place of their scores: the columns of 32 tokens hold the
// terms of these one after the other, 8 columns each.
template <int TERMS>
__device__ __forceinline__ void weigh_chunk(const uint32_t (&v)[16], const Scales& sc, int col, uint32_t s_addr,
                                            unsigned long long c22, unsigned long long sh2, unsigned long long (&sum)[2]) {
  // 16 columns' weights, times V's scales, as TERMS 8-bit terms of 4 columns each
  uint32_t out[TERMS][4];
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(sc.v + sc.at(col + (i & 8)) + (i & 4));
    uint32_t codes[TERMS][2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const unsigned long long e =
          fma2(pack2(__uint_as_float(v[i + 2 * z]), __uint_as_float(v[i + 2 * z + 1])), c22, sh2);
      float a, b;
      unpack2(e, a, b);
      unsigned long long x = pack2(ex2f(a), ex2f(b));
      sum[z] = add2(sum[z], x);
      x = mul2(x, z ? w.y : w.x);
#pragma unroll
      for (int n = 0; n < TERMS; ++n) {
        unpack2(x, a, b);
        if (n < TERMS - 1) {
          a = leading3(a), b = leading3(b);
          x = sub2(x, pack2(a, b));
        }
        codes[n][z] = e5m2_pair(a, b);
      }
    }
#pragma unroll
    for (int n = 0; n < TERMS; ++n) out[n][i >> 2] = codes[n][0] | codes[n][1] << 16;
  }
#pragma unroll
  for (int n = 0; n < TERMS; ++n) tmem_st4(s_addr + (col & ~31) + 8 * n + (col & 16) / 4, out[n]);
}

// The root of 2^d, d <= 0, to be multiplied by twice.  The reference of an 8-bit
// pool's weights follows V's scales, by up to 2^215, and their sum may be as
// large as 2^126: 2^d alone may be zero when its product with the sum is not.
__device__ __forceinline__ float half_step(float d) { return ex2f(0.5f * d); }

// Puts -inf where a column is masked (bit i of word c allows column 32 c + i),
// before the two passes.  8-bit pools: K's scales enter here, so that a scale
// of a masked column does not matter, and the passes take ones.
template <bool E4>
__device__ __forceinline__ void mask_tile(uint32_t s_addr, const Scales& sc, const uint32_t (&words)[4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t word = words[c];
    if (!E4 && __all_sync(0xffffffffu, word == ~0u)) continue;
#pragma unroll 1
    for (int z = 0; z < 2; ++z) {
      uint32_t v[16];
      tmem_ld16(s_addr + c * 32 + z * 16, v);
      tmem_wait_ld();
      if (E4) scale_chunk(v, sc, c * 32 + z * 16);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = word >> (z * 16 + i) & 1u ? v[i] : 0xff800000u;
      tmem_st16(s_addr + c * 32 + z * 16, v);
    }
  }
  tmem_wait_st();
}

// What a segment needs besides its tiles, by 64 threads: the queries in the
// products' layout, the parents, and whether a page is missing.  Plain loads
// take microseconds each behind a full queue of tiles, so the queries come by
// one TMA box for 64 columns where rows of whole nodes fill a row tile.
template <typename QT, int DP, bool E4, int SPLIT>
__device__ __forceinline__ void load_segment(const MmaParams& p, const CUtensorMap* qmap, const Walk& w, Control* s,
                                             unsigned char* q_tiles, unsigned char* q_terms, int buf, uint32_t phase,
                                             int tid) {
  constexpr int kTerms = std::is_same<QT, __nv_bfloat16>::value ? 2 : 3;
  constexpr int kCopies = SPLIT > 1 ? SPLIT : 1;
  const AttnParams& a = p.a;
  const int row0 = w.row0();
  const int rows = min(2 * w.pr + 1 < p.halves ? 2 * kTile : kTile, p.R - row0);
  constexpr int kUnits = DP / 8;        // runs of 8 elements a row
  constexpr int kStride = 64 / kUnits;  // rows a step
  const int D = a.c.dim, j = tid % kUnits, first = tid / kUnits;
  const auto place = [&](int rr) {
    return reinterpret_cast<uint4*>(q_tiles + (rr >> 7) * kTile * DP * 2 + (j >> 3) * p.qrows * 128 + (rr & 127) * 128 +
                                    (((j & 7) ^ (rr & 7)) * 16));
  };
  if (p.qbox) {
    if (tid == 0) {
      // boxes of qbox nodes: one for each row tile, or one for each copy
      const bool one = E4 || p.negate || p.zero;  // the copies are written below
      const int boxes = SPLIT > 1 ? (one ? 1 : SPLIT) : rows > kTile ? 2 : 1;
      mbar_arrive_expect_tx(&s->q_tma, boxes * p.qbox * a.G * DP * 2);
      for (int i = 0; i < boxes; ++i) {
        const int node = SPLIT > 1 ? 0 : (row0 + i * kTile) / a.G;
#pragma unroll
        for (int c = 0; c < DP / 64; ++c)
          tma_4d(smem_addr(q_tiles) + (SPLIT > 1 ? i * (kTile / kCopies) * 128 : i * kTile * DP * 2) + c * p.qrows * 128,
                 qmap, c * 64, w.h * a.G, node, w.b, &s->q_tma);
      }
    }
  } else {
    const QT* const q = static_cast<const QT*>(a.q.p) + w.b * a.q.sb + static_cast<long long>(w.h * a.G) * a.q.sh + j * 8;
#pragma unroll 1
    for (int rr = first; rr < rows; rr += kStride) {
      const int nd = quotient(row0 + rr, p.div_G);
      const uint16_t* src = reinterpret_cast<const uint16_t*>(q + nd * a.q.sn + (row0 + rr - nd * a.G) * a.q.sh);
      uint32_t y[4] = {0u, 0u, 0u, 0u};
      if (j * 8 < D) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = src[2 * i] | static_cast<uint32_t>(src[2 * i + 1]) << 16;
      }
      for (int i = 0; i < kCopies; ++i) *place(rr + i * (kTile / kCopies)) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  if (a.parent && tid < a.N) s->parent[buf][tid] = __ldg(a.parent + static_cast<long long>(w.b) * a.N + tid);
  bool miss = false;
  const long long lo = static_cast<long long>(w.t0) * kTile, hi = min(static_cast<long long>(w.t1) * kTile, w.total);
  if (lo < hi) {
    const int* row = a.c.table + static_cast<long long>(w.b) * a.c.table_stride;
    const int last = page_of(a.c, static_cast<int>(hi - 1));
#pragma unroll 4
    for (int pi = page_of(a.c, static_cast<int>(lo)) + tid; pi <= last; pi += 64)
      miss |= static_cast<unsigned int>(__ldg(row + pi)) >= static_cast<unsigned int>(a.c.num_pages);
  }
  if (miss) {
    s->bad[buf] = 1;
    raise_flag(a.ctrl, kFlagInvalidPage);
  }
  if (p.qbox) wait(s, &s->q_tma, phase, a.ctrl);
  if (E4 || p.negate || p.zero) {
    // (a row's copies are written from the first)
#pragma unroll 2
    for (int r0 = first; r0 - first < rows; r0 += kStride) {  // all lanes take part
      const bool in = r0 < rows;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (in) v = *place(r0);
      if (p.zero) v = make_uint4(0u, 0u, 0u, 0u);
      if (p.negate) v.x ^= 0x80008000u, v.y ^= 0x80008000u, v.z ^= 0x80008000u, v.w ^= 0x80008000u;
      if (!E4) {
        if (in) {
#pragma unroll
          for (int i = 0; i < kCopies; ++i) *place(r0 + i * (kTile / kCopies)) = v;
        }
        continue;
      }
      // a power of two brings the row's largest element to 2^7..2^8
      float f[8];
      load8(reinterpret_cast<const QT*>(&v), f);
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
#pragma unroll
      for (int o = 1; o < kUnits; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int ex = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
      const bool plain = top == 0.0f || !(top < INFINITY);
      const float up = plain ? 1.0f : __uint_as_float(static_cast<unsigned int>(7 - ex + 127) << 23);
      if (in && j == 0)
        s->qscale[buf][r0] = plain ? 1.0f : __uint_as_float(static_cast<unsigned int>(ex - 7 + 127) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] *= up;
        if (!(fabsf(f[i]) < INFINITY)) f[i] = __int_as_float(0x7fc00000);  // the 8-bit type has no infinity
      }
#pragma unroll
      for (int n = 0; n < kTerms; ++n) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          w[i >> 2] = 0u;
#pragma unroll
          for (int z = 0; z < 4; z += 2) {
            float &x = f[i + z], &y = f[i + z + 1];
            const uint32_t two = n == kTerms - 1 ? e4m3_pair(x, y) : e4m3_pair(leading4(x), leading4(y));
            w[i >> 2] |= two << (8 * z);
            // the next terms make up for what this code rounds: below the
            // smallest normal ones that is more than what leading4 cuts off
            if (n < kTerms - 1) {
              const float2 is = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3)));
              x -= is.x, y -= is.y;
            }
          }
        }
        if (in) {
#pragma unroll
          for (int i = 0; i < kCopies; ++i) {
            const int r = (r0 & 127) + i * (kTile / kCopies);
            *reinterpret_cast<uint2*>(q_terms + ((r0 >> 7) * kTerms + n) * p.qrows * 128 + r * 128 +
                                      (((j >> 1) ^ (r & 7)) * 16) + (j & 1) * 8) = make_uint2(w[0], w[1]);
          }
        }
      }
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  // Both warps have seen these queries arrive before the next ones are asked
  // for (on the same barrier, and for 8-bit pools in the same place).
  asm volatile("bar.sync 2, 64;" ::: "memory");
}

// What the infinities and NaN of the drafted tokens in `seen` add to one
// element of a row that sees them: weight times an infinity or a NaN is
// itself, whatever the weight.  (8-bit pools: such a token makes the row NaN.)
template <typename QT, bool E4>
__device__ __noinline__ float odd_sum(const AttnParams& a, int b, long long len, long long total, unsigned long long seen, int h,
                                      int col) {
  float sum = E4 ? __int_as_float(0x7fc00000) : 0.0f;
  if (E4 || col >= a.c.dim) return sum;
#pragma unroll 1
  for (; seen; seen &= seen - 1) {
    const long long tok = len + __ffsll(static_cast<long long>(seen)) - 1;
    int page, place;
    if (tok >= total || !find_place(a.c, b, tok, page, place, nullptr)) continue;
    const float y = elem_f32(static_cast<const QT*>(a.c.v)[page * a.c.page_stride + place * a.c.token_stride +
                                                           h * a.c.head_stride + col]);
    if (!isfinite(y)) sum += y;
  }
  return sum;
}

// A finished segment's rows, staged one after the other, to the output: a
// node's heads lie next to each other there, so each node is one bulk copy.
template <typename QT>
__device__ __forceinline__ void store_segment(const MmaParams& p, const Walk& w, const unsigned char* staged, int tid) {
  const AttnParams& a = p.a;
  const int row0 = w.row0();
  const int rows = min(2 * w.pr + 1 < p.halves ? 2 * kTile : kTile, p.R - row0);
  const int n0 = quotient(row0, p.div_G), n1 = quotient(row0 + rows - 1, p.div_G);
  for (int nd = n0 + tid; nd <= n1; nd += 64) {
    const int r0 = max(nd * a.G, row0), r1 = min((nd + 1) * a.G, row0 + rows);
    QT* dst = static_cast<QT*>(a.out) +
              ((static_cast<long long>(w.b) * a.N + nd) * a.Hq + w.h * a.G + (r0 - nd * a.G)) * a.c.dim;
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(smem_addr(staged) + (r0 - row0) * a.c.dim * 2), "r"((r1 - r0) * a.c.dim * 2)
                 : "memory");
  }
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Ring entries of a segment of T tiles, in the order the MMA warp needs them:
// alternate tiles (one row tile): K0 K1 V0 K2 V1 ...; two row tiles: K0 V0 K1 V1 ...
__device__ __forceinline__ int v_entry(bool two, int t, int T) { return two ? 2 * t + 1 : t == T - 1 ? 2 * T - 1 : 2 * t + 2; }

}  // namespace

// DP: head_dim rounded up to 64 or 128.  QT: queries and output; E4: 8-bit
// pool.  SPLIT: 0 for items of two row tiles, else the copies of the rows that
// fill the 128 lanes (1, or with few rows 2 or 4); each takes a share of a
// tile's columns, as a sequence of its own that is joined at the segment's end.
template <typename QT, int DP, bool E4, int SPLIT>
__global__ void __launch_bounds__(384, 1)
    attention_mma_kernel(const __grid_constant__ MmaParams p, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap ksmap,
                         const __grid_constant__ CUtensorMap vsmap, const __grid_constant__ CUtensorMap qmap) {
  constexpr int kRow = E4 ? 128 : DP * 2;            // bytes of a token's row in a tile
  constexpr uint32_t entry = kTile * kRow;
  constexpr int kLoader = 10;                        // first of the two warps that load queries ahead
  constexpr int kChunks = DP / 64;
  constexpr bool two = SPLIT == 0;
  constexpr int kCopies = two ? 1 : SPLIT;
  // How the softmax warpgroups share the tiles.  Two row tiles: each its rows of
  // every tile.  8-bit pools with 65 to 128 rows: each half of every tile's
  // tokens, with an output of its own (104 rows: 186 us for 204 with tiles by
  // turns; 40 rows 276 for 179 as two copies by turns; 16 bits the same either way).
  // Else tiles by turns.
  constexpr bool kHalves = E4 && SPLIT == 1, kTurns = !two && !kHalves;
  constexpr bool kWhole = two || (kTurns && kCopies == 1);  // a thread weighs whole tiles
  constexpr float kBase = std::is_same<QT, __nv_bfloat16>::value ? 0.0f : kBaseF16;
  constexpr bool kBf16 = !E4 && std::is_same<QT, __nv_bfloat16>::value;
  constexpr int kTerms = std::is_same<QT, __nv_bfloat16>::value ? 2 : 3;  // 8-bit terms of queries (e4m3),
  constexpr int kParts = kTerms + 1;                                      // and of weights (e5m2)
  constexpr uint32_t kShapeS = mma_shape(kBf16, kBf16, kTile, false);
  constexpr uint32_t kShapeO = mma_shape(kBf16 || E4, kBf16, DP, true);

  // A row tile of queries, and a buffer of an item's (16 bits, or the terms);
  // 8-bit pools: where the queries arrive in 16 bits, and the ring of scales.
  const uint32_t qtile = static_cast<uint32_t>(p.qrows) * (E4 ? kTerms * 128 : DP * 2);
  const uint32_t qbytes = p.qtiles * qtile;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* qs = smem;
  unsigned char* qraw = qs + p.qbufs * qbytes;
  unsigned char* ring = qraw + (E4 ? p.qtiles * p.qrows * DP * 2 : 0);
  unsigned char* scale_ring = ring + p.stages * entry;
  Control* s = reinterpret_cast<Control*>(scale_ring + (E4 ? 2 * p.scale_bytes << p.scale_log : 0));
  const AttnParams& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 288) {
    for (const CUtensorMap* m : {&kmap, &vmap, &ksmap, &vsmap, &qmap})
      asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&s->full[i], 1);
      mbar_init(&s->empty[i], 1);
    }
    for (int i = 0; i < kScaleRing; ++i) mbar_init(&s->scale_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s->s_full[i], 1);
      mbar_init(&s->pv_done[i], 1);
      for (int z = 0; z < 2; ++z) mbar_init(&s->p_ready[i][z], 4);
      s->bad[i] = 0;
      for (int z = 0; z < 2; ++z) s->odd[z][i] = 0u;
      mbar_init(&s->q_full[i], 2);
      mbar_init(&s->q_empty[i], 8);
    }
    mbar_init(&s->o_done, 1);
    mbar_init(&s->drained, 1);
    mbar_init(&s->q_tma, 1);
    s->abort = 0;
    s->stop = 0;
  }
  for (int i = tid; i < 4 * kTile; i += 384) s->ones[i] = 1.0f;
  if (tid == 0) {
    mbar_fence_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&s->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tmem_fence_before();
  }
  __syncthreads();
  tmem_fence_after();
  const int cta = blockIdx.x;
  // Launched as a programmatic dependent: all of the above may overlap the
  // kernel before this one, whose end is waited for here.
  dep_enter();
  find_share(a, p.pairs, gridDim.x, cta, s->sums, &s->found);
  const uint32_t tmem = s->tmem;
  static_assert(kMaxCtas * sizeof(Found) <= kPlanBytes, "every block's plan fits");
  if (tid == 0) static_cast<Found*>(a.scratch)[cta] = s->found;

  Walk w;
  if (s->found.b >= 0 && w.begin(a, s->found, s->found.split.start(cta + 1) - s->found.split.start(cta))) {
    if (warp == 8) {
      // ------------------------------------------------ producer: TMA loads
      const int nbox = kTile / p.box;
      uint32_t e = 0, slot = 0, phase = 0, tile = 0;  // ring entries filled, the next one's place; tiles of keys
      bool stop = false;  // the same in all lanes
      do {
        const int h = w.h;
        const int T = w.t1 - w.t0;
        // page (num_pages: none, which TMA fills with zeros) and place of this
        // lane's box in two tiles running
        const auto locate = [&](int t, int& page, int& place) {
          page = a.c.num_pages;
          place = 0;
          const long long tok = static_cast<long long>(w.t0 + t) * kTile + lane * p.box;
          if (t < T && lane < nbox && tok < w.total) {
            const int pi = page_of(a.c, static_cast<int>(tok));
            place = static_cast<int>(tok) - pi * a.c.page_size;
            const int g = __ldg(a.c.table + static_cast<long long>(w.b) * a.c.table_stride + pi);
            if (static_cast<unsigned int>(g) < static_cast<unsigned int>(a.c.num_pages)) page = g;
          }
        };
        const auto load = [&](bool values, int page, int place) {
          if (stop) return;
          wait(s, &s->empty[slot], phase ^ 1u, a.ctrl);
          if (__any_sync(0xffffffffu, gave_up(s))) stop = true;
          if (stop) return;
          const uint32_t dst = smem_addr(ring + slot * entry);
          const uint32_t ti = tile & ((1u << p.scale_log) - 1u);
          if (lane == 0) {
            mbar_arrive_expect_tx(&s->full[slot], entry);
            if (E4 && !values) mbar_arrive_expect_tx(&s->scale_full[ti], 2 * kTile * 4);
          }
          __syncwarp();
          if (lane < nbox) {
            const CUtensorMap* map = values ? &vmap : &kmap;
            const int y = p.head_first ? h : place, z = p.head_first ? place : h;
            if (E4) {
              tma_4d(dst + lane * p.box * kRow, map, 0, y, z, page, &s->full[slot]);
              if (!values) {
                const uint32_t sd = smem_addr(scale_ring) + ti * 2 * p.scale_bytes + lane * max(p.box * 4, 128);
                tma_3d(sd, &ksmap, place, h, page, &s->scale_full[ti]);
                tma_3d(sd + p.scale_bytes, &vsmap, place, h, page, &s->scale_full[ti]);
              }
            } else {
#pragma unroll
              for (int c = 0; c < kChunks; ++c)
                tma_4d(dst + c * kTile * 128 + lane * p.box * 128, map, c * 64, y, z, page, &s->full[slot]);
            }
          }
          if (!values) ++tile;
          ++e;
          if (++slot == static_cast<uint32_t>(p.stages)) slot = 0, phase ^= 1u;
        };
        int pg0, pl0, pg1, pl1;
        locate(0, pg0, pl0);
        if (!two) load(false, pg0, pl0);
        for (int t = 0; t < T && !stop; ++t) {
          locate(t + 1, pg1, pl1);
          if (two) {
            load(false, pg0, pl0);
            load(true, pg0, pl0);
          } else {
            if (t + 1 < T) load(false, pg1, pl1);
            load(true, pg0, pl0);
          }
          pg0 = pg1;
          pl0 = pl1;
        }
      } while (!stop && w.next(a, p.pairs));
      if (stop) {  // copies in flight land before the block ends
        const unsigned long long t0 = global_ns();
        const uint32_t n = min(e, static_cast<uint32_t>(p.stages));
        for (uint32_t i = e - n; i < e; ++i)
          while (!mbar_try_wait(&s->full[i % p.stages], (i / p.stages) & 1u) && global_ns() - t0 < kWaitLimitNs) {}
        if (E4)
          for (uint32_t i = tile - min(tile, 1u << p.scale_log); i < tile; ++i)
            while (!mbar_try_wait(&s->scale_full[i & ((1u << p.scale_log) - 1u)], (i >> p.scale_log) & 1u) &&
                   global_ns() - t0 < kWaitLimitNs) {}
      }
    } else if (warp == 9) {
      // ------------------------------------------------ MMA issue
      // The whole warp walks the loop, so that addresses and descriptors stay
      // in uniform registers; one elected thread issues.
      const uint32_t stages = p.stages;
      const uint32_t chunk = p.qrows * 128 >> 4;  // Q's next 64 columns, or its next term
      // The ring is read in its own order; a tile stays until its last product.
      uint32_t next = 0, next_phase = 0, kslot = 0, vslot = 0;
      const auto take = [&](uint32_t& slot) {
        slot = next;
        wait(s, &s->full[slot], next_phase, a.ctrl);
        if (++next == stages) next = 0, next_phase ^= 1u;
      };
      const uint32_t acc = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q0 = operand(smem_addr(qs), 16);
      const uint32_t k0 = operand(smem_addr(ring), 16);
      const uint32_t v0 = operand(smem_addr(ring), kTile * 128);
      uint32_t seg = 0, np = 0;  // np: phases of p_ready, one bit a warpgroup
      bool stop = false;
      do {
        const int T = __shfl_sync(0xffffffffu, w.t1 - w.t0, 0), U = two ? 2 * T : T;
        const uint32_t buf = p.qbufs == 2 ? seg & 1u : 0u;
        wait(s, &s->q_full[buf], (p.qbufs == 2 ? seg >> 1 : seg) & 1u, a.ctrl);
        const uint32_t q1 = q0 + buf * (qbytes >> 4);
#pragma unroll 1
        for (int x = 0; x <= U; ++x) {
          const uint32_t g = x & 1;
          const bool shared = two && g == 1;  // the second user of this tile
          if (x < U) {
            if (!shared) take(kslot);
            tmem_fence_after();
            const uint32_t qd = q1 + (shared ? qtile >> 4 : 0);
            const uint32_t kd = k0 + kslot * (entry >> 4);
            if (elect_one()) {
              // 32 bytes of a 128-byte row a step: 16 elements (64 are the next
              // block of rows), or 32 of 8 bits (then the next term)
#pragma unroll
              for (int k = 0; k < (E4 ? kTerms * DP / 32 : DP / 16); ++k) {
                constexpr int kSteps = E4 ? DP / 32 : 4;
                mma_ss<E4>(acc + g * kTile, qd + (k / kSteps) * chunk + (k % kSteps) * 2,
                           kd + (E4 ? 0 : (k / 4) * (kTile * 128 >> 4)) + (k % kSteps) * 2, kShapeS, k > 0);
              }
              mma_commit(&s->s_full[g]);
              if (!two || g == 1) mma_commit(&s->empty[kslot]);
            }
            __syncwarp();
          }
          if (x > 0) {
            const uint32_t f = g ^ 1u;  // unit x - 1
            if (!two || f == 0) take(vslot);
            const uint32_t vd = v0 + vslot * (entry >> 4);
            const uint32_t pw = acc + f * kTile;
            const auto accumulate = [&](int half) {
              const uint32_t o = acc + 2 * kTile + (kHalves ? half : f) * DP;
              const bool add = kHalves ? x > 1 : x > 2 || half > 0;
              if (E4) {
                // 32 tokens a step, each with the terms of the weights
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                  for (int n = 0; n < kParts; ++n)
                    mma_ts<E4>(o, pw + 64 * half + 32 * k + 8 * n, vd + (2 * half + k) * (32 * 128 >> 4), kShapeO,
                               add || k > 0 || n > 0);
              } else {
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k)
                  mma_ts<E4>(o, pw + half * 32 + k * 8, vd + (half * 4 + k) * (16 * 128 >> 4), kShapeO,
                             add || k > 0);
              }
            };
            wait(s, &s->p_ready[f][0], np >> f & 1u, a.ctrl);
            tmem_fence_after();
            if (elect_one()) {
              accumulate(0);
            }
            __syncwarp();
            wait(s, &s->p_ready[f][1], np >> f & 1u, a.ctrl);
            np ^= 1u << f;
            tmem_fence_after();
            if (elect_one()) {
              accumulate(1);
              if (!two || f == 1) mma_commit(&s->empty[vslot]);
              if (kHalves) mma_commit(&s->pv_done[f]);
              if (x == U) mma_commit(&s->o_done);
            }
            __syncwarp();
          }
        }
        ++seg;
        stop = __any_sync(0xffffffffu, gave_up(s));  // (after a wait ran out, none waits any more)
      } while (!stop && w.next(a, p.pairs));
      if (stop) {  // MMAs in flight finish before their memory goes away
        if (elect_one()) mma_commit(&s->drained);
        __syncwarp();
        const unsigned long long t0 = global_ns();
        while (!mbar_try_wait(&s->drained, 0) && global_ns() - t0 < kWaitLimitNs) {}
      }
      __syncwarp();
    } else if (warp >= kLoader) {
      // -------------------------- the next segment's queries, the last one's result
      const int lt = tid - kLoader * 32;
      Walk done = w;  // the oldest segment whose buffer has not been emptied
      uint32_t seg = 0, oldest = 0;
      bool stop = false, more = true;
      const auto buffer = [&](uint32_t x) { return p.qbufs == 2 ? x & 1u : 0u; };
      const auto turn = [&](uint32_t x) { return (p.qbufs == 2 ? x >> 1 : x) & 1u; };
      const auto empty = [&] {
        const uint32_t buf = buffer(oldest);
        wait(s, &s->q_empty[buf], turn(oldest), a.ctrl);
        const bool lost = gave_up(s);
        if (!lost && done.whole()) store_segment<QT>(p, done, qs + buf * qbytes, lt);
        ++oldest;
        done.next(a, p.pairs);
        // Both warps' copies have been read before either loads over them, and
        // both stop together.
        uint32_t any;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
            "bar.red.or.pred p, 2, 64, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(any)
            : "r"(static_cast<uint32_t>(lost))
            : "memory");
        stop = any != 0;
      };
      while (!stop && more) {
        if (seg >= static_cast<uint32_t>(p.qbufs)) empty();
        if (stop) break;
        const uint32_t buf = buffer(seg);
        load_segment<QT, DP, E4, SPLIT>(p, &qmap, w, s, E4 ? qraw : qs + buf * qbytes, qs + buf * qbytes, buf, seg & 1u, lt);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s->q_full[buf]);
        ++seg;
        more = w.next(a, p.pairs);
      }
      while (!stop && oldest < seg) empty();
    } else {
      // ------------------------------------------------ softmax warpgroups
      const int g = warp >> 2, r = tid & 127;
      const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 (warp % 4)
      uint32_t base = 0, tile_base = 0, ns = 0, seg = 0;
      do {
        const int h = w.h;
        const int T = w.t1 - w.t0;
        const int row0 = w.row0();
        const int rows = min(two ? 2 * kTile : kTile, p.R - row0);
        const uint32_t buf = p.qbufs == 2 ? seg & 1u : 0u;
        wait(s, &s->q_full[buf], (p.qbufs == 2 ? seg >> 1 : seg) & 1u, a.ctrl);
        if (tid == 0 && w.t0 == 0 && w.nodes > 0 && w.len + w.nodes > w.total) raise_flag(a.ctrl, kFlagCapacity);
        const bool missing = *reinterpret_cast<volatile int*>(&s->bad[buf]) != 0;

        constexpr int lanes = kTile / kCopies;
        const int copy = r / lanes;
        const int row = two ? g * kTile + r : r - copy * lanes;  // row within the item
        const bool live = row < rows;
        const bool warp_live = two ? g * kTile + (warp & 3) * 32 < rows : ((warp & 3) * 32) % lanes < rows;
        const int node = live ? quotient(row0 + row, p.div_G) : 0;
        // the node's ancestors and itself; nothing at or below an invalid parent
        unsigned long long mask = live && node < w.nodes ? 1ull << node : 0ull;
        if (mask && !a.parent) {
          mask |= mask - 1ull;
        } else if (mask) {
          for (int i = node; i > 0;) {
            const int up = s->parent[buf][i];
            if (up < 0 || up >= i) {
              raise_flag(a.ctrl, kFlagInvalidTree);
              mask = 0ull;
              break;
            }
            mask |= 1ull << up;
            i = up;
          }
        }
        const float c2 = E4 ? a.c2 * (live ? s->qscale[buf][row] : 0.0f) : a.c2;
        const uint32_t o_addr = tmem + lane_base + 2 * kTile + g * DP;
        float M = -INFINITY, l = 0.0f;
        int vexp = -200;  // log2 of the weights' common factor (8-bit pools)

        for (int t = kTurns ? g : 0; t < T; t += kTurns ? 2 : 1) {
          const int sb = kHalves ? t & 1 : g;  // where the scores are
          const uint32_t s_addr = tmem + lane_base + sb * kTile;
          const long long tok0 = static_cast<long long>(w.t0 + t) * kTile;
          const bool tail = tok0 + kTile > w.len;           // drafted tokens or the end
          const bool masked = tail || tok0 + kTile > w.total || missing;
          const uint32_t ti = (tile_base + t) & ((1u << p.scale_log) - 1u);
          Scales sc{};
          if (E4) {
            wait(s, &s->scale_full[ti], ((tile_base + t) >> p.scale_log) & 1u, a.ctrl);
            sc.k = reinterpret_cast<const float*>(scale_ring + ti * 2 * p.scale_bytes);
            sc.v = sc.k + p.scale_bytes / 4;
            sc.low = min(p.box, 32) - 1;
            sc.mul = 32 / min(p.box, 32);
            __syncwarp();
          }
          const auto scores = [&] {
            wait(s, &s->s_full[sb], ns >> sb & 1u, a.ctrl);
            ns ^= 1u << sb;
          };
          if (tail) {
            // The scores first: with them every ring entry up to this tile's keys
            // has been filled, so the slot of its values has at most one phase to
            // go, which is what a wait on a phase's parity can tell.
            scores();
            // Values of places past the end may be anything: zeros, so that a
            // zero weight stays zero.  A drafted token's infinities and NaN
            // are taken out as well and added by hand to the rows that see it.
            const long long tok = tok0 + r;
            if ((kTurns || g == 0) && tok >= w.len) {
              const uint32_t e = base + v_entry(two, t, T), slot = e % p.stages;
              wait(s, &s->full[slot], (e / p.stages) & 1u, a.ctrl);
              uint4* line = reinterpret_cast<uint4*>(ring + slot * entry + r * 128);
#pragma unroll 1
              for (int c = 0; c < (E4 ? 1 : kChunks); ++c, line += kTile * 8) {
                if (tok >= w.total) {
#pragma unroll
                  for (int q = 0; q < 8; ++q) line[q ^ (r & 7)] = make_uint4(0u, 0u, 0u, 0u);
                } else {
                  bool odd = false;
#pragma unroll
                  for (int q = 0; q < 8; ++q) {
                    const uint4 v = line[q ^ (r & 7)];
                    odd |= odd_word<QT, E4>(v.x) | odd_word<QT, E4>(v.y) | odd_word<QT, E4>(v.z) | odd_word<QT, E4>(v.w);
                  }
                  if (odd) {
                    uint32_t* y = reinterpret_cast<uint32_t*>(line);
#pragma unroll 1
                    for (int q = 0; q < 32; ++q) {
                      if (E4) {
                        if (odd_word<QT, E4>(y[q])) y[q] = 0u;
                      } else {
                        if (odd_word<QT, E4>(y[q] & 0xffffu)) y[q] &= 0xffff0000u;
                        if (odd_word<QT, E4>(y[q] & 0xffff0000u)) y[q] &= 0xffffu;
                      }
                    }
                    atomicOr(&s->odd[seg & 1][(tok - w.len) >> 5], 1u << ((tok - w.len) & 31));
                  }
                }
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (E4) {
              // The same for V's scales, by each warpgroup for itself (what two
              // write is the same).
              float* vs = const_cast<float*>(sc.v) + sc.at(r & ~7) + (r & 7);
              if (tok >= w.total) {
                *vs = 0.0f;
              } else if (tok >= w.len && !(fabsf(*vs) < INFINITY)) {
                *vs = 0.0f;
                atomicOr(&s->odd[seg & 1][(tok - w.len) >> 5], 1u << ((tok - w.len) & 31));
              }
              if (g == 0)
                asm volatile("bar.sync 3, 128;" ::: "memory");
              else
                asm volatile("bar.sync 4, 128;" ::: "memory");
            }
          }
          int ve = vexp;
          if (E4 && warp_live) {
            // The largest finite scale of V among the tokens that this row sees:
            // of the context four tokens a lane, of the drafted ones its own.
            __syncwarp();
            const auto finite = [](float y) { return fabsf(y) < INFINITY ? fabsf(y) : 0.0f; };
            const auto exponent = [](float y) {  // y <= 2^exponent
              return min(max(static_cast<int>(__float_as_uint(y) >> 23) - 126, kLeastScale), kMostScale);
            };
            const float4 x = *reinterpret_cast<const float4*>(sc.v + sc.at(lane * 4 & ~7) + (lane * 4 & 4));
            const float y[4] = {finite(x.x), finite(x.y), finite(x.z), finite(x.w)};
            const int drafted = tail ? static_cast<int>(w.len - tok0) : kTile;  // first column of the tree
            float old = 0.0f, young = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) (lane * 4 + i < drafted ? old : young) = fmaxf(lane * 4 + i < drafted ? old : young, y[i]);
            ve = max(vexp, exponent(warp_max(old)));
            if (tail && exponent(warp_max(young)) > ve) {
              young = 0.0f;
#pragma unroll 1
              for (unsigned long long m = mask; m; m &= m - 1) {
                const int col = drafted + __ffsll(static_cast<long long>(m)) - 1;
                if (static_cast<unsigned int>(col) < static_cast<unsigned int>(kTile)) young = fmaxf(young, finite(sc.v[sc.at(col)]));
              }
              ve = max(ve, exponent(young));
            }
          }
          if (!tail) scores();
          __syncwarp();
          tmem_fence_after();
          if (warp_live) {
            // the columns this thread weighs
            constexpr int kNC = kHalves ? 4 : 8 / kCopies;
            const int col0 = kHalves ? 64 * g : copy * (kTile / kCopies);
            constexpr int kWords = kNC / 2;
            uint32_t words[kWords];
            if (masked) {
#pragma unroll
              for (int c = 0; c < kWords; ++c) {
                const long long from = tok0 + col0 + 32 * c, off = from - w.len, lim = w.total - from;
                uint32_t y = ~0u;
                if (off >= 64) y = 0u;
                else if (off >= 0) y = static_cast<uint32_t>(mask >> off);
                else if (off > -32) y = static_cast<uint32_t>(mask << -off) | ((1u << -off) - 1u);
                if (lim <= 0) y = 0u;
                else if (lim < 32) y &= (1u << lim) - 1u;
                if (missing) {
                  bool in = false;
                  if (lane < lim) {
                    const int pi = page_of(a.c, static_cast<int>(from + lane));
                    in = static_cast<unsigned int>(__ldg(a.c.table + static_cast<long long>(w.b) * a.c.table_stride + pi)) <
                         static_cast<unsigned int>(a.c.num_pages);
                  }
                  y &= __ballot_sync(0xffffffffu, in);
                }
                words[c] = y;
              }
              if constexpr (kWhole) {
                mask_tile<E4>(s_addr, sc, words);
                sc.k = s->ones;
              }
            }
            // Scores that are read once and held: a share of a tile, or with two
            // row tiles and an 8-bit pool the second half.
            constexpr int kHeld = kWhole ? (E4 ? 4 : 1) : kNC;
            uint32_t held[kHeld][16];
            float top;
            if constexpr (!kWhole) {
#pragma unroll
              for (int c = 0; c < kNC; ++c) tmem_ld16(s_addr + col0 + c * 16, held[c]);
              tmem_wait_ld();
              if (kCopies > 1) {
                // the other copies' weights count as zero here
                const uint32_t none[E4 ? 8 : 16] = {};
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  if (c < copy * (4 / kCopies) || c >= (copy + 1) * (4 / kCopies)) {
                    if constexpr (E4) {
#pragma unroll
                      for (int n = 0; n < kParts; ++n) tmem_st8(s_addr + c * 32 + n * 8, none);
                    } else {
                      tmem_st16(s_addr + c * 16, none);
                    }
                  }
              }
              float t2[2] = {-INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < kNC; ++c) {
                if (E4) scale_chunk(held[c], sc, col0 + c * 16);
                if (masked) {
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    held[c][i] = words[c / 2] >> ((c & 1) * 16 + i) & 1u ? held[c][i] : 0xff800000u;
                }
                max_chunk(held[c], t2);
              }
              top = fmaxf(t2[0], t2[1]);
            } else if constexpr (E4) {
              float t2[2] = {-INFINITY, -INFINITY};
              tmem_ld16(s_addr + 64, held[0]);
#pragma unroll
              for (int c = 0; c < kHeld; ++c) {
                tmem_wait_ld();
                if (c < kHeld - 1) tmem_ld16(s_addr + (4 + c + 1) * 16, held[c + 1]);
                scale_chunk(held[c], sc, (4 + c) * 16);
                max_chunk(held[c], t2);
              }
#pragma unroll 2
              for (int c = 0; c < 4; ++c) {
                uint32_t v[16];
                tmem_ld16(s_addr + c * 16, v);
                tmem_wait_ld();
                scale_chunk(v, sc, c * 16);
                max_chunk(v, t2);
              }
              top = fmaxf(t2[0], t2[1]);
            } else {
              top = tile_max(s_addr);
            }
            // (lanes without a row hold anything: they must not make the others
            // raise their maximum, or the roundings differ from call to call)
            top = !live || top == -INFINITY ? -INFINITY : top * c2;
            bool raise;
            float Mn = M;
            if (E4) {
              raise = top > M - vexp + kLazy8 || ve > vexp;
              if (__any_sync(0xffffffffu, raise)) Mn = fmaxf(M - vexp + kBase8, top) - kBase8 + ve;
              vexp = ve;
            } else {
              raise = top > M + kBase + kLazy;
              if (__any_sync(0xffffffffu, raise)) Mn = fmaxf(M, top - kBase);
            }
            if (Mn != M) {
              const float f = M == -INFINITY ? 0.0f : E4 ? half_step(M - Mn) : ex2f(M - Mn);
              l *= f;
              if (E4) l *= f;
            }
            // the first tile's product overwrites O
            if (t > (kTurns ? 1 : 0) && __any_sync(0xffffffffu, Mn != M)) {
              if (kHalves) {
                // (elsewhere these scores came after that product)
                const int last = sb ^ 1;
                wait(s, &s->pv_done[last], (ns >> last & 1u) ^ 1u, a.ctrl);
                __syncwarp();
                tmem_fence_after();
              }
              const float f = M == -INFINITY ? 0.0f : Mn == M ? 1.0f : ex2f(M - Mn);
#pragma unroll 1
              for (int c = 0; c < DP / 16; ++c) {
                uint32_t v[16];
                tmem_ld16(o_addr + c * 16, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(f == 0.0f ? 0.0f : __uint_as_float(v[i]) * f);
                tmem_st16(o_addr + c * 16, v);
              }
            }
            M = Mn;
            const float shift = M == -INFINITY ? 0.0f : M;
            const unsigned long long c22 = splat2(c2), sh2 = splat2(-shift);
            unsigned long long sum[2] = {0ull, 0ull};
            if constexpr (E4) {
              if constexpr (kWhole) {
#pragma unroll 1
                for (int c = 0; c < 64; c += 32) {
                  uint32_t v[2][16];
                  tmem_ld16(s_addr + c, v[0]);
                  tmem_ld16(s_addr + c + 16, v[1]);
                  tmem_wait_ld();
#pragma unroll
                  for (int z = 0; z < 2; ++z) {
                    scale_chunk(v[z], sc, c + z * 16);
                    weigh_chunk<kParts>(v[z], sc, c + z * 16, s_addr, c22, sh2, sum);
                  }
                }
                hand_over(&s->p_ready[g][0]);
              }
              const int from = kWhole ? 64 : col0;
#pragma unroll
              for (int c = 0; c < kHeld; ++c) weigh_chunk<kParts>(held[c], sc, from + c * 16, s_addr, c22, sh2, sum);
              l += total2(sum);
            } else if constexpr (!kWhole) {
#pragma unroll
              for (int c = 0; c < kNC; ++c) {
                uint32_t out[8];
                weigh16<QT>(held[c], c22, sh2, sum, out);
                tmem_st8(s_addr + (copy * kNC + c) * 8, out);
              }
              l += total2(sum);
            } else {
              l += tile_weights<QT>(s_addr, c2, shift, &s->p_ready[g][0]);
            }
            tmem_wait_st();
          }
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (!kHalves && (!kWhole || !warp_live)) mbar_arrive(&s->p_ready[g][0]);
            mbar_arrive(kHalves ? &s->p_ready[sb][g] : &s->p_ready[g][1]);
          }
        }

        // ---- the segment's end: join the two groups, write
        wait(s, &s->o_done, seg & 1u, a.ctrl);
        __syncwarp();
        tmem_fence_after();
        if (mask == 0ull) M = -INFINITY, l = 0.0f;
        s->ml[g][r] = make_float2(M, l);
        softmax_sync();
        const unsigned int odd0 = s->odd[seg & 1][0], odd1 = s->odd[seg & 1][1];
        float f0 = 1.0f, f1 = 0.0f;
        if (!two) {
          // all copies of the row in both groups; a group without a tile has
          // sum 0, and a NaN sum comes with a maximum of -inf
          float top = -INFINITY, sum = 0.0f;
          float2 x[2 * kCopies];
#pragma unroll
          for (int z = 0; z < 2 * kCopies; ++z) {
            x[z] = s->ml[z & 1][row + (z >> 1) * lanes];
            top = fmaxf(top, x[z].x);
          }
#pragma unroll
          for (int z = 0; z < 2 * kCopies; ++z)
            if (x[z].y != 0.0f) {
              const float f = x[z].x == top ? 1.0f : E4 ? half_step(x[z].x - top) : ex2f(x[z].x - top);
              sum += (E4 ? x[z].y * f : x[z].y) * f;
            }
          const float2 x0 = s->ml[0][r], x1 = s->ml[1][r];
          f0 = x0.y == 0.0f ? 0.0f : x0.x == top ? 1.0f : ex2f(x0.x - top);
          f1 = x1.y == 0.0f ? 0.0f : x1.x == top ? 1.0f : ex2f(x1.x - top);
          M = top;
          l = sum;
        }
        const bool whole = w.whole();
        const bool none = mask == 0ull || l == 0.0f;
        const float inv = none ? 0.0f : whole ? 1.0f / l : 1.0f;
        const unsigned long long seen = mask & (static_cast<unsigned long long>(odd1) << 32 | odd0);
        const int col0 = two ? 0 : g * (DP / 2), ncol = two ? DP : DP / 2;
        const int D = a.c.dim, head = h * a.G + (row0 + row - node * a.G);
        const int slot = 2 * cta + (w.first ? 0 : 1);
        float* part = static_cast<float*>(a.scratch) + kPlanBytes / 4 +
                      (static_cast<size_t>(slot) * p.qtiles + (row >> 7)) * slot_floats(DP);
        // The queries are done with: their buffer takes the result's rows, one
        // after the other, and behind them what the copies hand over.
        unsigned char* const staged = qs + buf * qbytes;
        float4* const handed =
            reinterpret_cast<float4*>(staged + lanes * DP * 2) + g * (kCopies - 1) * 4 * lanes;
#pragma unroll 2
        for (int c = 0; c < ncol; c += 16) {
          float o[16];
          if (warp_live) {
            uint32_t v[16], v1[16];
            const uint32_t at = tmem + lane_base + 2 * kTile + col0 + c;
            __syncwarp();
            tmem_ld16(at + (two ? g * DP : 0), v);
            if (!two) tmem_ld16(at + DP, v1);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float y = f0 == 0.0f ? 0.0f : __uint_as_float(v[i]) * f0;
              if (!two && f1 != 0.0f) y = fmaf(__uint_as_float(v1[i]), f1, y);
              o[i] = none ? 0.0f : y * inv;
            }
          }
          if (SPLIT > 1) {
            if (live && copy > 0) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                handed[((copy - 1) * 4 + i / 4) * lanes + row] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
            softmax_sync();
            if (live && copy == 0) {
              for (int z = 1; z < SPLIT; ++z)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                  const float4 y = handed[((z - 1) * 4 + i / 4) * lanes + row];
                  o[i] += y.x, o[i + 1] += y.y, o[i + 2] += y.z, o[i + 3] += y.w;
                }
            }
            softmax_sync();
          }
          if (live && copy == 0) {
            if (seen && !none) {
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] += odd_sum<QT, E4>(a, w.b, w.len, w.total, seen, h, col0 + c + i);
            }
            if (whole) {
              QT* dst = reinterpret_cast<QT*>(staged) + row * D + col0 + c;
#pragma unroll
              for (int i = 0; i < 16; i += 8) {
                if (col0 + c + i < D) {
                  const float y[8] = {o[i], o[i + 1], o[i + 2], o[i + 3], o[i + 4], o[i + 5], o[i + 6], o[i + 7]};
                  store8(dst + i, y);
                }
              }
            } else {
              float4* dst = reinterpret_cast<float4*>(part) + static_cast<size_t>((col0 + c) / 4) * kTile + (row & 127);
#pragma unroll
              for (int i = 0; i < 16; i += 4) dst[i / 4 * kTile] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
          }
        }
        if (live && copy == 0 && (two || g == 0)) {
          if (whole) {
            if (a.lse)
              a.lse[(static_cast<long long>(w.b) * a.N + node) * a.Hq + head] = none ? -INFINITY : (M + log2f(l)) * kLn2;
          } else {
            float2* ml = reinterpret_cast<float2*>(part + static_cast<size_t>(kTile) * DP);
            ml[row & 127] = make_float2(none ? -INFINITY : M, none ? 0.0f : l);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the staged rows
        tmem_fence_before();
        if (tid == 0) s->stop = gave_up(s);
        softmax_sync();  // O, ml and odd may be overwritten now
        if (tid < 2) s->odd[seg & 1][tid] = 0u;
        if (tid == 2) s->bad[buf] = 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s->q_empty[buf]);
        base += 2 * T;
        tile_base += T;
        ++seg;
      } while (!*reinterpret_cast<volatile int*>(&s->stop) && w.next(a, p.pairs));
    }
  }
  __syncthreads();
  if (warp == 9) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// ----------------------------------------------------------------- joining
//
// Block j looks at the boundary between shares j and j + 1, which the first
// grid's block j + 1 left in its plan.  The blocks whose boundaries cut one
// item share its rows' columns (runs of 8), so that each reads about as much
// as one share wrote.
template <typename QT, int DP, bool E4>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const __grid_constant__ MmaParams p) {
  dep_enter();
  const AttnParams& a = p.a;
  const int j = blockIdx.x + 1;
  const Found found = static_cast<const Found*>(a.scratch)[j];
  const Split split = found.split;
  const int b = found.b, h = found.h;
  if (b < 0 || found.into <= split.extra) return;  // no such share, or one that starts with an item
  const long long lo = split.start(j) - found.into, hi = lo + split.extra + found.tiles;
  int first = j, last = j;  // boundaries inside the item
  while (first > 1 && split.start(first - 1) > lo + split.extra) --first;
  while (last + 1 < split.n && split.start(last + 1) < hi) ++last;
  const int parts = last - first + 2;
  const bool two = 2 * found.pr + 1 < p.halves;
  const int row0 = found.pr * 2 * kTile;
  const int rows = min(two ? 2 * kTile : kTile, p.R - row0);
  const int D = a.c.dim;
  const int units = rows * (D / 8), blocks = last - first + 1, me = j - first;
  const int u0 = static_cast<int>(static_cast<long long>(units) * me / blocks);
  const int u1 = static_cast<int>(static_cast<long long>(units) * (me + 1) / blocks);
  const float* scratch = static_cast<const float*>(a.scratch) + kPlanBytes / 4;
  const int slot0 = 2 * (first - 1) + (split.start(first - 1) < lo ? 1 : 0);
  const UDiv& by_rows = two && rows == 2 * kTile ? p.div_two : p.div_one;
  const auto part = [&](int i, int row) {
    const int slot = i == 0 ? slot0 : 2 * (first - 1 + i);
    return scratch + (static_cast<size_t>(slot) * p.qtiles + (row >> 7)) * slot_floats(DP);
  };
  const auto stats = [&](int i, int row) {
    return reinterpret_cast<const float2*>(part(i, row) + static_cast<size_t>(kTile) * DP)[row & 127];
  };
  constexpr int kAhead = 4;  // parts whose loads are in flight together
  for (int i = u0 + static_cast<int>(threadIdx.x); i < u1; i += kJoinThreads) {
    int c = quotient(i, by_rows), row = i - c * static_cast<int>(by_rows.d);
    if (static_cast<int>(by_rows.d) != rows) c = i / rows, row = i - c * rows;
    float M = -INFINITY, L = 0.0f, o[8] = {};
    for (int x0 = 0; x0 < parts; x0 += kAhead) {
      float2 ml[kAhead];
      float4 y0[kAhead], y1[kAhead];
#pragma unroll
      for (int z = 0; z < kAhead; ++z) {
        ml[z] = make_float2(-INFINITY, 0.0f);
        if (x0 + z < parts) {
          const float4* q = reinterpret_cast<const float4*>(part(x0 + z, row));
          ml[z] = stats(x0 + z, row);
          y0[z] = q[static_cast<size_t>(2 * c) * kTile + (row & 127)];
          y1[z] = q[static_cast<size_t>(2 * c + 1) * kTile + (row & 127)];
        }
      }
      float top = M;
#pragma unroll
      for (int z = 0; z < kAhead; ++z) top = fmaxf(top, ml[z].x);
      const float step = M == top ? 1.0f : E4 ? half_step(M - top) : ex2f(M - top);
      const float keep = E4 ? step * step : step;
      L *= step;
      if (E4) L *= step;
#pragma unroll
      for (int x = 0; x < 8; ++x) o[x] = keep == 0.0f ? 0.0f : o[x] * keep;
      M = top;
#pragma unroll
      for (int z = 0; z < kAhead; ++z) {
        if (ml[z].y == 0.0f) continue;
        const float s = ml[z].x == M ? 1.0f : E4 ? half_step(ml[z].x - M) : ex2f(ml[z].x - M);
        const float f = E4 ? s * s : s;
        L = fmaf(E4 ? ml[z].y * s : ml[z].y, s, L);
        if (f == 0.0f) continue;
        o[0] = fmaf(y0[z].x, f, o[0]), o[1] = fmaf(y0[z].y, f, o[1]), o[2] = fmaf(y0[z].z, f, o[2]);
        o[3] = fmaf(y0[z].w, f, o[3]), o[4] = fmaf(y1[z].x, f, o[4]), o[5] = fmaf(y1[z].y, f, o[5]);
        o[6] = fmaf(y1[z].z, f, o[6]), o[7] = fmaf(y1[z].w, f, o[7]);
      }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int x = 0; x < 8; ++x) o[x] *= inv;
    const int node = quotient(row0 + row, p.div_G), head = h * a.G + (row0 + row - node * a.G);
    const long long out_row = (static_cast<long long>(b) * a.N + node) * a.Hq + head;
    store8(static_cast<QT*>(a.out) + out_row * D + c * 8, o);
    if (a.lse && c == 0) a.lse[out_row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}

// --------------------------------------------------------------- launching

namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
  static EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// One of the pool's tensors: (element, place, head, page), the place and head
// axes ordered by their strides.
bool pool_map(CUtensorMap* m, const CacheView& c, void* base, int dtype, int box, bool head_first) {
  const int es = dtype == 3 ? 1 : 2;
  const CUtensorMapDataType type = dtype == 3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int dp = c.dim <= 64 ? 64 : 128;
  cuuint64_t dim[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page_size),
                       static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.num_pages)};
  cuuint64_t st[3] = {static_cast<cuuint64_t>(c.token_stride) * es, static_cast<cuuint64_t>(c.head_stride) * es,
                      static_cast<cuuint64_t>(c.page_stride) * es};
  // an axis of one entry may have any stride: give it a valid one
  for (int i = 0; i < 3; ++i)
    if (dim[i + 1] == 1) st[i] = (i == 0 ? static_cast<cuuint64_t>(dp) * es : st[i - 1]);
  cuuint32_t bx[4] = {static_cast<cuuint32_t>(dtype == 3 ? 128 : 64), static_cast<cuuint32_t>(box), 1, 1};
  if (head_first) {
    const cuuint64_t d = dim[1];
    dim[1] = dim[2], dim[2] = d;
    const cuuint64_t s = st[0];
    st[0] = st[1], st[1] = s;
    bx[2] = bx[1], bx[1] = 1;
  }
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return encoder()(m, type, 4, base, dim, st, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool scale_map(CUtensorMap* m, const CacheView& c, void* base, int box) {
  const cuuint64_t dim[3] = {static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.heads),
                             static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t st[2] = {static_cast<cuuint64_t>(c.page_size) * 4, static_cast<cuuint64_t>(c.page_size) * c.heads * 4};
  const cuuint32_t bx[3] = {static_cast<cuuint32_t>(box), 1, 1}, one[3] = {1, 1, 1};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dim, st, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries: (element, head, node, sequence), boxes of one group of heads.
bool query_map(CUtensorMap* m, const AttnParams& a, int q_dtype, int nodes) {
  const cuuint64_t dim[4] = {static_cast<cuuint64_t>(a.c.dim), static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.N),
                             static_cast<cuuint64_t>(a.B)};
  long long st[3] = {a.q.sh, a.q.sn, a.q.sb};
  for (int i = 0; i < 3; ++i) {
    if (dim[i + 1] == 1) st[i] = i == 0 ? (a.c.dim + 7) / 8 * 8 : st[i - 1];  // any valid one will do
    if (st[i] <= 0 || st[i] % 8 || st[i] >= (1ll << 38)) return false;
  }
  if (reinterpret_cast<uintptr_t>(a.q.p) % 16 || a.G > 256) return false;
  const cuuint64_t bytes[3] = {static_cast<cuuint64_t>(st[0]) * 2, static_cast<cuuint64_t>(st[1]) * 2,
                               static_cast<cuuint64_t>(st[2]) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(nodes), 1}, one[4] = {1, 1, 1, 1};
  return encoder()(m, q_dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                   const_cast<void*>(a.q.p), dim, bytes, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename QT, int DP, bool E4, int SPLIT>
cudaError_t launch_mma(MmaParams& p, const CUtensorMap (&maps)[5], int grid, cudaStream_t st) {
  constexpr int kLimit = 227 * 1024;
  const int boxes = kTile / p.box;
  p.scale_bytes = E4 ? boxes * (p.box * 4 > 128 ? p.box * 4 : 128) : 0;
  const int entry = kTile * (E4 ? 128 : DP * 2);
  constexpr int kTerms = std::is_same<QT, __nv_bfloat16>::value ? 2 : 3;
  p.qrows = p.qtiles == 2 || p.split > 1 ? kTile : (p.R + 7) / 8 * 8;
  p.qbufs = p.qtiles == 2 ? 1 : 2;  // (the trees of 26 nodes with 1: 134 us for 122)
  const int qrow = E4 ? kTerms * 128 : DP * 2;
  int fixed = 0;
  for (p.scale_log = 3; p.scale_log >= 2; --p.scale_log) {
    fixed = p.qtiles * p.qrows * (p.qbufs * qrow + (E4 ? DP * 2 : 0)) + (E4 ? 2 * p.scale_bytes << p.scale_log : 0) +
            static_cast<int>(sizeof(Control));
    p.stages = (kLimit - fixed) / entry;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    if (p.stages > 4 || p.scale_log == 2) break;
  }
  // Keys of the next tile have to fit beside the values of this one, and with
  // one row tile the values of the last one too (the wait for a tail's values).
  if (p.stages < (p.qtiles == 2 ? 2 : 3)) return cudaErrorNotSupported;
  const size_t smem = fixed + static_cast<size_t>(p.stages) * entry;
  const auto kernel = attention_mma_kernel<QT, DP, E4, SPLIT>;
  static std::atomic<bool> done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLimit);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  e = counted(launch_k(SV_PDL >= 1, kernel, dim3(grid), dim3(384), smem, st, p, maps[0], maps[1], maps[2],
                       maps[3], maps[4]),
              1);
  if (e != cudaSuccess || grid < 2) return e;
  return counted(launch_k(SV_PDL >= 1, attention_join_kernel<QT, DP, E4>, dim3(grid - 1), dim3(kJoinThreads), 0, st, p), 1);
}

template <typename QT, bool E4>
cudaError_t launch_split(MmaParams& p, const CUtensorMap (&maps)[5], int grid, cudaStream_t st) {
  const bool wide = p.a.c.dim > 64;
  if constexpr (E4)
    if (p.split == 4) return wide ? launch_mma<QT, 128, E4, 4>(p, maps, grid, st) : launch_mma<QT, 64, E4, 4>(p, maps, grid, st);
  if (p.split == 2) return wide ? launch_mma<QT, 128, E4, 2>(p, maps, grid, st) : launch_mma<QT, 64, E4, 2>(p, maps, grid, st);
  if (p.split == 1) return wide ? launch_mma<QT, 128, E4, 1>(p, maps, grid, st) : launch_mma<QT, 64, E4, 1>(p, maps, grid, st);
  return wide ? launch_mma<QT, 128, E4, 0>(p, maps, grid, st) : launch_mma<QT, 64, E4, 0>(p, maps, grid, st);
}

}  // namespace

size_t attention_scratch_bytes(int N, int G, int dim) {
  const int halves = (N * G + kTile - 1) / kTile;
  return kPlanBytes + static_cast<size_t>(2 * kMaxCtas) * (halves > 1 ? 2 : 1) * slot_floats(dim <= 64 ? 64 : 128) * 4;
}

bool attention_mma_takes(const AttnParams& a, int cache_dtype) {
  const CacheView& c = a.c;
  const int es = cache_dtype == 3 ? 1 : 2;
  const auto on16 = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  if (c.dim > 128 || c.dim * es % 16 || c.dim % 8 || c.page_size % 8 || !encoder()) return false;
  if (!on16(c.k) || !on16(c.v) || !on16(a.out) || (cache_dtype == 3 && (!on16(c.ks) || !on16(c.vs)))) return false;
  const auto ok = [&](long long stride, int n) { return n == 1 || (stride > 0 && stride * es % 16 == 0 && stride * es < (1ll << 40)); };
  return ok(c.token_stride, c.page_size) && ok(c.head_stride, c.heads) && ok(c.page_stride, c.num_pages);
}

cudaError_t launch_attention_mma(const AttnParams& a, int q_dtype, int cache_dtype, int sms, cudaStream_t st) {
  MmaParams p{};
  p.a = a;
  p.R = a.N * a.G;
  p.div_G = make_udiv(static_cast<unsigned int>(a.G));
  p.div_one = make_udiv(static_cast<unsigned int>(p.R < kTile ? p.R : kTile));
  p.div_two = make_udiv(2 * kTile);
  p.halves = (p.R + kTile - 1) / kTile;
  p.pairs = (p.halves + 1) / 2;
  p.qtiles = p.halves > 1 ? 2 : 1;
  p.box = 8;
  while (p.box < kTile && a.c.page_size % (2 * p.box) == 0) p.box *= 2;
  p.head_first = a.c.heads > 1 && a.c.page_size > 1 && a.c.head_stride < a.c.token_stride;
  p.negate = a.c2 < 0.0f;
  p.zero = a.c2 == 0.0f;
  p.a.c2 = p.zero ? 1.0f : a.c2 < 0.0f ? -a.c2 : a.c2;
  // Few rows: copies of them share a tile's columns.  Two 125,000-token
  // sequences, 20 rows (us, 1 / 2 / 4 copies): 8 bits 277 / 170 / 152, 64
  // sequences 175 / 134 / 117; 16 bits 170 / 160 / 161.
  p.split = p.R <= 32 && cache_dtype == 3 ? 4 : p.R <= 64 ? 2 : p.R <= kTile ? 1 : 0;
  CUtensorMap maps[5] = {};
  bool ok = pool_map(&maps[0], a.c, a.c.k, cache_dtype, p.box, p.head_first) &&
            pool_map(&maps[1], a.c, a.c.v, cache_dtype, p.box, p.head_first);
  if (cache_dtype == 3) ok = ok && scale_map(&maps[2], a.c, a.c.ks, p.box) && scale_map(&maps[3], a.c, a.c.vs, p.box);
  if (!ok) return cudaErrorNotSupported;  // nothing launched: the plain form takes the call
  // rows of whole nodes that fill a row tile, or all rows at once
  const int box = p.R <= kTile ? a.N : kTile % a.G == 0 ? kTile / a.G : 0;
  p.qbox = box > 0 && query_map(&maps[4], a, q_dtype, box) ? box : 0;
  // no more blocks than tiles there can be
  const long long per_seq = (static_cast<long long>(a.c.max_pages) * a.c.page_size + kTile - 1) / kTile;
  const long long most = static_cast<long long>(a.B) * a.c.heads * p.pairs * per_seq;
  int grid = sms < kMaxCtas ? sms : kMaxCtas;
  if (most < grid) grid = static_cast<int>(most);
  const bool e4 = cache_dtype == 3;
  if (q_dtype == 1)
    return e4 ? launch_split<__nv_bfloat16, true>(p, maps, grid, st) : launch_split<__nv_bfloat16, false>(p, maps, grid, st);
  return e4 ? launch_split<__half, true>(p, maps, grid, st) : launch_split<__half, false>(p, maps, grid, st);
}

}  // namespace sv
