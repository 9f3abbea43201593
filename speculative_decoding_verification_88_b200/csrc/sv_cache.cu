// sv_cache.cu -- rotary positions, the paged cache's write (as it is, or in
// 8 bits with one scale a row), its read-back and the move of accepted rows.
// All four move data once.  Long inputs are bound by memory (16-bit rotary of
// 16,000 tokens with 40 heads of 128: 60 us, 5.5 TB/s; read-back of 32
// sequences from 8 bits: 76 us, 5.3 TB/s; 64 accepted paths in 32 layers: 18
// us, 3.4 TB/s), but for the write into 8 bits, which is bound by the
// instructions of exact codes (8 x 1000 tokens, 8 + 8 cache heads and 32 query
// heads: 52 us, 3.5 TB/s; into 16 bits 39 us).  A few tokens take one launch's
// latency, 4 to 6 us on the GPU.
#include <type_traits>

#include "sv_cache_device.cuh"

namespace sv {

// ------------------------------------------------- rotary and cache write
//
// A unit is 16 elements of a row (a head of q, k or v): 8 whole pairs, or 16
// neighbours past rotary_dim.  A block takes a few tokens at a time: each of
// its threads first has the loads of its (up to four) units in flight, then
// the block turns position * f into (cos, sin) pairs in shared memory, once
// for all heads, and then the units are turned and stored.  The angle is
// reduced as turns (position * f / 2 pi, minus the nearest integer).  Near
// position 2^31 that integer has up to 29 bits, so the product is formed as a
// sum of two 64-bit numbers, and what is left is exact to 2^-53 turns at any
// 32-bit position; cos and sin then work on a half turn at most.
//
// Rows whose parts are multiples of 16 elements on 16-byte boundaries (8-bit
// pools: 8) move 16 bytes a load (VEC), others one element: rotary 60 against
// 568 us at the size above, the 8-bit write 52 against 181, the 16-bit one 39
// against 124.
//
// 8-bit rows: the codes are those of exact arithmetic, rounded once.  32-bit
// arithmetic decides nearly all of them: a code is taken when the values an
// error bound below and above give the same one, and only the others (about
// one in 10^5) are computed again in 64 bits.  The scale needs the row's
// exact largest magnitude: the elements within the bound of the 32-bit
// maximum, one or two a row, are computed in 64 bits.

constexpr int kRotThreads = 256;

struct Unit {
  int a, b;    // first elements of the two runs of 8
  int na, nb;  // elements of each (runs of a vectorised unit are whole)
  bool pair;   // rotary pairs
  bool weave;  // pairs are neighbours: each run holds four (VEC), or the unit's run of 16 eight
};
// `turn`: the row has a rotary part.  Vectorised units take their second run
// half a part further on, so that neighbouring lanes read neighbouring runs.
template <bool VEC>
__device__ __forceinline__ Unit unit_at(int u, bool turn, int rd, int D, bool inter) {
  Unit x;
  const int np = turn ? (rd / 2 + 7) / 8 : 0;
  x.pair = u < np;
  x.weave = x.pair && inter;
  if (x.pair && (VEC || !inter)) {
    x.na = x.nb = min(8, rd / 2 - 8 * u);
    x.a = 8 * u;
    x.b = rd / 2 + 8 * u;
  } else if (x.pair) {
    x.na = x.nb = min(8, rd / 2 - 8 * u);
    x.a = 16 * u;
    x.b = x.a + 1;
  } else {
    const int base = turn ? rd : 0, v = u - np;
    x.a = base + (VEC ? 8 : 16) * v;
    x.b = VEC ? base + (D - base) / 2 + 8 * v : x.a + 8;
    x.na = max(0, min(8, (VEC ? base + (D - base) / 2 : D) - x.a));
    x.nb = VEC ? x.na : max(0, min(8, D - x.b));
  }
  return x;
}
// Angle of pair z of a unit (its lane among the row's units, rotary_dim).
template <bool VEC>
__device__ __forceinline__ int angle_of(int z, int lane, int rd, bool weave) {
  return VEC && weave ? (z < 4 ? 0 : rd / 4 - 4) + 4 * lane + z : 8 * lane + z;
}

// A unit's elements as they are in memory.
template <typename T>
struct Raw {
  alignas(16) T a[8];  // first members (or the first 8 elements)
  alignas(16) T b[8];  // second members (the next 8)
};
template <typename T, bool VEC>
__device__ __forceinline__ void load_raw(const T* row, const Unit& u, Raw<T>& r) {
  if (VEC) {
    if (u.na == 0) return;
    constexpr int kWords = sizeof(T) * 8 / 16;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      reinterpret_cast<uint4*>(r.a)[i] = reinterpret_cast<const uint4*>(row + u.a)[i];
      reinterpret_cast<uint4*>(r.b)[i] = reinterpret_cast<const uint4*>(row + u.b)[i];
    }
  } else {
    const int step = u.weave ? 2 : 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < u.na) r.a[i] = row[u.a + i * step];
      if (i < u.nb) r.b[i] = row[u.b + i * step];
    }
  }
}
// f: first members (or the first 8 elements), g: second members (the next 8).
template <typename T, bool VEC>
__device__ __forceinline__ void unpack_raw(const Raw<T>& r, const Unit& u, float (&f)[8], float (&g)[8]) {
  float x[8], y[8];
  if (VEC) {
    load8(r.a, x);
    load8(r.b, y);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < u.na ? elem_f32(r.a[i]) : 0.0f, y[i] = i < u.nb ? elem_f32(r.b[i]) : 0.0f;
  }
  const bool weave = VEC && u.weave;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = weave ? x[2 * i] : x[i];
    g[i] = weave ? x[2 * i + 1] : y[i];
    f[4 + i] = weave ? y[2 * i] : x[4 + i];
    g[4 + i] = weave ? y[2 * i + 1] : y[4 + i];
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T* row, const Unit& u, const float (&f)[8], const float (&g)[8]) {
  if (VEC) {
    if (u.na == 0) return;
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = u.weave ? f[i] : f[2 * i];
      x[2 * i + 1] = u.weave ? g[i] : f[2 * i + 1];
      y[2 * i] = u.weave ? f[4 + i] : g[2 * i];
      y[2 * i + 1] = u.weave ? g[4 + i] : g[2 * i + 1];
    }
    store8(row + u.a, x);
    store8(row + u.b, y);
  } else {
    const int step = u.weave ? 2 : 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < u.na) row[u.a + i * step] = from_f32<T>(f[i]);
      if (i < u.nb) row[u.b + i * step] = from_f32<T>(g[i]);
    }
  }
}

__device__ __forceinline__ float code_value(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
}
// The code of x c - y s (64-bit c, s) over `scale`, given the two neighbouring
// codes it lies between: on which side of their midpoint m it is, is the sign
// of one fused multiply-add (x c - y s) - m scale; the midpoint itself goes to
// the even code.
__device__ __noinline__ uint32_t nearer_code(uint32_t lo, uint32_t hi, float x, float y, double c, double s, float scale) {
  const double m = 0.5 * (static_cast<double>(code_value(lo)) + code_value(hi));
  const double v = fma(static_cast<double>(x), c, -(static_cast<double>(y) * s));
  const double d = fma(-m, static_cast<double>(scale), v);
  return d > 0.0 ? hi : d < 0.0 ? lo : (hi & 1u ? lo : hi);
}

// x / s for an element that is held exactly, rounded to odd: the last bit says
// whether anything was cut off, so that rounding it again, to 4 significant
// bits, gives what rounding the exact quotient gives (Boldo and Melquiond,
// "Emulation of FMA and correctly rounded sums: proved algorithms using
// rounding to odd", 2008).  The remainder of a quotient that is right to a
// unit in the last place is exact in one fused multiply-add.
__device__ __forceinline__ float quotient_odd(float x, float s, float inv) {
  const float q0 = x * inv;
  const float q = fmaf(fmaf(-q0, s, x), inv, q0);
  const float r = fmaf(-q, s, x);
  const uint32_t bits = __float_as_uint(q);
  const uint32_t cut = (__float_as_uint(r) ^ bits) & 0x80000000u ? bits - 1u : bits;  // towards zero
  return r == 0.0f ? q : __uint_as_float(cut | 1u);
}

struct RotatePlan {
  int UP;         // lanes of a row (8-bit pools: a power of two, for the row's reduction)
  int units;      // of them in use
  int rows;       // rows a block takes at a time
  int turn;       // rows of a warp
  int passes;     // until a token's rows are done
  int group;      // tokens whose angles a block prepares together
  UDiv div_N, div_half;  // / N, / (rd / 2)
};

// A group's warps wait for one another twice; with up to 16 tokens (4) the
// 8-bit write takes 52 (60) us and rotary 64 (66).
constexpr int kRotGroup = 16;     // most tokens of a group
constexpr int kRotAngles = 1024;  // their (cos, sin) pairs: rotary_dim <= 512

// 1 / 2 pi as a sum.
constexpr double kTurn = 0.15915494309189533577, kTurnLow = -9.839338337591243e-18;

// Places (dst: element offset, -1: none, -2: padding; sdst: the scales') and
// (cos, sin) of a group of tokens.
template <bool E4>
__device__ __forceinline__ void prepare_tokens(const RotateParams& p, const RotatePlan& n, long long t0, int group, float2* cs,
                                               double2* csd, long long* dst, long long* sdst, long long* pos) {
  const int tid = threadIdx.x, half_rd = p.rd / 2;
  __syncthreads();  // the last group's are done with
  if (tid < group) {
    const int t = static_cast<int>(t0) + tid;
    const int b = quotient(t, n.div_N), j = t - b * p.N;
    long long at = -1, sat = 0, where = 0;
    if (p.count && j >= __ldg(p.count + b)) {
      at = -2;
    } else if (p.positions) {
      where = __ldg(p.positions + t);
    } else {
      int depth = j;
      if (p.parent) {
        const int* par = p.parent + static_cast<long long>(b) * p.N;
        depth = 0;
        for (int x = j; x > 0; ++depth) {  // parents decrease, so this ends
          const int up = __ldg(par + x);
          if (up < 0 || up >= x) {
            raise_flag(p.ctrl, kFlagInvalidTree);
            break;
          }
          x = up;
        }
      }
      const long long len = max(0, __ldg(p.cache_len + b));
      where = len + depth;
      int page, place;
      if (p.write && find_place(p.c, b, len + j, page, place, p.ctrl)) {
        at = page * p.c.page_stride + place * p.c.token_stride;
        sat = static_cast<long long>(page) * p.c.heads * p.c.page_size + place;
      }
    }
    dst[tid] = at;
    sdst[tid] = sat;
    pos[tid] = where;
  }
  __syncthreads();
  if (!p.inv_freq) return;
  for (int i = tid; i < group * half_rd; i += blockDim.x) {
    const int k = quotient(i, n.div_half), f = i - k * half_rd;
    const double at = static_cast<double>(pos[k]), freq = __ldg(p.inv_freq + f);
    const double angle = at * freq, rest = fma(at, freq, -angle);
    const double turns = angle * kTurn, low = fma(angle, kTurn, -turns) + fma(angle, kTurnLow, rest * kTurn);
    const double half = 2.0 * ((turns - rint(turns)) + low);
    float s, c;
    sincospif(static_cast<float>(half), &s, &c);
    s = p.inverse ? -s : s;
    cs[i] = make_float2(c * p.magnitude, s * p.magnitude);
    if (E4) {
      double sd, cd;
      sincospi(half, &sd, &cd);
      csd[i] = make_double2(cd * p.magnitude, sd * p.magnitude);
    }
  }
  __syncthreads();
}

// The (cos, sin) of a unit's eight pairs: two runs of four.
template <bool VEC>
__device__ __forceinline__ void load_angles(const float2* run0, const float2* run1, int n, float2 (&w)[8]) {
  if (VEC) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = reinterpret_cast<const float4*>(run0)[i], y = reinterpret_cast<const float4*>(run1)[i];
      w[2 * i] = make_float2(x.x, x.y), w[2 * i + 1] = make_float2(x.z, x.w);
      w[4 + 2 * i] = make_float2(y.x, y.y), w[5 + 2 * i] = make_float2(y.z, y.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i] = i < 4 ? run0[i] : run1[i - 4];
  }
}

// Turns a unit in 32 bits.
template <bool VEC>
__device__ __forceinline__ void turn_unit(const Unit& u, const float2 (&w)[8], float (&f)[8], float (&g)[8]) {
#pragma unroll
  for (int z = 0; z < 8; ++z) {
    if (VEC || z < u.na) {
      const float x = f[z], y = g[z];
      f[z] = fmaf(x, w[z].x, -y * w[z].y);
      g[z] = fmaf(y, w[z].x, x * w[z].y);
    }
  }
}

// Members of pair z of a unit (or elements z of its two runs), z a constant.
template <typename T, bool VEC>
__device__ __forceinline__ void member(const Raw<T>& r, const Unit& u, bool weave, int z, float& f, float& g) {
  if (VEC && weave) {
    f = elem_f32(z < 4 ? r.a[2 * z] : r.b[2 * z - 8]);
    g = elem_f32(z < 4 ? r.a[2 * z + 1] : r.b[2 * z - 7]);
  } else {
    f = VEC || z < u.na ? elem_f32(r.a[z]) : 0.0f;
    g = VEC || z < u.nb ? elem_f32(r.b[z]) : 0.0f;
  }
}

// A unit of a row that is not turned: 16 exact elements in two runs of 8.  A
// code is taken when x / scale from below and from above, 2^-21 of it apart
// from the product with the rounded reciprocal (off by 2^-22 at most), give the
// same one; others (16-bit elements are often 448ths of one another, and then
// close to the middle of two codes), and rows whose scale is tiny, zero or NaN,
// are divided with rounding to odd.
template <typename T>
__device__ __forceinline__ void code_exact_unit(const Raw<T>& raw, const Unit& u, int UP, bool first_lane, bool live,
                                                uint8_t* out, float* scale_out) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.0f;
  if (live) {
    float f[8], g[8];
    load8(raw.a, f);
    load8(raw.b, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = f[i], x[8 + i] = g[i];
  }
  float top = 0.0f;
  unsigned long long zero = 0ull;  // stays so unless an element is an infinity or a NaN
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    top = fmax3(top, fabsf(x[i]), fabsf(x[i + 1]));
    zero = fma2(pack2(x[i], x[i + 1]), 0ull, zero);
  }
  float z0, z1;
  unpack2(zero, z0, z1);
  const uint32_t odd = __ballot_sync(0xffffffffu, !(z0 + z1 == 0.0f));
  for (int o = UP >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float scale = __fdiv_rn(top, 448.0f);
  const int lane = threadIdx.x & 31;
  const uint32_t row = (UP == 32 ? 0xffffffffu : (1u << UP) - 1u) << (lane & ~(UP - 1));
  if (odd & row) scale = __int_as_float(0x7fc00000);
  if (!live) return;
  const float inv = 1.0f / scale;
  const unsigned long long lo = splat2(inv * (1.0f - 0x1p-21f)), hi = splat2(inv * (1.0f + 0x1p-21f));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (scale >= 0x1p-60f) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      float a, b, c, d;
      unpack2(mul2(pack2(x[i], x[i + 1]), lo), a, b);
      unpack2(mul2(pack2(x[i], x[i + 1]), hi), c, d);
      uint32_t two = e4m3_pair(a, b);
      if (two != e4m3_pair(c, d)) two = e4m3_pair(quotient_odd(x[i], scale, inv), quotient_odd(x[i + 1], scale, inv));
      w[i >> 2] |= two << (i & 2 ? 16 : 0);
    }
  } else {
    const float up = 0x1p80f, s = scale * up, is = scale > 0.0f ? 1.0f / s : 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 2)
      w[i >> 2] |= e4m3_pair(quotient_odd(x[i] * up, s, is), quotient_odd(x[i + 1] * up, s, is)) << (i & 2 ? 16 : 0);
  }
  *reinterpret_cast<uint2*>(out + u.a) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(out + u.b) = make_uint2(w[2], w[3]);
  if (first_lane) *scale_out = scale;
}

// A unit of a turned row, 8 pairs of which `pair` says whether they are turned.
// |f| + |g| of a pair is at most 2 / magnitude of the row's largest result, so
// that bounds every element's 32-bit error.
template <typename T, bool INTER>
__device__ __forceinline__ void code_turned_unit(const Raw<T>& raw, const Unit& u, int UP, bool first_lane, bool live, bool pair,
                                                 float magnitude, const float2* w0, const float2* w1, const double2* cd0,
                                                 const double2* cd1, uint8_t* out, float* scale_out) {
  const bool weave = INTER && u.weave;
  const auto exact = [&](int z) { return pair ? (z < 4 ? cd0[z] : cd1[z - 4]) : make_double2(1.0, 0.0); };
  float x[8], y[8], top = 0.0f;
  unsigned long long zero = 0ull;  // stays so unless an element is an infinity or a NaN
#pragma unroll
  for (int z = 0; z < 8; ++z) {
    float f = 0.0f, g = 0.0f;
    if (live) member<T, true>(raw, u, weave, z, f, g);
    zero = fma2(pack2(f, g), 0ull, zero);
    x[z] = f, y[z] = g;
    if (pair) {
      const float2 w = z < 4 ? w0[z] : w1[z - 4];
      x[z] = fmaf(f, w.x, -g * w.y);
      y[z] = fmaf(g, w.x, f * w.y);
    }
    top = fmax3(top, fabsf(x[z]), fabsf(y[z]));
  }
  float z0, z1;
  unpack2(zero, z0, z1);
  const uint32_t odd = __ballot_sync(0xffffffffu, !(z0 + z1 == 0.0f));
  for (int o = UP >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  double most = 0.0;
  // Twice the error bound, 2^-20 of at most 2 top.  In rows near the type's end,
  // where sums may overflow, every element is computed in 64 bits.
  const bool huge = !(top < 0x1p120f);
  const float near = huge ? 0.0f : top - top * 0x1.1p-18f;
#pragma unroll
  for (int z = 0; z < 8; ++z) {
    if (fmaxf(fabsf(x[z]), fabsf(y[z])) >= near) {
      float f = 0.0f, g = 0.0f;
      if (live) member<T, true>(raw, u, weave, z, f, g);
      const double2 d = exact(z);
      const double a = f, b = g;
      most = fmax(most, fmax(fabs(fma(a, d.x, -(b * d.y))), fabs(fma(b, d.x, a * d.y))));
    }
  }
  for (int o = UP >> 1; o > 0; o >>= 1) most = fmax(most, __shfl_xor_sync(0xffffffffu, most, o));
  float scale = static_cast<float>(most / 448.0);
  const int lane = threadIdx.x & 31;
  const uint32_t row = (UP == 32 ? 0xffffffffu : (1u << UP) - 1u) << (lane & ~(UP - 1));
  if ((odd & row) || !(scale < INFINITY)) scale = __int_as_float(0x7fc00000);
  if (!live) return;
  // Small rows are multiplied up, huge ones down (by a power of two): neither
  // the reciprocal nor a sum may leave the normal range.
  const float up = huge ? 0x1p-8f : scale < 0x1p-60f ? 0x1p80f : 1.0f;
  if (up != 1.0f) {
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      float f, g;
      member<T, true>(raw, u, weave, z, f, g);
      f *= up, g *= up;
      const float2 w = pair ? (z < 4 ? w0[z] : w1[z - 4]) : make_float2(1.0f, 0.0f);
      x[z] = fmaf(f, w.x, -g * w.y);
      y[z] = fmaf(g, w.x, f * w.y);
    }
  }
  const float s = scale * up, inv = scale > 0.0f ? 1.0f / s : 0.0f;
  // per |f| + |g|: 2^-20 for the turn, 2^-21 for the quotient
  const float grain = pair ? fabsf(magnitude) * 0x1.8p-20f * inv : 0x1p-21f * inv;
  uint32_t wa[2] = {0u, 0u}, wb[2] = {0u, 0u};
#pragma unroll
  for (int z = 0; z < 8; ++z) {
    float f, g;
    member<T, true>(raw, u, weave, z, f, g);
    const float d = fmaf(fabsf(g), up, fabsf(f) * up) * grain;
    const unsigned long long q = mul2(pack2(x[z], y[z]), splat2(inv));
    float a, b, c, e;
    unpack2(sub2(q, splat2(d)), a, b);
    unpack2(add2(q, splat2(d)), c, e);
    uint32_t two = e4m3_pair(a, b);
    const uint32_t over = e4m3_pair(c, e);
    if (two != over) {
      const double2 t = exact(z);
      uint32_t cx = two & 0xffu, cy = two >> 8;
      if (cx != (over & 0xffu)) cx = nearer_code(cx, over & 0xffu, f, g, t.x, t.y, scale);
      if (cy != over >> 8) cy = nearer_code(cy, over >> 8, g, f, t.x, -t.y, scale);
      two = cx | cy << 8;
    }
    if (weave) {
      (z < 4 ? wa : wb)[(z & 3) >> 1] |= two << (z & 1 ? 16 : 0);
    } else {
      wa[z >> 2] |= (two & 0xffu) << 8 * (z & 3);
      wb[z >> 2] |= (two >> 8) << 8 * (z & 3);
    }
  }
  *reinterpret_cast<uint2*>(out + u.a) = make_uint2(wa[0], wa[1]);
  *reinterpret_cast<uint2*>(out + u.b) = make_uint2(wb[0], wb[1]);
  if (first_lane) *scale_out = scale;
}

// The same for a unit of any layout, turned or not: codes, and the scale from
// the row's first lane.  All lanes of the row take part (live: whether this one stores; the
// others' elements are zeros).  Elements are unpacked and turned twice, for
// the maximum and for the codes, rather than held.
template <typename T, bool INTER>
__device__ __forceinline__ void code_unit(const Raw<T>& raw, const Unit& u, int UP, bool first_lane, bool live, bool pair,
                                          bool turned_row, float magnitude, const float2* w0, const float2* w1,
                                          const double2* cd0, const double2* cd1, uint8_t* out, float* scale_out) {
  const bool weave = INTER && u.weave;
  // e: a bound of the 32-bit error of both members of a pair (angle and
  // functions, two products, a sum: under 8 roundings of each term).
  const float grain = pair ? fabsf(magnitude) * 0x1p-20f : 0.0f;
  const auto at = [&](int z, float& f, float& g, float& x, float& y, float up = 1.0f) {
    f = g = 0.0f;
    if (live) member<T, false>(raw, u, weave, z, f, g);
    f *= up, g *= up;
    x = f, y = g;
    if (pair && z < u.na) {
      const float2 w = z < 4 ? w0[z] : w1[z - 4];
      x = fmaf(f, w.x, -g * w.y);
      y = fmaf(g, w.x, f * w.y);
    }
  };
  const auto exact = [&](int z) {
    return pair && z < u.na ? (z < 4 ? cd0[z] : cd1[z - 4]) : make_double2(1.0, 0.0);
  };
  float top = 0.0f, slack = 0.0f;
  bool odd = false;  // an infinity or a NaN
#pragma unroll
  for (int z = 0; z < 8; ++z) {
    float f, g, x, y;
    at(z, f, g, x, y);
    odd |= !(fabsf(f) < INFINITY) | !(fabsf(g) < INFINITY);
    top = fmax3(top, fabsf(x), fabsf(y));
    slack = fmaxf(slack, fabsf(f) + fabsf(g));
  }
  slack *= grain;
  for (int o = UP >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  odd = __any_sync(0xffffffffu, odd);
  if (odd) {  // some row of the warp: which one
    odd = false;
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      float f, g, x, y;
      at(z, f, g, x, y);
      odd |= !(fabsf(f) < INFINITY) | !(fabsf(g) < INFINITY);
    }
    for (int o = UP >> 1; o > 0; o >>= 1) odd |= __shfl_xor_sync(0xffffffffu, static_cast<int>(odd), o) != 0;
  }
  float scale;
  if (__any_sync(0xffffffffu, turned_row)) {
    for (int o = UP >> 1; o > 0; o >>= 1) slack = fmaxf(slack, __shfl_xor_sync(0xffffffffu, slack, o));
    double most = 0.0;
    const float near = top < 0x1p120f ? top - 2.0f * slack : 0.0f;  // (sums may overflow)
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      float f, g, x, y;
      at(z, f, g, x, y);
      if (fmaxf(fabsf(x), fabsf(y)) >= near) {
        const double2 d = exact(z);
        const double a = f, b = g;
        most = fmax(most, fmax(fabs(fma(a, d.x, -(b * d.y))), fabs(fma(b, d.x, a * d.y))));
      }
    }
    for (int o = UP >> 1; o > 0; o >>= 1) most = fmax(most, __shfl_xor_sync(0xffffffffu, most, o));
    scale = static_cast<float>(most / 448.0);
  } else {
    scale = __fdiv_rn(top, 448.0f);
  }
  if (odd || !(scale < INFINITY)) scale = __int_as_float(0x7fc00000);
  if (!live) return;
  // Small rows are multiplied up, huge ones down (by a power of two): neither
  // the reciprocal nor a remainder or a sum may leave the normal range.
  const float up = !(top < 0x1p120f) ? 0x1p-8f : scale < 0x1p-60f ? 0x1p80f : 1.0f;
  const float s = scale * up, inv = scale > 0.0f ? 1.0f / s : 0.0f;
#pragma unroll
  for (int z = 0; z < 8; ++z) {
    float f, g, x, y;
    at(z, f, g, x, y, up);
    uint32_t cx, cy;
    if (turned_row) {
      const float qx = x * inv, qy = y * inv, e = (fabsf(f) + fabsf(g)) * grain * inv;
      const float dx = fmaf(fabsf(qx), 0x1p-21f, e), dy = fmaf(fabsf(qy), 0x1p-21f, e);
      cx = e4m3_pair(qx - dx, qx + dx);
      cy = e4m3_pair(qy - dy, qy + dy);
      if (((cx ^ cx >> 8) | (cy ^ cy >> 8)) & 0xffu) {
        const double2 d = exact(z);
        if ((cx ^ cx >> 8) & 0xffu) cx = nearer_code(cx & 0xffu, cx >> 8 & 0xffu, f, g, d.x, d.y, s);
        if ((cy ^ cy >> 8) & 0xffu) cy = nearer_code(cy & 0xffu, cy >> 8 & 0xffu, g, f, d.x, -d.y, s);
      }
      cx &= 0xffu, cy &= 0xffu;
    } else {
      const uint32_t two = e4m3_pair(quotient_odd(x, s, inv), quotient_odd(y, s, inv));
      cx = two & 0xffu, cy = two >> 8;
    }
    const int step = u.weave ? 2 : 1;
    if (z < u.na) out[u.a + z * step] = static_cast<uint8_t>(cx);
    if (z < u.nb) out[u.b + z * step] = static_cast<uint8_t>(cy);
  }
  if (first_lane) *scale_out = scale;
}

// A thread keeps its lane of the row and goes through rows (passes) and
// tokens; the next row's loads are in flight while it turns and codes one, the
// first one's while the block prepares the angles (two rows at a time spill:
// 16-bit writes 56 us for 39).
// WRITE: k and v rows as well, into the pool; E4: in 8 bits.
template <typename T, bool WRITE, bool E4, bool VEC, bool INTER>
__global__ void __launch_bounds__(kRotThreads, E4 ? 3 : VEC ? 4 : 2)
    rotate_kernel(const __grid_constant__ RotateParams p, const __grid_constant__ RotatePlan n) {
  dep_enter();
  __shared__ __align__(16) float2 cs[kRotAngles];
  __shared__ __align__(16) double2 csd[E4 ? kRotAngles : 1];
  __shared__ long long dst[kRotGroup], sdst[kRotGroup], pos[kRotGroup];
  const int tid = threadIdx.x;
  const bool turn = p.inv_freq != nullptr;
  const int half_rd = p.rd / 2;
  const int slot = tid / n.UP, lane = tid - slot * n.UP;
  const Unit turned = unit_at<VEC>(lane, turn, p.rd, p.D, INTER), plain = unit_at<VEC>(lane, false, 0, p.D, false);
  const int a0 = angle_of<VEC>(0, lane, p.rd, turned.weave), a1 = angle_of<VEC>(4, lane, p.rd, turned.weave);
  const int rows = p.Hq + (WRITE ? 2 * p.c.heads : 0);
  // an even share of the tokens, a group at a time
  const long long t1 = p.tokens * (blockIdx.x + 1ll) / gridDim.x;
  for (long long t0 = p.tokens * blockIdx.x / gridDim.x; t0 < t1; t0 += n.group) {
    const int group = static_cast<int>(min(static_cast<long long>(n.group), t1 - t0));
    int k = 0, pass = 0, place = slot;  // next row to load, and its token's places in q, k and v
    int b = quotient(static_cast<int>(t0), n.div_N), j = static_cast<int>(t0) - b * p.N;
    const T *q_at = nullptr, *k_at = nullptr, *v_at = nullptr;
    const int all = group * n.passes;
    struct Row {
      Raw<T> raw;
      int k, r;
    };
    const auto fetch = [&](Row& x, int it) {
      if (pass == 0 && it < all) {
        q_at = static_cast<const T*>(p.q.p) + b * p.q.sb + j * p.q.sn;
        if (WRITE) {
          k_at = static_cast<const T*>(p.k.p) + b * p.k.sb + j * p.k.sn;
          v_at = static_cast<const T*>(p.v.p) + b * p.v.sb + j * p.v.sn;
        }
      }
      const int r = pass * n.rows + place;
      const bool in = it < all && slot < n.rows && r < rows;
      x.k = k;
      x.r = in ? r : -1;
      if (in) {
        if (!WRITE || r < p.Hq)
          load_raw<T, VEC>(q_at + r * p.q.sh, turned, x.raw);
        else if (r < p.Hq + p.c.heads)
          load_raw<T, VEC>(k_at + (r - p.Hq) * p.k.sh, turned, x.raw);
        else
          load_raw<T, VEC>(v_at + (r - p.Hq - p.c.heads) * p.v.sh, plain, x.raw);
      }
      if (++pass == n.passes) {
        pass = 0;
        ++k;
        // a warp's rows move on with the tokens: some are more work
        if (E4 && (place += n.turn) >= n.rows) place -= n.rows;
        if (++j == p.N) {
          j = 0;
          ++b;
        }
      }
    };
    const auto finish = [&](const Row& x, int it) {
      if (it >= all) return;
      const int r = x.r;
      const long long at = dst[x.k];
      const int base = x.k * half_rd;
      float f[8], g[8];
      float2 w[8];
      if (!WRITE || r < p.Hq) {
        if (r >= 0 && at != -2 && turned.na > 0) {
          unpack_raw<T, VEC>(x.raw, turned, f, g);
          if (turned.pair) {
            load_angles<VEC>(cs + base + a0, cs + base + a1, turned.na, w);
            turn_unit<VEC>(turned, w, f, g);
          }
          store_unit<T, VEC>(static_cast<T*>(p.q_out) + (t0 + x.k) * p.qo_st + r * p.qo_sh, turned, f, g);
        }
      }
      if (WRITE) {
        const bool mine = r >= p.Hq, key = mine && r < p.Hq + p.c.heads;
        const int h = r - p.Hq - (key ? 0 : p.c.heads);
        const Unit& u = key ? turned : plain;
        const bool live = mine && at >= 0;
        const bool pair = key && turned.pair;
        if (E4) {
          if (__any_sync(0xffffffffu, live)) {
            uint8_t* const to = static_cast<uint8_t*>(key ? p.c.k : p.c.v) + at + h * p.c.head_stride;
            float* const scale = (key ? p.c.ks : p.c.vs) + sdst[x.k] + static_cast<long long>(h) * p.c.page_size;
            const float2 *w0 = cs + base + a0, *w1 = cs + base + a1;
            const double2 *cd0 = csd + (E4 ? base + a0 : 0), *cd1 = csd + (E4 ? base + a1 : 0);
            const bool mine_live = live && u.na > 0;
            if constexpr (!VEC)
              code_unit<T, INTER>(x.raw, u, n.UP, lane == 0, mine_live, pair, key && turn, p.magnitude, w0, w1, cd0, cd1, to, scale);
            else if (__any_sync(0xffffffffu, live && key && turn))
              code_turned_unit<T, INTER>(x.raw, u, n.UP, lane == 0, mine_live, pair, p.magnitude, w0, w1, cd0, cd1, to, scale);
            else
              code_exact_unit<T>(x.raw, u, n.UP, lane == 0, mine_live, to, scale);
          }
        } else if (live && u.na > 0) {
          unpack_raw<T, VEC>(x.raw, u, f, g);
          if (pair) {
            load_angles<VEC>(cs + base + a0, cs + base + a1, u.na, w);
            turn_unit<VEC>(u, w, f, g);
          }
          store_unit<T, VEC>(static_cast<T*>(key ? p.c.k : p.c.v) + at + h * p.c.head_stride, u, f, g);
        }
      }
    };
    Row x, y;
    fetch(x, 0);
    prepare_tokens<E4>(p, n, t0, group, cs, csd, dst, sdst, pos);
#pragma unroll 1
    for (int it = 0; it < all; ++it) {
      fetch(y, it + 1);
      finish(x, it);
      if (WRITE) {  // (long code: not twice)
        x = y;
      } else {
        ++it;
        fetch(x, it + 1);
        finish(y, it);
      }
    }
  }
}

template <typename T>
static cudaError_t launch_rotate_t(const RotateParams& p, bool e4, bool vec, int sms, cudaStream_t st) {
  RotatePlan n{};
  const int np = p.inv_freq ? (p.rd / 2 + 7) / 8 + (p.D - p.rd + 15) / 16 : 0;
  n.units = p.write || !p.inv_freq ? (p.D + 15) / 16 : 0;
  if (np > n.units) n.units = np;
  n.UP = n.units;
  if (e4)
    for (n.UP = 1; n.UP < n.units;) n.UP <<= 1;
  // As few passes as the block's size allows, with as few idle threads.
  const int rows = p.Hq + (p.write ? 2 * p.c.heads : 0);
  const int most = kRotThreads / n.UP;  // whole rows that a block has threads for
  n.passes = (rows + most - 1) / most;
  n.rows = (rows + n.passes - 1) / n.passes;
  n.turn = n.rows > 32 / n.UP ? 32 / n.UP : 0;
  const int threads = (n.rows * n.UP + 31) / 32 * 32;
  // blocks that fit at once (64 registers a thread, 80 or 128 in the larger forms)
  const long long fit = static_cast<long long>(sms) * ((e4 ? 768 : vec ? 1024 : 512) / threads);
  const int blocks = static_cast<int>(p.tokens < fit ? p.tokens : fit);
  n.group = kRotGroup;
  if (p.rd > 0 && n.group > kRotAngles / (p.rd / 2)) n.group = kRotAngles / (p.rd / 2);
  // groups of one size in a block's share
  const long long share = (p.tokens + blocks - 1) / blocks, rounds = (share + n.group - 1) / n.group;
  n.group = static_cast<int>((share + rounds - 1) / rounds);
  n.div_N = make_udiv(static_cast<unsigned int>(p.N));
  n.div_half = make_udiv(static_cast<unsigned int>(p.rd > 0 ? p.rd / 2 : 1));
  const auto pick = [&](auto write, auto coded, auto wide) {
    constexpr bool W = decltype(write)::value, E = decltype(coded)::value, V = decltype(wide)::value;
    return p.interleaved ? rotate_kernel<T, W, E, V, true> : rotate_kernel<T, W, E, V, false>;
  };
  const std::true_type yes{};
  const std::false_type no{};
  void (*k)(const RotateParams, const RotatePlan) =
      !p.write ? (vec ? pick(no, no, yes) : pick(no, no, no))
      : e4     ? (vec ? pick(yes, yes, yes) : pick(yes, yes, no))
               : (vec ? pick(yes, no, yes) : pick(yes, no, no));
  return counted(launch_k(SV_PDL >= 2, k, dim3(blocks), dim3(threads), 0, st, p, n), 1);
}

cudaError_t launch_rotate(const RotateParams& p, int dtype, int cache_dtype, bool vec, int sms,
                          cudaStream_t st) {
  if (p.tokens <= 0) return cudaSuccess;
  const bool e4 = p.write && cache_dtype == 3;
  if (dtype == 0) return launch_rotate_t<float>(p, e4, vec, sms, st);
  if (dtype == 1) return launch_rotate_t<__nv_bfloat16>(p, e4, vec, sms, st);
  return launch_rotate_t<__half>(p, e4, vec, sms, st);
}

// ------------------------------------------------------------ read-back
//
// A block takes up to 32 packed rows (fewer where there are few): one lane a
// row finds its sequence (the last b with offsets[b] <= r) and its page, then
// all threads convert (row, k or v, head) runs of 16 elements (8 where a head
// has no whole number of them or 8-bit rows lie on 8-byte boundaries only, or
// single ones where rows are unaligned: 74, 92 and 233 us for 32 sequences of
// 500 to 4096 tokens), four of a thread's runs in flight at once.

constexpr int kReadRows = 32;

template <typename C, typename O, bool VEC, int RUN>
__global__ void __launch_bounds__(256) cache_read_kernel(const __grid_constant__ CacheReadParams p, int rows, UDiv div_row,
                                                         UDiv div_kv, UDiv div_head) {
  dep_enter();
  __shared__ long long src[kReadRows];   // element offset of the token, -1: zeros, -2: no row
  __shared__ long long ssrc[kReadRows];  // scale offset of head 0
  const long long r0 = static_cast<long long>(blockIdx.x) * rows;
  if (threadIdx.x < rows) {
    const long long r = r0 + threadIdx.x;
    long long at = -2, sat = 0;
    if (r < p.total && r >= __ldg(p.offsets) && r < __ldg(p.offsets + p.B)) {
      int lo = 0, hi = p.B;  // offsets[lo] <= r < offsets[hi]
      while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (__ldg(p.offsets + m) <= r) lo = m; else hi = m;
      }
      long long pos = r - __ldg(p.offsets + lo);
      if (p.start) pos += max(0, __ldg(p.start + lo));
      int page, place;
      at = -1;
      if (pos >= 0 && find_place(p.c, lo, pos, page, place, p.ctrl)) {
        at = page * p.c.page_stride + place * p.c.token_stride;
        sat = static_cast<long long>(page) * p.c.heads * p.c.page_size + place;
      }
    }
    src[threadIdx.x] = at;
    ssrc[threadIdx.x] = sat;
  }
  __syncthreads();
  constexpr bool kCodes = sizeof(C) == 1;
  constexpr int kAhead = 4;
  const int runs = static_cast<int>(div_head.d), per_kv = static_cast<int>(div_kv.d), per_row = static_cast<int>(div_row.d);
  const int all = rows * per_row;
  for (int i0 = threadIdx.x; i0 < all; i0 += 256 * kAhead) {
    alignas(16) C c[kAhead][RUN];
    float scale[kAhead];
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      const int i = i0 + z * 256;
      if (i >= all) continue;
      const int row = quotient(i, div_row), x = i - row * per_row;
      const int kv = quotient(x, div_kv), y = x - kv * per_kv;
      const int h = quotient(y, div_head), e = (y - h * runs) * RUN;
      const long long at = src[row];
      if (at < 0) continue;
      const C* from = static_cast<const C*>(kv ? p.c.v : p.c.k) + at + h * p.c.head_stride + e;
      if (VEC) {
        constexpr int kBytes = RUN * sizeof(C);
        if (kBytes == 8) {
          *reinterpret_cast<uint2*>(c[z]) = *reinterpret_cast<const uint2*>(from);
        } else {
#pragma unroll
          for (int w = 0; w < kBytes / 16; ++w) reinterpret_cast<uint4*>(c[z])[w] = reinterpret_cast<const uint4*>(from)[w];
        }
      } else {
#pragma unroll
        for (int m = 0; m < RUN; ++m)
          if (e + m < p.c.dim) c[z][m] = from[m];
      }
      if (kCodes) scale[z] = __ldg((kv ? p.c.vs : p.c.ks) + ssrc[row] + static_cast<long long>(h) * p.c.page_size);
    }
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      const int i = i0 + z * 256;
      if (i >= all) continue;
      const int row = quotient(i, div_row), x = i - row * per_row;
      const int kv = quotient(x, div_kv), y = x - kv * per_kv;
      const int h = quotient(y, div_head), e = (y - h * runs) * RUN;
      const long long at = src[row];
      if (at == -2) continue;
      O* o = static_cast<O*>(kv ? p.v_out : p.k_out) + ((r0 + row) * p.c.heads + h) * p.c.dim + e;
#pragma unroll
      for (int half = 0; half < RUN; half += 8) {
        float f[8] = {};
        if (at >= 0) {
          if (VEC) {
            load8(c[z] + half, f);
          } else {
#pragma unroll
            for (int m = 0; m < 8; ++m)
              if (e + m < p.c.dim) f[m] = elem_f32(c[z][m]);
          }
          if (kCodes) {
#pragma unroll
            for (int m = 0; m < 8; ++m) f[m] *= scale[z];
          }
        }
        if (VEC) {
          store8(o + half, f);
        } else {
#pragma unroll
          for (int m = 0; m < 8; ++m)
            if (e + m < p.c.dim) o[m] = from_f32<O>(f[m]);
        }
      }
    }
  }
}

template <typename C>
static cudaError_t launch_read_c(const CacheReadParams& p, int out_dtype, bool vec, bool on16, int sms, cudaStream_t st) {
  int rows = kReadRows;  // a block's: as many as leave two blocks for each SM
  while (rows > 1 && p.total < 2ll * sms * rows) rows /= 2;
  const dim3 grid(static_cast<unsigned int>((p.total + rows - 1) / rows));
  void (*k)(const CacheReadParams, int, UDiv, UDiv, UDiv);
  const bool wide = vec && on16 && p.c.dim % 16 == 0;  // 16 codes are one 16-byte load
  const auto pick = [&](auto out) {
    using O = decltype(out);
    return wide ? cache_read_kernel<C, O, true, 16> : vec ? cache_read_kernel<C, O, true, 8> : cache_read_kernel<C, O, false, 8>;
  };
  k = out_dtype == 0 ? pick(float{}) : out_dtype == 1 ? pick(__nv_bfloat16{}) : pick(__half{});
  const unsigned int runs = static_cast<unsigned int>(wide ? p.c.dim / 16 : (p.c.dim + 7) / 8), heads = static_cast<unsigned int>(p.c.heads);
  return counted(launch_k(SV_PDL >= 2, k, grid, dim3(256), 0, st, p, rows, make_udiv(2 * heads * runs), make_udiv(heads * runs),
                          make_udiv(runs)),
                 1);
}

cudaError_t launch_cache_read(const CacheReadParams& p, int cache_dtype, int out_dtype, bool vec, bool on16, int sms,
                              cudaStream_t st) {
  if (p.total <= 0 || p.B <= 0) return cudaSuccess;
  if (cache_dtype == 0) return launch_read_c<float>(p, out_dtype, vec, on16, sms, st);
  if (cache_dtype == 1) return launch_read_c<__nv_bfloat16>(p, out_dtype, vec, on16, sms, st);
  if (cache_dtype == 2) return launch_read_c<__half>(p, out_dtype, vec, on16, sms, st);
  return launch_read_c<__nv_fp8_e4m3>(p, out_dtype, vec, on16, sms, st);
}

// ---------------------------------------------------------------- commit
//
// A thread owns one column (16 bytes, or one element) of one (layer, k or v,
// head) and moves it through the sequence's accepted nodes in order, four at a
// time.  Row j only receives from rows after j, so a row is always read before
// it is overwritten (those of one four are read before any of them is
// written), and no two threads touch the same bytes.  64 paths of up to 8
// nodes in 32 layers: 18 us, with single elements 57.

__device__ __forceinline__ void write_len(const CacheCommitParams& p, int b, int n, long long len) {
  const long long end = len + n + 1;
  long long cap = static_cast<long long>(p.c.max_pages) * p.c.page_size;
  if (cap > 0x7fffffffll) cap = 0x7fffffffll;
  if (end > cap) raise_flag(p.ctrl, kFlagCapacity);
  p.new_len[b] = static_cast<int>(end < cap ? end : cap);
}

template <typename W>
__global__ void __launch_bounds__(256) cache_commit_kernel(const CacheCommitParams p, int words, int es) {
  dep_enter();
  const int b = blockIdx.y;
  const int n = min(max(__ldg(p.accepted + b), 0), p.N - 1);
  const long long len = max(0, __ldg(p.cache_len + b));
  __shared__ long long off[64], soff[64], dst[64], sdst[64];  // element and scale offsets of the moves
  __shared__ int moves;
  if (threadIdx.x < 64) {
    const int j = threadIdx.x;
    long long a = -1, as = -1, d = -1, ds = -1;
    if (p.path && j >= 1 && j <= n) {
      const int from = __ldg(p.path + static_cast<long long>(b) * p.N + j);
      Ctrl* ctrl = blockIdx.x == 0 ? p.ctrl : nullptr;
      int page, place;
      if (from < j || from >= p.N) {
        raise_flag(ctrl, kFlagInvalidTree);
      } else if (from > j && find_place(p.c, b, len + j, page, place, ctrl)) {
        d = page * p.c.page_stride + place * p.c.token_stride;
        ds = static_cast<long long>(page) * p.c.heads * p.c.page_size + place;
        if (find_place(p.c, b, len + from, page, place, ctrl)) {
          a = page * p.c.page_stride + place * p.c.token_stride;
          as = static_cast<long long>(page) * p.c.heads * p.c.page_size + place;
        }
      }
    }
    // the moves in order, without gaps
    __shared__ unsigned int in[2];
    const unsigned int word = __ballot_sync(0xffffffffu, a >= 0);
    if ((j & 31) == 0) in[j >> 5] = word;
    asm volatile("bar.sync 1, 64;" ::: "memory");
    if (a >= 0) {
      const int at = __popc(word & ((1u << (j & 31)) - 1u)) + (j >= 32 ? __popc(in[0]) : 0);
      off[at] = a, soff[at] = as, dst[at] = d, sdst[at] = ds;
    }
    if (j == 0) moves = __popc(in[0]) + __popc(in[1]);
  }
  __syncthreads();
  // When new_len is cache_len or accepted_len, which other blocks may still
  // have to read, the lengths are written by a grid of their own instead.
  if (!p.apart && blockIdx.x == 0 && threadIdx.x == 0) write_len(p, b, n, len);
  const int per_head = words + (p.c.ks ? 1 : 0);
  const long long items = static_cast<long long>(p.c.layers) * 2 * p.c.heads * per_head;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < items; i += gridDim.x * 256ll) {
    const int w = static_cast<int>(i % per_head);
    long long x = i / per_head;
    const int h = static_cast<int>(x % p.c.heads);
    x /= p.c.heads;
    const int kv = static_cast<int>(x & 1);
    const long long layer = x >> 1;
    if (w < words) {
      unsigned char* base = static_cast<unsigned char*>(kv ? p.c.v : p.c.k);
      const long long col = layer * p.c.layer_stride + h * p.c.head_stride;
      for (int j = 0; j < moves; j += 4) {
        W v[4];
#pragma unroll
        for (int z = 0; z < 4; ++z)
          if (j + z < moves) v[z] = reinterpret_cast<const W*>(base + (col + off[j + z]) * es)[w];
#pragma unroll
        for (int z = 0; z < 4; ++z)
          if (j + z < moves) reinterpret_cast<W*>(base + (col + dst[j + z]) * es)[w] = v[z];
      }
    } else {
      float* base = (kv ? p.c.vs : p.c.ks) + layer * p.c.scale_layer_stride +
                    static_cast<long long>(h) * p.c.page_size;
      for (int j = 0; j < moves; ++j) base[sdst[j]] = base[soff[j]];
    }
  }
}

__global__ void cache_len_kernel(const CacheCommitParams p) {
  dep_enter();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.B) return;
  write_len(p, b, min(max(p.accepted[b], 0), p.N - 1), max(0, p.cache_len[b]));
}

cudaError_t launch_cache_commit(const CacheCommitParams& p, int es, bool vec, int sms, cudaStream_t st) {
  if (p.B <= 0) return cudaSuccess;
  const bool moves = p.path && p.N > 1;
  if (moves) {
    const int wb = vec ? 16 : es;
    const int words = p.c.dim * es / wb;
    const long long items = static_cast<long long>(p.c.layers) * 2 * p.c.heads * (words + (p.c.ks ? 1 : 0));
    // one wave of blocks: each looks up its sequence's places once
    const long long blocks = (items + 255) / 256, most = 8ll * sms / p.B + 1;
    const dim3 grid(static_cast<unsigned int>(blocks < most ? blocks : most), static_cast<unsigned int>(p.B));
    void (*k)(const CacheCommitParams, int, int) = wb == 16  ? cache_commit_kernel<uint4>
                                                   : wb == 4 ? cache_commit_kernel<uint32_t>
                                                   : wb == 2 ? cache_commit_kernel<uint16_t>
                                                             : cache_commit_kernel<uint8_t>;
    const cudaError_t e = counted(launch_k(SV_PDL >= 2, k, grid, dim3(256), 0, st, p, words, es), 1);
    if (e != cudaSuccess || !p.apart) return e;
  }
  return counted(
      launch_k(SV_PDL >= 2, cache_len_kernel, dim3((p.B + 127) / 128), dim3(128), 0, st, p), 1);
}

}  // namespace sv
