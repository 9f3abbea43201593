// sv_cache.cu -- rotary positions, the paged cache's write (as it is, or in
// 8 bits with one scale a row), its read-back and the move of accepted rows.
// All four move data once and are bound by memory, or, for a few tokens, by
// one launch's latency.
#include "sv_cache_device.cuh"

namespace sv {

// ------------------------------------------------- rotary and cache write
//
// One block takes one token at a time: its threads first turn position * f
// into (cos, sin) pairs in shared memory, once for all heads, then each
// group of UP lanes takes one row (a head of q, k or v) and each lane of it
// one unit of 16 elements: 8 whole pairs, or 16 neighbours past rotary_dim.
// The angle is reduced as turns in 64 bits (position * f / 2 pi, minus the
// nearest integer), so it is exact to 1e-10 turns at any 32-bit position;
// cos and sin then work on a half turn at most.
//
// K rows bound for 8 bits are turned in 64 bits, so that their codes are the
// exact rotation's, rounded once; a row's scale needs the largest magnitude
// over the row, one shuffle reduction over its lanes.

constexpr int kRotThreads = 256;

struct Unit {
  int a, b;  // first elements of the two runs of 8 (pairs: first and second members)
  int na, nb;
  bool pair, inter;
};
// `turn`: the row has a rotary part.
__device__ __forceinline__ Unit unit_at(int u, bool turn, int rd, int D, bool inter) {
  Unit x;
  const int np = turn ? (rd / 2 + 7) / 8 : 0;
  x.pair = u < np;
  x.inter = inter;
  if (x.pair) {
    const int n = min(8, rd / 2 - 8 * u);
    x.na = x.nb = n;
    x.a = inter ? 16 * u : 8 * u;
    x.b = inter ? x.a + 1 : rd / 2 + 8 * u;
  } else {
    x.a = (turn ? rd : 0) + 16 * (u - np);
    x.b = x.a + 8;
    x.na = max(0, min(8, D - x.a));
    x.nb = max(0, min(8, D - x.b));
  }
  return x;
}

// f: first members (or the first 8 elements), g: second members (the next 8).
template <typename T, bool VEC>
__device__ __forceinline__ void load_unit(const T* row, const Unit& u, float (&f)[8], float (&g)[8]) {
  if (VEC) {
    if (u.na == 0) return;
    if (u.pair && u.inter) {
      float x[8], y[8];
      load8(row + u.a, x);
      load8(row + u.a + 8, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = x[2 * i], g[i] = x[2 * i + 1];
        f[4 + i] = y[2 * i], g[4 + i] = y[2 * i + 1];
      }
    } else {
      load8(row + u.a, f);
      load8(row + u.b, g);
    }
  } else {
    const int step = u.pair && u.inter ? 2 : 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < u.na) f[i] = elem_f32(row[u.a + i * step]);
      if (i < u.nb) g[i] = elem_f32(row[u.b + i * step]);
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T* row, const Unit& u, const float (&f)[8],
                                           const float (&g)[8]) {
  if (VEC) {
    if (u.na == 0) return;
    if (u.pair && u.inter) {
      float x[8], y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = f[i], x[2 * i + 1] = g[i];
        y[2 * i] = f[4 + i], y[2 * i + 1] = g[4 + i];
      }
      store8(row + u.a, x);
      store8(row + u.a + 8, y);
    } else {
      store8(row + u.a, f);
      store8(row + u.b, g);
    }
  } else {
    const int step = u.pair && u.inter ? 2 : 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < u.na) row[u.a + i * step] = from_f32<T>(f[i]);
      if (i < u.nb) row[u.b + i * step] = from_f32<T>(g[i]);
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* row, const Unit& u, const float (&f)[8],
                                            const float (&g)[8]) {
  uint32_t lo[4], hi[4];  // two codes each
  if (u.pair && u.inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = e4m3_pair(f[i], g[i]);
      hi[i] = e4m3_pair(f[4 + i], g[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = e4m3_pair(f[2 * i], f[2 * i + 1]);
      hi[i] = e4m3_pair(g[2 * i], g[2 * i + 1]);
    }
  }
  const int second = u.pair && u.inter ? u.a + 8 : u.b;
  if (VEC) {
    if (u.na == 0) return;
    *reinterpret_cast<uint2*>(row + u.a) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    *reinterpret_cast<uint2*>(row + second) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
  } else {
    // counts in elements of each run of 8 neighbours
    const int n0 = u.pair && u.inter ? min(8, 2 * u.na) : u.na;
    const int n1 = u.pair && u.inter ? max(0, 2 * u.na - 8) : u.nb;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < n0) row[u.a + i] = static_cast<uint8_t>(lo[i >> 1] >> (8 * (i & 1)));
      if (i < n1) row[second + i] = static_cast<uint8_t>(hi[i >> 1] >> (8 * (i & 1)));
    }
  }
}

// E4: the pool holds codes and scales.  UP: lanes of a row (a power of two).
template <typename T, bool E4, bool VEC>
__global__ void __launch_bounds__(kRotThreads) rotate_kernel(const RotateParams p, int UP) {
  dep_enter();
  __shared__ float2 cs[2][256];
  __shared__ double2 csd[E4 ? 2 : 1][E4 ? 128 : 1];  // cache heads have at most 256 elements
  __shared__ int par[2][64];
  const int tid = threadIdx.x;
  const int lane = tid & (UP - 1);
  const int rows = p.Hq + (p.write ? 2 * p.c.heads : 0);
  const int per_pass = kRotThreads / UP;
  const bool turn = p.inv_freq != nullptr;
  int buf = 0;
  for (long long t = blockIdx.x; t < p.tokens; t += gridDim.x, buf ^= 1) {
    const int b = static_cast<int>(t / p.N);
    const int j = static_cast<int>(t - static_cast<long long>(b) * p.N);
    if (p.count && j >= __ldg(p.count + b)) {
      __syncthreads();
      continue;
    }
    long long len = 0, pos = 0;
    if (p.positions) {
      pos = __ldg(p.positions + t);
    } else {
      len = max(0, __ldg(p.cache_len + b));
      pos = len + j;
      if (p.parent) {
        if (tid < p.N) par[buf][tid] = __ldg(p.parent + static_cast<long long>(b) * p.N + tid);
        __syncthreads();
        int depth = 0;
        for (int x = j; x > 0; ++depth) {  // parents decrease, so this ends
          const int up = par[buf][x];
          if (up < 0 || up >= x) {
            if (tid == 0) raise_flag(p.ctrl, kFlagInvalidTree);
            break;
          }
          x = up;
        }
        pos = len + depth;
      }
    }
    if (turn) {
      for (int i = tid; i < p.rd / 2; i += kRotThreads) {
        const double turns = static_cast<double>(pos) * __ldg(p.inv_freq + i) * 0.15915494309189533577;
        const double half = 2.0 * (turns - rint(turns));
        float s, c;
        sincospif(static_cast<float>(half), &s, &c);
        s = p.inverse ? -s : s;
        cs[buf][i] = make_float2(c * p.magnitude, s * p.magnitude);
        if (E4) {
          double sd, cd;
          sincospi(half, &sd, &cd);
          csd[buf][i] = make_double2(cd * p.magnitude, sd * p.magnitude);
        }
      }
    }
    int page = 0, place = 0;
    const bool placed = p.write && find_place(p.c, b, len + j, page, place, tid == 0 ? p.ctrl : nullptr);
    __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += per_pass) {
      const int r = r0 + tid / UP;
      const int kind = r < p.Hq ? 0 : r < p.Hq + p.c.heads ? 1 : 2;
      const bool live = r < rows && (kind == 0 || placed);
      const int h = kind == 0 ? r : kind == 1 ? r - p.Hq : r - p.Hq - p.c.heads;
      const bool turned = turn && kind < 2;
      const Unit u = unit_at(lane, turned, p.rd, p.D, p.interleaved != 0);
      float f[8] = {}, g[8] = {};
      if (live) {
        const RowsView& src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
        load_unit<T, VEC>(static_cast<const T*>(src.p) + b * src.sb + j * src.sn + h * src.sh, u, f, g);
      }
      if (!E4 || kind == 0) {
        if (u.pair && turned) {
          const int first = 8 * lane;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (VEC || i < u.na) {
              const float2 w = cs[buf][first + i];
              const float x = f[i], y = g[i];
              f[i] = fmaf(x, w.x, -y * w.y);
              g[i] = fmaf(y, w.x, x * w.y);
            }
          }
        }
        if (live) {
          T* dst;
          if (kind == 0)
            dst = static_cast<T*>(p.q_out) + t * p.qo_st + h * p.qo_sh;
          else
            dst = static_cast<T*>(kind == 1 ? p.c.k : p.c.v) + page * p.c.page_stride +
                  place * p.c.token_stride + h * p.c.head_stride;
          store_unit<T, VEC>(dst, u, f, g);
        }
      }
      if (E4) {
        // Every lane takes part in the row's reduction.
        double x[8], y[8];
        double top = 0.0;
        bool odd = false;  // an infinity or a NaN
        if (kind != 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = f[i], y[i] = g[i];
            odd |= !isfinite(f[i]) || !isfinite(g[i]);
            if (u.pair && turned && (VEC || i < u.na)) {
              const double2 w = csd[buf][8 * lane + i];
              const double a = x[i], d = y[i];
              x[i] = fma(a, w.x, -d * w.y);
              y[i] = fma(d, w.x, a * w.y);
            }
            top = fmax(top, fmax(fabs(x[i]), fabs(y[i])));
          }
        }
        for (int o = UP >> 1; o > 0; o >>= 1) {
          top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o, 32));
          odd |= __shfl_xor_sync(0xffffffffu, static_cast<int>(odd), o, 32) != 0;
        }
        if (live && kind != 0) {
          float scale = static_cast<float>(top / 448.0);
          const double s = scale, inv = scale > 0.0f ? 1.0 / s : 0.0;
          if (odd || !isfinite(scale)) scale = __int_as_float(0x7fc00000);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[i] = quotient_odd(x[i], s, inv);
            g[i] = quotient_odd(y[i], s, inv);
          }
          const long long at = page * p.c.page_stride + place * p.c.token_stride + h * p.c.head_stride;
          store_codes<VEC>(static_cast<uint8_t*>(kind == 1 ? p.c.k : p.c.v) + at, u, f, g);
          if (lane == 0)
            (kind == 1 ? p.c.ks : p.c.vs)[(static_cast<long long>(page) * p.c.heads + h) * p.c.page_size +
                                          place] = scale;
        }
      }
    }
  }
}

template <typename T>
static cudaError_t launch_rotate_t(const RotateParams& p, bool e4, bool vec, int sms, cudaStream_t st) {
  const int np = p.inv_freq ? (p.rd / 2 + 7) / 8 + (p.D - p.rd + 15) / 16 : 0;
  int units = p.write || !p.inv_freq ? (p.D + 15) / 16 : 0;
  if (np > units) units = np;
  int up = 1;
  while (up < units) up <<= 1;
  const long long most = static_cast<long long>(sms) * (2048 / kRotThreads);
  const dim3 grid(static_cast<unsigned int>(p.tokens < most ? p.tokens : most));
  void (*k)(const RotateParams, int) = e4 ? (vec ? rotate_kernel<T, true, true> : rotate_kernel<T, true, false>)
                                          : (vec ? rotate_kernel<T, false, true> : rotate_kernel<T, false, false>);
  return counted(launch_k(SV_PDL >= 2, k, grid, dim3(kRotThreads), 0, st, p, up), 1);
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
// A block takes 16 packed rows: one lane a row finds its sequence (the last b
// with offsets[b] <= r) and its page, then all threads convert (row, k or v,
// head) runs of 8 elements.

constexpr int kReadRows = 16;

template <typename C, typename O, bool VEC>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheReadParams p) {
  dep_enter();
  __shared__ long long src[kReadRows];   // element offset of the token, -1: zeros, -2: no row
  __shared__ long long ssrc[kReadRows];  // scale offset of head 0
  const long long r0 = static_cast<long long>(blockIdx.x) * kReadRows;
  if (threadIdx.x < kReadRows) {
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
  const int runs = (p.c.dim + 7) / 8;
  const int per_row = 2 * p.c.heads * runs;
  for (int i = threadIdx.x; i < kReadRows * per_row; i += 256) {
    const int row = i / per_row;
    int x = i - row * per_row;
    const int kv = x / (p.c.heads * runs);
    x -= kv * p.c.heads * runs;
    const int h = x / runs, e = (x - h * runs) * 8;
    const long long at = src[row];
    if (at == -2) continue;
    float f[8] = {};
    const int n = min(8, p.c.dim - e);
    if (at >= 0) {
      const C* c = static_cast<const C*>(kv ? p.c.v : p.c.k) + at + h * p.c.head_stride + e;
      if (VEC) {
        load8(c, f);
      } else {
#pragma unroll
        for (int m = 0; m < 8; ++m)
          if (m < n) f[m] = elem_f32(c[m]);
      }
      if (kCodes) {
        const float s = __ldg((kv ? p.c.vs : p.c.ks) + ssrc[row] + static_cast<long long>(h) * p.c.page_size);
#pragma unroll
        for (int m = 0; m < 8; ++m) f[m] *= s;
      }
    }
    O* o = static_cast<O*>(kv ? p.v_out : p.k_out) + ((r0 + row) * p.c.heads + h) * p.c.dim + e;
    if (VEC) {
      store8(o, f);
    } else {
#pragma unroll
      for (int m = 0; m < 8; ++m)
        if (m < n) o[m] = from_f32<O>(f[m]);
    }
  }
}

template <typename C>
static cudaError_t launch_read_c(const CacheReadParams& p, int out_dtype, bool vec, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned int>((p.total + kReadRows - 1) / kReadRows));
  void (*k)(const CacheReadParams);
  if (out_dtype == 0)
    k = vec ? cache_read_kernel<C, float, true> : cache_read_kernel<C, float, false>;
  else if (out_dtype == 1)
    k = vec ? cache_read_kernel<C, __nv_bfloat16, true> : cache_read_kernel<C, __nv_bfloat16, false>;
  else
    k = vec ? cache_read_kernel<C, __half, true> : cache_read_kernel<C, __half, false>;
  return counted(launch_k(SV_PDL >= 2, k, grid, dim3(256), 0, st, p), 1);
}

cudaError_t launch_cache_read(const CacheReadParams& p, int cache_dtype, int out_dtype, bool vec,
                              cudaStream_t st) {
  if (p.total <= 0 || p.B <= 0) return cudaSuccess;
  if (cache_dtype == 0) return launch_read_c<float>(p, out_dtype, vec, st);
  if (cache_dtype == 1) return launch_read_c<__nv_bfloat16>(p, out_dtype, vec, st);
  if (cache_dtype == 2) return launch_read_c<__half>(p, out_dtype, vec, st);
  return launch_read_c<__nv_fp8_e4m3>(p, out_dtype, vec, st);
}

// ---------------------------------------------------------------- commit
//
// A thread owns one column (16 bytes, or one element) of one (layer, k or v,
// head) and moves it through the sequence's accepted nodes in order.  Row j
// only receives from rows at or after j, so a row is always read before it is
// overwritten, and no two threads touch the same bytes.

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
  __shared__ long long off[64], soff[64], dst[64], sdst[64];  // element and scale offsets, -1: no move
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
    off[j] = a, soff[j] = as, dst[j] = d, sdst[j] = ds;
  }
  __syncthreads();
  // When new_len is cache_len, which other blocks may still have to read, the
  // lengths are written by a grid of their own instead.
  if (p.new_len != p.cache_len && blockIdx.x == 0 && threadIdx.x == 0) write_len(p, b, n, len);
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
      for (int j = 1; j <= n; ++j) {
        if (off[j] < 0) continue;
        const W v = reinterpret_cast<const W*>(base + (col + off[j]) * es)[w];
        reinterpret_cast<W*>(base + (col + dst[j]) * es)[w] = v;
      }
    } else {
      float* base = (kv ? p.c.vs : p.c.ks) + layer * p.c.scale_layer_stride +
                    static_cast<long long>(h) * p.c.page_size;
      for (int j = 1; j <= n; ++j)
        if (off[j] >= 0) base[sdst[j]] = base[soff[j]];
    }
  }
}

__global__ void cache_len_kernel(const CacheCommitParams p) {
  dep_enter();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.B) return;
  write_len(p, b, min(max(__ldg(p.accepted + b), 0), p.N - 1), max(0, p.cache_len[b]));
}

cudaError_t launch_cache_commit(const CacheCommitParams& p, int es, bool vec, cudaStream_t st) {
  if (p.B <= 0) return cudaSuccess;
  const bool moves = p.path && p.N > 1;
  if (moves) {
    const int wb = vec ? 16 : es;
    const int words = p.c.dim * es / wb;
    const long long items = static_cast<long long>(p.c.layers) * 2 * p.c.heads * (words + (p.c.ks ? 1 : 0));
    const long long blocks = (items + 255) / 256;
    const dim3 grid(static_cast<unsigned int>(blocks < 4096 ? blocks : 4096), static_cast<unsigned int>(p.B));
    void (*k)(const CacheCommitParams, int, int) = wb == 16  ? cache_commit_kernel<uint4>
                                                   : wb == 4 ? cache_commit_kernel<uint32_t>
                                                   : wb == 2 ? cache_commit_kernel<uint16_t>
                                                             : cache_commit_kernel<uint8_t>;
    const cudaError_t e = counted(launch_k(SV_PDL >= 2, k, grid, dim3(256), 0, st, p, words, es), 1);
    if (e != cudaSuccess || p.new_len != p.cache_len) return e;
  }
  return counted(
      launch_k(SV_PDL >= 2, cache_len_kernel, dim3((p.B + 127) / 128), dim3(128), 0, st, p), 1);
}

}  // namespace sv
