// sv_attention.cu -- attention of drafted tokens over the paged cache.
//
// Row (b, i, h): softmax over the context and node i's ancestors, in one pass
// with a running maximum m, sum l and output o: a new score s > m scales l
// and o by 2^(m - s) (scores in log2 units).
#include "sv_cache_device.cuh"

namespace sv {

// Node i's ancestors and itself as a bit set; 0 for a padding node or one at
// or below an invalid parent.
__device__ __forceinline__ unsigned long long ancestor_bits(const int* parent, int i, int n_nodes,
                                                            Ctrl* ctrl) {
  if (i >= n_nodes) return 0ull;
  if (!parent) return i == 63 ? ~0ull : (2ull << i) - 1ull;
  unsigned long long m = 1ull << i;
  while (i > 0) {
    const int up = __ldg(parent + i);
    if (up < 0 || up >= i) {
      raise_flag(ctrl, kFlagInvalidTree);
      return 0ull;
    }
    m |= 1ull << up;
    i = up;
  }
  return m;
}

// The plain form, for the layouts that the tensor cores' form does not take
// (heads over 128 elements, or rows, pages or scales that a tensor map cannot
// address): one block a row, its warps take every fourth token, a lane every
// 32nd element of the head.  Each row reads all keys and values itself, which
// bounds it: one user's chain of 5 over 500 tokens takes 109 us for the other
// form's 12, 64 trees of 26 nodes 23.7 ms for 0.14.  Over ten tokens both take
// a launch's latency (8.6 and 11 us).
template <typename T, typename C>
__global__ void __launch_bounds__(128) attention_plain_kernel(const AttnParams p) {
  dep_enter();
  constexpr int kE = 8;  // head_dim <= 256
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = blockIdx.x;
  const int h = static_cast<int>(x % p.Hq);
  x /= p.Hq;
  const int i = static_cast<int>(x % p.N);
  const int b = static_cast<int>(x / p.N);
  const int D = p.c.dim, hk = h / p.G;
  const int nodes = p.count ? min(max(__ldg(p.count + b), 0), p.N) : p.N;
  const long long len = max(0, __ldg(p.cache_len + b));
  const unsigned long long bits =
      ancestor_bits(p.parent ? p.parent + static_cast<long long>(b) * p.N : nullptr, i, nodes, p.ctrl);
  const T* q = static_cast<const T*>(p.q.p) + b * p.q.sb + i * p.q.sn + h * p.q.sh;
  float qf[kE], o[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    qf[e] = lane + 32 * e < D ? elem_f32(q[lane + 32 * e]) : 0.0f;
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  // (tokens past the capacity have no place: no look at each of them)
  const long long cap = min(static_cast<long long>(p.c.max_pages) * p.c.page_size, 0x7fffffffll);
  const long long end = bits ? min(len + nodes, cap) : 0;
  if (threadIdx.x == 0 && i == 0 && h == 0 && nodes > 0 && len + nodes > cap) raise_flag(p.ctrl, kFlagCapacity);
  for (long long t = warp; t < end; t += 4) {
    if (t >= len && !(bits >> (t - len) & 1ull)) continue;
    int page, place;
    if (!find_place(p.c, b, t, page, place, p.ctrl)) continue;
    const long long at = page * p.c.page_stride + place * p.c.token_stride + hk * p.c.head_stride;
    const C* k = static_cast<const C*>(p.c.k) + at;
    const C* v = static_cast<const C*>(p.c.v) + at;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (lane + 32 * e < D) s = fmaf(qf[e], elem_f32(k[lane + 32 * e]), s);
    s = warp_sum(s) * p.c2;
    float vs = 1.0f;
    if (sizeof(C) == 1) {
      const long long sat = (static_cast<long long>(page) * p.c.heads + hk) * p.c.page_size + place;
      s *= p.c.ks[sat];
      vs = p.c.vs[sat];
    }
    if (s == -INFINITY) continue;
    const float mn = fmaxf(m, s);
    const float w = exp2f(s - mn);
    const float r = m == -INFINITY ? 0.0f : exp2f(m - mn);
    m = mn;
    l = fmaf(l, r, w);
    const float wv = w * vs;
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (lane + 32 * e < D) o[e] = fmaf(o[e], r, wv * elem_f32(v[lane + 32 * e]));
  }
  __shared__ float sm[4], sl[4], so[4][256];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int e = 0; e < kE; ++e) so[warp][lane + 32 * e] = o[e];
  __syncthreads();
  const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float r[4], L = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    r[w] = sm[w] == -INFINITY ? 0.0f : exp2f(sm[w] - M);
    // a NaN score leaves no maximum behind, only a NaN sum
    if (sl[w] != sl[w]) r[w] = sl[w];
    L += sl[w] * r[w];
  }
  const long long row = (static_cast<long long>(b) * p.N + i) * p.Hq + h;
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  for (int d = threadIdx.x; d < D; d += 128) {
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (r[w] != 0.0f) y += so[w][d] * r[w];
    static_cast<T*>(p.out)[row * D + d] = from_f32<T>(L == 0.0f ? 0.0f : y * inv);
  }
  if (p.lse && threadIdx.x == 0) p.lse[row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
}

cudaError_t launch_attention_plain(const AttnParams& p, int q_dtype, int cache_dtype,
                                   cudaStream_t st) {
  const dim3 grid(static_cast<unsigned int>(static_cast<long long>(p.B) * p.N * p.Hq));
  void (*k)(const AttnParams);
  if (q_dtype == 1)
    k = cache_dtype == 3 ? attention_plain_kernel<__nv_bfloat16, __nv_fp8_e4m3>
                         : attention_plain_kernel<__nv_bfloat16, __nv_bfloat16>;
  else
    k = cache_dtype == 3 ? attention_plain_kernel<__half, __nv_fp8_e4m3>
                         : attention_plain_kernel<__half, __half>;
  return counted(launch_k(SV_PDL >= 2, k, grid, dim3(128), 0, st, p), 1);
}

}  // namespace sv
