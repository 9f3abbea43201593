// sv_cache_api.cu -- C ABI of the cache-side calls (include/spec_verify.h):
// argument validation, frequencies, dispatch and the status word.
#include <cmath>

#include "spec_verify.h"
#include "sv_cache.h"

namespace sv {
namespace {

constexpr double kPi = 3.14159265358979323846;

int bytes_of(int dtype) { return dtype == SV_F32 ? 4 : dtype == SV_E4M3 ? 1 : 2; }
bool type_ok(int dtype, bool f32, bool e4m3) {
  return dtype == SV_BF16 || dtype == SV_F16 || (f32 && dtype == SV_F32) || (e4m3 && dtype == SV_E4M3);
}
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool overlap(const int32_t* a, int64_t n, const int32_t* b, int64_t m) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + 4 * m && y < x + 4 * n;
}
bool strides_ok(const sv_rows* r) { return r->stride_b >= 0 && r->stride_n >= 0 && r->stride_h >= 0; }
// Row starts of a strided tensor all on `bytes` boundaries.
bool rows_on(const sv_rows* r, int es, int bytes) {
  return aligned(r->data, bytes) && r->stride_b * es % bytes == 0 && r->stride_n * es % bytes == 0 &&
         r->stride_h * es % bytes == 0;
}
bool pool_on(const sv_kv_cache* c, int es, int bytes) {
  return aligned(c->k, bytes) && aligned(c->v, bytes) && c->page_stride * es % bytes == 0 &&
         c->token_stride * es % bytes == 0 && c->head_stride * es % bytes == 0 &&
         c->layer_stride * es % bytes == 0;
}

// The pool, its table and the batch; `f32`: an fp32 pool is allowed.
int check_cache(const sv_kv_cache* c, const int32_t* table, int64_t table_stride, int max_pages, int B,
                bool f32) {
  if (!c || !c->k || !c->v || !table) return SV_ERR_INVALID_ARG;
  if (!type_ok(c->dtype, f32, true)) return SV_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1 || c->num_heads < 1 || c->num_heads > 1024 || c->head_dim < 1 ||
      c->head_dim > 256 || c->num_layers < 1)
    return SV_ERR_INVALID_ARG;
  if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0 || c->layer_stride < 0 ||
      c->scale_layer_stride < 0 || max_pages < 1 || table_stride < 0 || B > 65535)
    return SV_ERR_INVALID_ARG;
  if ((c->dtype == SV_E4M3) != (c->k_scale != nullptr) || (c->dtype == SV_E4M3) != (c->v_scale != nullptr))
    return SV_ERR_INVALID_ARG;
  const int es = bytes_of(c->dtype);
  if (!aligned(c->k, es) || !aligned(c->v, es) || !aligned(table, 4) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4))
    return SV_ERR_MISALIGNED;
  return SV_OK;
}

CacheView view(const sv_kv_cache* c, const int32_t* table, int64_t table_stride, int max_pages) {
  CacheView v{};
  v.k = c->k, v.v = c->v, v.ks = c->k_scale, v.vs = c->v_scale;
  v.num_pages = c->num_pages, v.page_size = c->page_size, v.heads = c->num_heads, v.dim = c->head_dim;
  v.page_stride = c->page_stride, v.token_stride = c->token_stride, v.head_stride = c->head_stride;
  v.layers = c->num_layers, v.layer_stride = c->layer_stride, v.scale_layer_stride = c->scale_layer_stride;
  v.table = table, v.table_stride = table_stride, v.max_pages = max_pages;
  v.div_page = make_udiv(static_cast<unsigned int>(c->page_size));
  return v;
}

int check_rope(const sv_rotary* r, int D) {
  if (!r->inv_freq || r->rotary_dim < 2 || r->rotary_dim > D || r->rotary_dim % 2 || !std::isfinite(r->magnitude))
    return SV_ERR_INVALID_ARG;
  return aligned(r->inv_freq, 8) ? SV_OK : SV_ERR_MISALIGNED;
}

RowsView rows_view(const sv_rows* r) { return RowsView{r->data, r->stride_b, r->stride_n, r->stride_h}; }

int sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  return n;
}

// Where calls without a workspace report their flags: held by the library, so
// that a captured graph may be replayed at any time.
__device__ Ctrl g_status;

// The control block of a call: the workspace's, or the current device's own.
// Its address is looked up by every call (on the host, under 0.1 us): one kept
// from before the device's primary context was reset would be stale.
int ctrl_of(void* workspace, Ctrl** ctrl) {
  *ctrl = static_cast<Ctrl*>(workspace);
  if (workspace) return SV_OK;
  void* at = nullptr;
  if (cudaGetSymbolAddress(&at, g_status) != cudaSuccess || !at) return SV_ERR_CUDA;
  *ctrl = static_cast<Ctrl*>(at);
  return SV_OK;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int spec_verify_rotary_frequencies(double* inv_freq, float* magnitude, int rotary_dim, double base,
                                              int scaling, double factor, double original_len, double low,
                                              double high) {
  if (!inv_freq || !magnitude || rotary_dim < 2 || rotary_dim > 512 || rotary_dim % 2) return SV_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base) || scaling < SV_ROPE_NONE || scaling > SV_ROPE_YARN)
    return SV_ERR_INVALID_ARG;
  if (scaling != SV_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return SV_ERR_INVALID_ARG;
  if (scaling >= SV_ROPE_BANDS && (!(original_len > 0.0) || !std::isfinite(original_len) || !(low > 0.0) ||
                                   !(high > low) || !std::isfinite(high)))
    return SV_ERR_INVALID_ARG;
  *magnitude = 1.0f;
  double from = 0.0, to = 0.0;  // YaRN: pair indices between which the ramp runs
  if (scaling == SV_ROPE_YARN) {
    // pair index (of rotary_dim / 2) that turns `r` times over original_len
    const auto pair = [&](double r) {
      return rotary_dim * std::log(original_len / (r * 2.0 * kPi)) / (2.0 * std::log(base));
    };
    from = std::fmax(std::floor(pair(high)), 0.0);
    to = std::fmin(std::ceil(pair(low)), rotary_dim - 1.0);
    if (to <= from) to = from + 0.001;
    *magnitude = factor > 1.0 ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rotary_dim);
    double keep = 1.0;  // share of the unscaled frequency
    if (scaling == SV_ROPE_LINEAR) {
      keep = 0.0;
    } else if (scaling == SV_ROPE_BANDS) {
      keep = (original_len * f / (2.0 * kPi) - low) / (high - low);
    } else if (scaling == SV_ROPE_YARN) {
      keep = 1.0 - (i - from) / (to - from);
    }
    keep = std::fmin(std::fmax(keep, 0.0), 1.0);
    inv_freq[i] = scaling == SV_ROPE_NONE ? f : f * (keep + (1.0 - keep) / factor);
  }
  return SV_OK;
}

extern "C" int spec_verify_rotary(const void* x, int dtype, int64_t x_stride_t, int64_t x_stride_h,
                                  const int32_t* positions, const sv_rotary* rope, int inverse, int64_t T,
                                  int H, int D, void* out, int64_t o_stride_t, int64_t o_stride_h,
                                  void* stream) {
  if (!type_ok(dtype, true, false) || T < 0 || T > 0x7fffffffll || H < 1 || H > 1024 || D < 2 || D > 512 ||
      x_stride_t < 0 || x_stride_h < 0 || o_stride_t < 0 || o_stride_h < 0 || !rope)
    return SV_ERR_INVALID_ARG;
  if (T == 0) return SV_OK;
  if (!x || !out || !positions) return SV_ERR_INVALID_ARG;
  if (const int e = check_rope(rope, D)) return e;
  const int es = bytes_of(dtype);
  if (!aligned(x, es) || !aligned(out, es) || !aligned(positions, 4)) return SV_ERR_MISALIGNED;
  RotateParams p{};
  p.q = RowsView{x, 0, x_stride_t, x_stride_h};
  p.Hq = H;
  p.q_out = out, p.qo_st = o_stride_t, p.qo_sh = o_stride_h;
  p.positions = positions;
  p.tokens = T, p.N = static_cast<int>(T), p.D = D;
  p.inv_freq = rope->inv_freq, p.rd = rope->rotary_dim, p.interleaved = rope->interleaved;
  p.magnitude = rope->magnitude, p.inverse = inverse;
  const sv_rows in{x, 0, x_stride_t, x_stride_h}, to{out, 0, o_stride_t, o_stride_h};
  const bool vec = D % 16 == 0 && p.rd % 16 == 0 && rows_on(&in, es, 16) && rows_on(&to, es, 16);
  const int n = sms();
  if (n <= 0) return SV_ERR_CUDA;
  return launch_rotate(p, dtype, dtype, vec, n, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SV_OK
                                                                                                  : SV_ERR_CUDA;
}

extern "C" int spec_verify_cache_write(const sv_kv_cache* cache, const int32_t* page_table,
                                       int64_t table_stride, int max_pages, const int32_t* cache_len,
                                       const int32_t* parent, const int32_t* count, const sv_rows* k,
                                       const sv_rows* v, int dtype, int B, int N, const sv_rotary* rope,
                                       const sv_rows* q, int Hq, void* q_out, void* workspace, void* stream) {
  if (B < 0 || N < 0 || !type_ok(dtype, true, false) || (parent && N > 64)) return SV_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return SV_OK;
  if (const int e = check_cache(cache, page_table, table_stride, max_pages, B, true)) return e;
  if (cache->dtype != dtype && cache->dtype != SV_E4M3) return SV_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * N > 0x7fffffffll) return SV_ERR_INVALID_ARG;
  if (!cache_len || !k || !v || !k->data || !v->data || !strides_ok(k) || !strides_ok(v)) return SV_ERR_INVALID_ARG;
  if (q && (!rope || !q->data || !q_out || !strides_ok(q) || Hq < 1 || Hq > 1024)) return SV_ERR_INVALID_ARG;
  const int D = cache->head_dim;
  if (rope)
    if (const int e = check_rope(rope, D)) return e;
  const int es = bytes_of(dtype), ces = bytes_of(cache->dtype);
  if (!aligned(k->data, es) || !aligned(v->data, es) || (q && (!aligned(q->data, es) || !aligned(q_out, es))) ||
      !aligned(cache_len, 4) || !aligned(parent, 4) || !aligned(count, 4) || !aligned(workspace, 16))
    return SV_ERR_MISALIGNED;
  RotateParams p{};
  if (q) p.q = rows_view(q);
  p.Hq = q ? Hq : 0;
  p.q_out = q_out, p.qo_st = static_cast<long long>(Hq) * D, p.qo_sh = D;
  p.k = rows_view(k), p.v = rows_view(v), p.write = 1;
  p.cache_len = cache_len, p.parent = parent, p.count = count;
  p.tokens = static_cast<long long>(B) * N, p.N = N, p.D = D;
  if (rope) {
    p.inv_freq = rope->inv_freq, p.rd = rope->rotary_dim, p.interleaved = rope->interleaved;
    p.magnitude = rope->magnitude;
  }
  p.c = view(cache, page_table, table_stride, max_pages);
  if (const int e = ctrl_of(workspace, &p.ctrl)) return e;
  const bool vec = D % 16 == 0 && p.rd % 16 == 0 && rows_on(k, es, 16) && rows_on(v, es, 16) &&
                   (!q || (rows_on(q, es, 16) && aligned(q_out, 16))) && pool_on(cache, ces, ces == 1 ? 8 : 16);
  const int n = sms();
  if (n <= 0) return SV_ERR_CUDA;
  return launch_rotate(p, dtype, cache->dtype, vec, n, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

extern "C" int spec_verify_cache_read(const sv_kv_cache* cache, const int32_t* page_table, int64_t table_stride,
                                      int max_pages, const int32_t* offsets, const int32_t* start, int B,
                                      int64_t total, void* k_out, void* v_out, int out_dtype, void* workspace,
                                      void* stream) {
  if (B < 0 || total < 0 || total > 0x7fffffffll || !type_ok(out_dtype, true, false)) return SV_ERR_INVALID_ARG;
  if (B == 0 || total == 0) return SV_OK;
  if (const int e = check_cache(cache, page_table, table_stride, max_pages, B, true)) return e;
  if (!offsets || !k_out || !v_out) return SV_ERR_INVALID_ARG;
  const int oes = bytes_of(out_dtype), ces = bytes_of(cache->dtype);
  if (!aligned(offsets, 4) || !aligned(start, 4) || !aligned(k_out, oes) || !aligned(v_out, oes) ||
      !aligned(workspace, 16))
    return SV_ERR_MISALIGNED;
  CacheReadParams p{};
  p.c = view(cache, page_table, table_stride, max_pages);
  p.offsets = offsets, p.start = start, p.B = B, p.total = total;
  p.k_out = k_out, p.v_out = v_out;
  if (const int e = ctrl_of(workspace, &p.ctrl)) return e;
  const bool vec = cache->head_dim % 8 == 0 && aligned(k_out, 16) && aligned(v_out, 16) &&
                   pool_on(cache, ces, ces == 1 ? 8 : 16);
  const int n = sms();
  if (n <= 0) return SV_ERR_CUDA;
  return launch_cache_read(p, cache->dtype, out_dtype, vec, pool_on(cache, ces, 16), n, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

extern "C" int spec_verify_cache_read_device_status(uint32_t* flags_host, int clear, void* stream) {
  if (!flags_host) return SV_ERR_INVALID_ARG;
  Ctrl* ctrl = nullptr;
  if (const int e = ctrl_of(nullptr, &ctrl)) return e;
  return spec_verify_read_device_status(ctrl, flags_host, clear, stream);
}

extern "C" int spec_verify_cache_commit(const sv_kv_cache* cache, const int32_t* page_table,
                                        int64_t table_stride, int max_pages, const int32_t* cache_len,
                                        const int32_t* accepted_len, const int32_t* path, int B, int N,
                                        int32_t* new_len, void* workspace, void* stream) {
  if (B < 0 || N < 1 || N > 64) return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (const int e = check_cache(cache, page_table, table_stride, max_pages, B, true)) return e;
  if (!cache_len || !accepted_len || !new_len) return SV_ERR_INVALID_ARG;
  if (!aligned(cache_len, 4) || !aligned(accepted_len, 4) || !aligned(path, 4) || !aligned(new_len, 4) ||
      !aligned(workspace, 16))
    return SV_ERR_MISALIGNED;
  const bool apart = new_len == cache_len || new_len == accepted_len;
  if ((new_len != cache_len && overlap(new_len, B, cache_len, B)) ||
      (new_len != accepted_len && overlap(new_len, B, accepted_len, B)) ||
      (path && overlap(new_len, B, path, static_cast<int64_t>(B) * N)))
    return SV_ERR_INVALID_ARG;
  CacheCommitParams p{};
  p.c = view(cache, page_table, table_stride, max_pages);
  p.cache_len = cache_len, p.accepted = accepted_len, p.path = path;
  p.B = B, p.N = N, p.new_len = new_len, p.apart = apart;
  if (const int e = ctrl_of(workspace, &p.ctrl)) return e;
  const int es = bytes_of(cache->dtype);
  const bool vec = cache->head_dim * es % 16 == 0 && pool_on(cache, es, 16);
  const int n = sms();
  if (n <= 0) return SV_ERR_CUDA;
  return launch_cache_commit(p, es, vec, n, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

extern "C" size_t spec_verify_tree_attention_scratch_size(int B, int N, int Hq, int num_heads, int head_dim) {
  if (B < 0 || B > 65535 || N < 1 || N > 64 || num_heads < 1 || Hq < 1 || Hq > 1024 || Hq % num_heads ||
      head_dim < 1 || head_dim > 256)
    return 0;
  const size_t n = head_dim <= 128 ? attention_scratch_bytes(N, Hq / num_heads, head_dim) : 256;
  return (n + 255) / 256 * 256;
}

extern "C" int spec_verify_tree_attention(const sv_rows* q, int q_dtype, const sv_kv_cache* cache,
                                          const int32_t* page_table, int64_t table_stride, int max_pages,
                                          const int32_t* cache_len, const int32_t* parent, const int32_t* count,
                                          int B, int N, int Hq, float scale, void* out, float* lse,
                                          void* workspace, void* scratch, size_t scratch_bytes, void* stream) {
  if (B < 0 || N < 1 || N > 64 || !type_ok(q_dtype, false, false) || !std::isfinite(scale)) return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (const int e = check_cache(cache, page_table, table_stride, max_pages, B, false)) return e;
  if (cache->dtype != q_dtype && cache->dtype != SV_E4M3) return SV_ERR_INVALID_ARG;
  if (!q || !q->data || !strides_ok(q) || !cache_len || !out || !scratch || Hq < 1 || Hq > 1024 ||
      Hq % cache->num_heads || static_cast<long long>(B) * N * Hq > 0x7fffffffll)
    return SV_ERR_INVALID_ARG;
  if (!aligned(q->data, 2) || !aligned(out, 2) || !aligned(lse, 4) || !aligned(cache_len, 4) ||
      !aligned(parent, 4) || !aligned(count, 4) || !aligned(workspace, 16) || !aligned(scratch, 16))
    return SV_ERR_MISALIGNED;
  if (scratch_bytes < spec_verify_tree_attention_scratch_size(B, N, Hq, cache->num_heads, cache->head_dim))
    return SV_ERR_WORKSPACE;
  AttnParams p{};
  p.q = rows_view(q);
  p.c = view(cache, page_table, table_stride, max_pages);
  p.cache_len = cache_len, p.parent = parent, p.count = count;
  p.B = B, p.N = N, p.Hq = Hq, p.G = Hq / cache->num_heads;
  p.c2 = static_cast<float>(1.4426950408889634 * scale);
  p.out = out, p.lse = lse, p.scratch = scratch;
  if (const int e = ctrl_of(workspace, &p.ctrl)) return e;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int n = sms();
  if (n <= 0) return SV_ERR_CUDA;
  cudaError_t e = cudaErrorNotSupported;
  if (attention_mma_takes(p, cache->dtype)) e = launch_attention_mma(p, q_dtype, cache->dtype, n, st);
  if (e == cudaErrorNotSupported) e = launch_attention_plain(p, q_dtype, cache->dtype, st);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
