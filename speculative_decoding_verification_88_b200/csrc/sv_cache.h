// sv_cache.h -- parameter blocks shared by the cache-side host layer
// (sv_cache_api.cu) and its kernels (sv_cache.cu, sv_attention.cu).  Not part
// of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "sv_internal.h"

namespace sv {

// A pool and its page table as the kernels see them (strides in elements).
struct CacheView {
  void* k;
  void* v;
  float* ks;  // e4m3: [page][head][place]
  float* vs;
  int num_pages, page_size, heads, dim;
  long long page_stride, token_stride, head_stride;
  int layers;
  long long layer_stride, scale_layer_stride;
  const int* table;
  long long table_stride;
  int max_pages;
  UDiv div_page;  // / page_size
};

struct RowsView {
  const void* p;
  long long sb, sn, sh;
};

// Rotary turn of q rows and, with cache heads, the cache write of k and v rows.
struct RotateParams {
  RowsView q;  // Hq heads; sb unused when N covers all tokens
  int Hq;
  void* q_out;
  long long qo_st, qo_sh;  // by token b*N + j, by head
  RowsView k, v;           // cache.heads heads (absent when write == 0)
  int write;
  const int* positions;  // [T], or nullptr: cache_len + depth
  const int* cache_len;
  const int* parent;
  const int* count;
  long long tokens;  // B * N
  int N, D;
  const double* inv_freq;  // nullptr: K is not turned
  int rd, interleaved;
  float magnitude;
  int inverse;
  CacheView c;
  Ctrl* ctrl;  // nullable
};

struct CacheReadParams {
  CacheView c;
  const int* offsets;
  const int* start;  // nullable
  int B;
  long long total;
  void* k_out;
  void* v_out;
  Ctrl* ctrl;
};

struct CacheCommitParams {
  CacheView c;
  const int* cache_len;
  const int* accepted;
  const int* path;  // nullable
  int B, N;
  int* new_len;
  bool apart;  // new_len is cache_len or accepted
  Ctrl* ctrl;
};

struct AttnParams {
  RowsView q;
  CacheView c;
  const int* cache_len;
  const int* parent;
  const int* count;
  int B, N, Hq, G;  // G = Hq / cache heads
  float c2;         // log2(e) * scale
  void* out;
  float* lse;
  Ctrl* ctrl;
  void* scratch;
};

// es / cache codes follow sv_dtype.  `vec`: vectors may be used: of 16 bytes,
// or of 8 codes of an 8-bit pool, whose rows need only lie on 8-byte boundaries
// (`on16`: they lie on 16-byte ones).
cudaError_t launch_rotate(const RotateParams& p, int dtype, int cache_dtype, bool vec, int sms,
                          cudaStream_t st);
cudaError_t launch_cache_read(const CacheReadParams& p, int cache_dtype, int out_dtype, bool vec,
                              bool on16, int sms, cudaStream_t st);
cudaError_t launch_cache_commit(const CacheCommitParams& p, int elem_bytes, bool vec, int sms,
                                cudaStream_t st);
cudaError_t launch_attention_plain(const AttnParams& p, int q_dtype, int cache_dtype,
                                   cudaStream_t st);
// The tensor-core form: whether it takes this layout, its scratch, its launch.
bool attention_mma_takes(const AttnParams& p, int cache_dtype);
size_t attention_scratch_bytes(int N, int G, int dim);
cudaError_t launch_attention_mma(const AttnParams& p, int q_dtype, int cache_dtype, int sms,
                                 cudaStream_t st);

}  // namespace sv
