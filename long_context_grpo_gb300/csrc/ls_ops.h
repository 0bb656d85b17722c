// Internal launch interface of the policy loss, the rotary positions and the paged cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace ls {

// ----- policy loss (k_policy.cu)
struct PolicyArgs {
  int64_t T, V, ldx, ldd;
  const uint16_t* logits;     // bf16, row t at logits + t * ldx
  const int32_t* ids;
  const float* old;
  const float* ref;           // nullptr: no KL term
  const float* adv;
  const float* weight;
  double clip_lo, clip_hi;    // 1 - eps_low, 1 + eps_high
  float log_lo[2], log_hi[2]; // their logarithms, each as a sum of two
  double beta;
  int kl;                     // ls_kl_kind
  float* loss;
  uint16_t* dlogits;          // row t at dlogits + t * ldd; may be the logits
  uint8_t* clip_mask;
  float* logp_out;            // or nullptr
  float* kl_out;              // or nullptr
  float2* logp_pair;          // workspace [T]: log-probabilities as sums of two
  double* partial;            // workspace [kMaxPartials]
  unsigned* counter;          // workspace
  uint32_t* status;
  uint64_t wait_ns;           // limit of a bounded wait
};
constexpr int kMaxPartials = 512;
cudaError_t launch_policy_loss(const PolicyArgs& a, cudaStream_t s);

// ----- paged cache
struct CacheView {
  uint16_t* k;
  uint16_t* v;
  int64_t page_stride, tok_stride, head_stride;   // elements
  int64_t num_pages;
  int ps_log2, Hq, Hkv, D;
  int num_rows, width;
  int32_t* table;             // [num_rows][width]
  int32_t* len;               // [num_rows]
  int32_t* ref;               // [num_pages]
};

// ----- rotary positions and the append (k_rope.cu)
constexpr int kMaxRot = 128;  // pairs
struct RopeArgs {
  int64_t T;
  int Hq, Hk, D, rot;         // rot = 0: no rotation (append only)
  int interleaved, inverse;
  float factor;
  const int64_t* positions;   // or nullptr: pos0 + t
  int64_t pos0;
  const uint16_t* q;
  int64_t qs;
  uint16_t* qo;
  int64_t qos;
  const uint16_t* k;
  int64_t ks;
  uint16_t* ko;
  int64_t kos;
  // append: keys go to the cache's pages, and the values v with them
  int append;
  const uint16_t* v;
  int64_t vs;
  int S;
  const int32_t* rows;
  const int32_t* cu;
  CacheView c;
  uint32_t* status;
  uint64_t turns[kMaxRot];    // inv_freq / 2 pi modulo 1 in units of 2^-64
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);

// ----- page management (k_pages.cu); ws as cache_pages_ws_bytes() lays it out
size_t cache_pages_ws_bytes(int64_t num_pages);
constexpr int kMaxList = 1024;
cudaError_t launch_cache_reset(const CacheView& c, cudaStream_t s);
cudaError_t launch_cache_extend(const CacheView& c, int n, const int32_t* rows, const int32_t* add,
                                void* ws, uint32_t* status, cudaStream_t s);
cudaError_t launch_cache_fork(const CacheView& c, int n, const int32_t* parents,
                              const int32_t* children, void* ws, uint32_t* status, cudaStream_t s);
cudaError_t launch_cache_free(const CacheView& c, int n, const int32_t* rows, uint32_t* status,
                              cudaStream_t s);
cudaError_t launch_cache_compact(const CacheView& src, const CacheView& dst, bool inplace,
                                 int32_t* n_live, void* ws, uint32_t* status, cudaStream_t s);

// ----- attention over pages (k_cache_attn.cu)
constexpr int kMaxSeqs = 2048;
struct CacheAttnArgs {
  CacheView c;
  float scale;
  int S;
  int64_t T;
  const int32_t* rows;
  const int32_t* cu;
  int max_new;
  int64_t max_len;
  const uint16_t* q;
  int64_t qs;
  uint16_t* o;
  float* lse;
  int group;
  const int32_t* shared;
  void* ws;
  const CUtensorMap* tm_k;    // pages: see ls_cache.cu
  const CUtensorMap* tm_v;
  int layout;                 // 0: [page_size, Hkv, D] inside a page, 1: [Hkv, page_size, D]
  bool wide;                  // cache_attn_wide of the bounds
  CUtensorMap tm_q;           // {64, g, 128 / g} boxes of [T][Hq][D]; with wide only
  CUtensorMap tm_qn;          // {64, g, 64 / g} boxes
  uint32_t* status;
};
// Workspace of a call: sizes come from the host's bounds alone.
struct CacheAttnLayout {
  size_t info, segs, lims, narrow, wide, lse, o, total;   // byte offsets, bytes
  int64_t max_narrow, max_wide;                           // job list capacities
  int64_t rows_narrow, rows_wide;                         // rows of partial results
};
CacheAttnLayout cache_attn_layout(const CacheView& c, int S, int64_t T);
bool cache_attn_wide(const CacheView& c, int64_t T, int max_new, int group);
cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t s);

}  // namespace ls
