// Host side of the paged cache: handle, argument checks, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <new>

#include "../../include/longstraw.h"
#include "ls_host.h"
#include "ls_internal.h"
#include "ls_ops.h"
#include "ls_rope_host.h"

struct ls_cache_s {
  uint32_t magic;
  int device;
  int page_size, layout;
  float scale;
  ls::CacheView view;
  CUtensorMap tm_k, tm_v;   // boxes of one head and min(page_size, 128) tokens of one page
};

namespace {

using namespace ls;

constexpr uint32_t kMagic = 0x4c534341u;  // "LSCA"

ls_status check_cache(ls_cache_t h) {
  return h == nullptr || h->magic != kMagic ? LS_ERR_NOT_PREPARED : LS_OK;
}

// The current device is the handle's and the stream belongs to it.
ls_status enter_cache(ls_cache_t h, void* stream, uint32_t** status) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return static_cast<ls_status>(launch_failed(e, "cudaGetDevice"));
  if (dev != h->device) return LS_ERR_WRONG_DEVICE;
  return static_cast<ls_status>(enter_call(stream, status));
}

template <class F>
ls_status run_launch(int kernel, void* stream, const char* what, F launch) {
  cudaError_t e;
  {
    LaunchTimer t(kernel, static_cast<cudaStream_t>(stream));
    e = injected_failure() ? cudaErrorLaunchFailure : launch(static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? LS_OK : static_cast<ls_status>(launch_failed(e, what));
}

ls_status check_pages_ws(ls_cache_t h, const void* ws, size_t bytes) {
  if (ws == nullptr || bytes < ls_cache_pages_workspace_bytes(h)) return LS_ERR_WORKSPACE;
  return aligned16(ws) ? LS_OK : LS_ERR_MISALIGNED;
}

}  // namespace

extern "C" {

ls_status ls_cache_create(const ls_cache_desc* d, ls_cache_t* out) {
  NvtxRange nvtx_range("ls_cache_create");
  if (d == nullptr || out == nullptr) return LS_ERR_INVALID_ARGUMENT;
  if (d->k_pages == nullptr || d->v_pages == nullptr || d->page_table == nullptr ||
      d->seq_len == nullptr || d->refcount == nullptr)
    return LS_ERR_INVALID_ARGUMENT;
  if (d->num_pages < 1 || d->num_rows < 1 || d->table_width < 1 || d->Hq < 1 || d->Hkv < 1)
    return LS_ERR_INVALID_ARGUMENT;
  if (!(d->softmax_scale >= 0.0f) || !std::isfinite(d->softmax_scale))
    return LS_ERR_INVALID_ARGUMENT;
  if (d->layout != LS_CACHE_NHD && d->layout != LS_CACHE_HND) return LS_ERR_INVALID_ARGUMENT;
  if (d->D != 64 && d->D != 128) return LS_ERR_UNSUPPORTED;
  if (d->Hq % d->Hkv != 0 || d->Hq / d->Hkv > 16 || d->Hq > 65536) return LS_ERR_UNSUPPORTED;
  int log2 = 0;
  while ((1 << log2) < d->page_size && log2 < 9) ++log2;
  if ((1 << log2) != d->page_size || log2 < 4 || log2 > 8) return LS_ERR_UNSUPPORTED;
  if (d->num_pages >= (int64_t(1) << 31)) return LS_ERR_UNSUPPORTED;
  // a row's tokens are counted in int32
  if (static_cast<int64_t>(d->table_width) * d->page_size >= (int64_t(1) << 31))
    return LS_ERR_UNSUPPORTED;
  const int64_t page = static_cast<int64_t>(d->page_size) * d->Hkv * d->D;
  if (d->page_stride < page) return LS_ERR_INVALID_ARGUMENT;
  if (d->page_stride % 8 != 0) return LS_ERR_MISALIGNED;
  if (d->page_stride >= (int64_t(1) << 38)) return LS_ERR_UNSUPPORTED;
  if (!aligned16(d->k_pages) || !aligned16(d->v_pages) || !aligned_n(d->page_table, 4) ||
      !aligned_n(d->seq_len, 4) || !aligned_n(d->refcount, 4))
    return LS_ERR_MISALIGNED;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return static_cast<ls_status>(launch_failed(e, "cudaGetDevice"));
  ls_cache_s* h = new (std::nothrow) ls_cache_s();
  if (h == nullptr) return LS_ERR_INVALID_ARGUMENT;
  h->device = dev;
  h->page_size = d->page_size;
  h->layout = d->layout;
  h->scale = d->softmax_scale > 0.0f ? d->softmax_scale : 1.0f / std::sqrt(static_cast<float>(d->D));
  CacheView& v = h->view;
  v.k = static_cast<uint16_t*>(d->k_pages);
  v.v = static_cast<uint16_t*>(d->v_pages);
  v.page_stride = d->page_stride;
  v.tok_stride = d->layout == LS_CACHE_NHD ? static_cast<int64_t>(d->Hkv) * d->D : d->D;
  v.head_stride = d->layout == LS_CACHE_NHD ? d->D : static_cast<int64_t>(d->page_size) * d->D;
  v.num_pages = d->num_pages;
  v.ps_log2 = log2;
  v.Hq = d->Hq;
  v.Hkv = d->Hkv;
  v.D = d->D;
  v.num_rows = d->num_rows;
  v.width = d->table_width;
  v.table = d->page_table;
  v.len = d->seq_len;
  v.ref = d->refcount;
  const cuuint64_t D = d->D, H = d->Hkv, ps = d->page_size, N = static_cast<cuuint64_t>(d->num_pages);
  const cuuint32_t bt = d->page_size < 128 ? d->page_size : 128;
  const bool nhd = d->layout == LS_CACHE_NHD;
  const cuuint64_t dims[4] = {D, nhd ? H : ps, nhd ? ps : H, N};
  const cuuint64_t strides[3] = {D * 2, (nhd ? H : ps) * D * 2, static_cast<cuuint64_t>(d->page_stride) * 2};
  const cuuint32_t box[4] = {64, nhd ? 1 : bt, nhd ? bt : 1, 1};
  int st = encode_bf16_map(&h->tm_k, d->k_pages, 4, dims, strides, box);
  if (st == LS_OK) st = encode_bf16_map(&h->tm_v, d->v_pages, 4, dims, strides, box);
  if (st != LS_OK) {
    delete h;
    return static_cast<ls_status>(st);
  }
  h->magic = kMagic;
  *out = h;
  return LS_OK;
}

ls_status ls_cache_destroy(ls_cache_t h) {
  if (h == nullptr) return LS_OK;
  if (h->magic != kMagic) return LS_ERR_NOT_PREPARED;
  h->magic = 0;
  delete h;
  return LS_OK;
}

ls_status ls_cache_reset(ls_cache_t h, void* stream) {
  NvtxRange nvtx_range("ls_cache_reset");
  ls_status st = check_cache(h);
  if (st != LS_OK) return st;
  uint32_t* status = nullptr;
  st = enter_cache(h, stream, &status);
  if (st != LS_OK) return st;
  return run_launch(LS_KERNEL_CACHE_PAGES, stream, "cache reset launch",
                    [&](cudaStream_t s) { return launch_cache_reset(h->view, s); });
}

size_t ls_cache_pages_workspace_bytes(ls_cache_t h) {
  if (check_cache(h) != LS_OK) return 0;
  return align_up(cache_pages_ws_bytes(h->view.num_pages), 256);
}

ls_status ls_cache_extend(ls_cache_t h, int32_t n, const int32_t* rows, const int32_t* add,
                          void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("ls_cache_extend");
  ls_status st = check_cache(h);
  if (st != LS_OK) return st;
  if (n < 0 || (n > 0 && (rows == nullptr || add == nullptr))) return LS_ERR_INVALID_ARGUMENT;
  if (n > kMaxList) return LS_ERR_UNSUPPORTED;
  if (!aligned_n(rows, 4) || !aligned_n(add, 4)) return LS_ERR_MISALIGNED;
  st = check_pages_ws(h, workspace, workspace_bytes);
  if (st != LS_OK) return st;
  uint32_t* status = nullptr;
  st = enter_cache(h, stream, &status);
  if (st != LS_OK || n == 0) return st;
  return run_launch(LS_KERNEL_CACHE_PAGES, stream, "cache extend launch", [&](cudaStream_t s) {
    return launch_cache_extend(h->view, n, rows, add, workspace, status, s);
  });
}

ls_status ls_cache_fork(ls_cache_t h, int32_t n, const int32_t* parents, const int32_t* children,
                        void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("ls_cache_fork");
  ls_status st = check_cache(h);
  if (st != LS_OK) return st;
  if (n < 0 || (n > 0 && (parents == nullptr || children == nullptr))) return LS_ERR_INVALID_ARGUMENT;
  if (n > kMaxList) return LS_ERR_UNSUPPORTED;
  if (!aligned_n(parents, 4) || !aligned_n(children, 4)) return LS_ERR_MISALIGNED;
  st = check_pages_ws(h, workspace, workspace_bytes);
  if (st != LS_OK) return st;
  uint32_t* status = nullptr;
  st = enter_cache(h, stream, &status);
  if (st != LS_OK || n == 0) return st;
  return run_launch(LS_KERNEL_CACHE_PAGES, stream, "cache fork launch", [&](cudaStream_t s) {
    return launch_cache_fork(h->view, n, parents, children, workspace, status, s);
  });
}

ls_status ls_cache_free(ls_cache_t h, int32_t n, const int32_t* rows, void* stream) {
  NvtxRange nvtx_range("ls_cache_free");
  ls_status st = check_cache(h);
  if (st != LS_OK) return st;
  if (n < 0 || (n > 0 && rows == nullptr)) return LS_ERR_INVALID_ARGUMENT;
  if (n > kMaxList) return LS_ERR_UNSUPPORTED;
  if (!aligned_n(rows, 4)) return LS_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  st = enter_cache(h, stream, &status);
  if (st != LS_OK || n == 0) return st;
  return run_launch(LS_KERNEL_CACHE_PAGES, stream, "cache free launch", [&](cudaStream_t s) {
    return launch_cache_free(h->view, n, rows, status, s);
  });
}

ls_status ls_cache_compact(ls_cache_t src, ls_cache_t dst, int32_t* n_live, void* workspace,
                           size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("ls_cache_compact");
  ls_status st = check_cache(src);
  if (st == LS_OK) st = check_cache(dst);
  if (st != LS_OK) return st;
  const CacheView &a = src->view, &b = dst->view;
  if (src->device != dst->device) return LS_ERR_WRONG_DEVICE;
  if (src != dst) {
    if (a.ps_log2 != b.ps_log2 || a.Hkv != b.Hkv || a.D != b.D || src->layout != dst->layout ||
        a.num_rows != b.num_rows || a.width != b.width)
      return LS_ERR_UNSUPPORTED;
    // another pool means other arrays
    if (a.k == b.k || a.v == b.v || a.table == b.table || a.len == b.len || a.ref == b.ref)
      return LS_ERR_INVALID_ARGUMENT;
  }
  if (!aligned_n(n_live, 4)) return LS_ERR_MISALIGNED;
  st = check_pages_ws(src, workspace, workspace_bytes);
  if (st != LS_OK) return st;
  uint32_t* status = nullptr;
  st = enter_cache(src, stream, &status);
  if (st != LS_OK) return st;
  return run_launch(LS_KERNEL_CACHE_PAGES, stream, "cache compact launch", [&](cudaStream_t s) {
    return launch_cache_compact(a, b, src == dst, n_live, workspace, status, s);
  });
}

ls_status ls_cache_append(ls_cache_t h, const ls_cache_append_desc* d, void* stream) {
  NvtxRange nvtx_range("ls_cache_append");
  ls_status st = check_cache(h);
  if (st != LS_OK) return st;
  if (d == nullptr || d->cu_new == nullptr || d->k_new == nullptr || d->v_new == nullptr)
    return LS_ERR_INVALID_ARGUMENT;
  if (d->S < 1 || d->T < 1) return LS_ERR_INVALID_ARGUMENT;
  if (d->S > kMaxSeqs || d->T >= (int64_t(1) << 31)) return LS_ERR_UNSUPPORTED;
  const CacheView& c = h->view;
  const int64_t nk = static_cast<int64_t>(c.Hkv) * c.D, nq = static_cast<int64_t>(c.Hq) * c.D;
  if (d->k_stride < nk || d->v_stride < nk) return LS_ERR_INVALID_ARGUMENT;
  RopeArgs a{};
  if (d->inv_freq != nullptr) {
    if (d->rot_dim < 2 || d->rot_dim > c.D || d->rot_dim % 2 != 0) return LS_ERR_INVALID_ARGUMENT;
    if (!rope_turns(d->inv_freq, d->rot_dim, d->attn_factor, &a)) return LS_ERR_INVALID_ARGUMENT;
  } else if (d->q != nullptr) {
    return LS_ERR_INVALID_ARGUMENT;
  }
  if (d->q != nullptr) {
    if (d->q_out == nullptr || d->q_stride < nq || d->q_out_stride < nq) return LS_ERR_INVALID_ARGUMENT;
    if (d->q == d->q_out && d->q_stride != d->q_out_stride) return LS_ERR_INVALID_ARGUMENT;
    if (!aligned_n(d->q, 2) || !aligned_n(d->q_out, 2)) return LS_ERR_MISALIGNED;
  }
  if (!aligned_n(d->k_new, 2) || !aligned_n(d->v_new, 2) || !aligned_n(d->rows, 4) ||
      !aligned_n(d->cu_new, 4))
    return LS_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  st = enter_cache(h, stream, &status);
  if (st != LS_OK) return st;
  a.T = d->T;
  a.Hq = d->q != nullptr ? c.Hq : 0;
  a.Hk = c.Hkv;
  a.D = c.D;
  a.interleaved = d->interleaved != 0;
  a.q = static_cast<const uint16_t*>(d->q);
  a.qs = d->q_stride;
  a.qo = static_cast<uint16_t*>(d->q_out);
  a.qos = d->q_out_stride;
  a.k = static_cast<const uint16_t*>(d->k_new);
  a.ks = d->k_stride;
  a.append = 1;
  a.v = static_cast<const uint16_t*>(d->v_new);
  a.vs = d->v_stride;
  a.S = d->S;
  a.rows = d->rows;
  a.cu = d->cu_new;
  a.c = c;
  a.status = status;
  return run_launch(LS_KERNEL_CACHE_APPEND, stream, "cache append launch",
                    [&](cudaStream_t s) { return launch_rope(a, s); });
}

size_t ls_cache_attn_workspace_bytes(ls_cache_t h, int32_t S, int64_t T, int32_t max_new,
                                     int64_t max_len) {
  if (check_cache(h) != LS_OK || S < 1 || T < 1 || max_new < 1 || max_len < 1) return 0;
  return cache_attn_layout(h->view, S, T).total;
}

ls_status ls_cache_attn(ls_cache_t h, const ls_cache_attn_desc* d, void* workspace,
                        size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("ls_cache_attn");
  ls_status st = check_cache(h);
  if (st != LS_OK) return st;
  if (d == nullptr || d->cu_new == nullptr || d->q == nullptr || d->o == nullptr || d->lse == nullptr)
    return LS_ERR_INVALID_ARGUMENT;
  if (d->S < 1 || d->T < 1 || d->max_new < 1 || d->max_len < 1 || d->group < 1)
    return LS_ERR_INVALID_ARGUMENT;
  if (d->S % d->group != 0 || (d->group > 1 && d->shared_len == nullptr))
    return LS_ERR_INVALID_ARGUMENT;
  const CacheView& c = h->view;
  if (d->S > kMaxSeqs || d->T >= (int64_t(1) << 31) || d->max_len >= (int64_t(1) << 31))
    return LS_ERR_UNSUPPORTED;
  if (d->q_stride < static_cast<int64_t>(c.Hq) * c.D) return LS_ERR_INVALID_ARGUMENT;
  if (d->q_stride >= (int64_t(1) << 38)) return LS_ERR_UNSUPPORTED;
  const size_t need = ls_cache_attn_workspace_bytes(h, d->S, d->T, d->max_new, d->max_len);
  if (workspace == nullptr || workspace_bytes < need) return LS_ERR_WORKSPACE;
  if (!aligned16(d->q) || !aligned16(d->o) || d->q_stride % 8 != 0 || !aligned16(workspace) ||
      !aligned_n(d->lse, 4) || !aligned_n(d->rows, 4) || !aligned_n(d->cu_new, 4) ||
      !aligned_n(d->shared_len, 4))
    return LS_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  st = enter_cache(h, stream, &status);
  if (st != LS_OK) return st;
  CacheAttnArgs a{};
  a.c = c;
  a.scale = h->scale;
  a.S = d->S;
  a.T = d->T;
  a.rows = d->rows;
  a.cu = d->cu_new;
  a.max_new = d->max_new;
  a.max_len = d->max_len;
  a.q = static_cast<const uint16_t*>(d->q);
  a.qs = d->q_stride;
  a.o = static_cast<uint16_t*>(d->o);
  a.lse = d->lse;
  a.group = d->group;
  a.shared = d->group > 1 ? d->shared_len : nullptr;
  a.ws = workspace;
  a.tm_k = &h->tm_k;
  a.tm_v = &h->tm_v;
  a.layout = h->layout;
  a.status = status;
  const cuuint32_t g = c.Hq / c.Hkv;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.Hq),
                              static_cast<cuuint64_t>(d->T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.D) * 2, static_cast<cuuint64_t>(d->q_stride) * 2};
  const cuuint32_t box[3] = {64, g, 128 / g}, boxn[3] = {64, g, 64 / g};
  a.wide = cache_attn_wide(c, d->T, d->max_new, d->group);
  if (a.wide) st = static_cast<ls_status>(encode_bf16_map(&a.tm_q, d->q, 3, dims, strides, box));
  if (st == LS_OK) st = static_cast<ls_status>(encode_bf16_map(&a.tm_qn, d->q, 3, dims, strides, boxn));
  if (st != LS_OK) return st;
  return run_launch(LS_KERNEL_CACHE_ATTN, stream, "cache attention launch",
                    [&](cudaStream_t s) { return launch_cache_attn(a, s); });
}

}  // extern "C"
