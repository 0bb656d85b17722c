// Page management of the cache: extend, fork, free, compact, reset.
//
// Free pages are those with count 0.  Allocation takes the lowest ones in list order, so the
// result is a function of the arrays alone: a scan of the counts writes the free (or live)
// pages' indices in ascending order, one block decides on every entry of the list (sizes,
// ranks among the free pages, refusals), and the entries' table rows, counts and page copies
// run on the whole grid.  Counts change by integer atomics, whose order cannot change them.
#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"

namespace ls {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kCopyThreads = 256;

// Workspace: a header, the list's plan, one int32 a page.
struct Plan {
  int32_t n_free;                     // free pages found (or live pages, compact)
  int32_t pad[63];
  int32_t row[kMaxList];              // table row the entry writes; -1: left out
  int32_t from[kMaxList];             // fork: parent row
  int32_t first[kMaxList];            // extend: first new table column; fork: whole pages
  int32_t count[kMaxList];            // extend: new pages; fork: tokens of the part-filled page
  int32_t rank[kMaxList];             // the entry's first free page
};
__host__ __device__ inline int32_t* page_list(void* ws) {
  return reinterpret_cast<int32_t*>(static_cast<char*>(ws) + sizeof(Plan));
}

// Exclusive sum over the block of one int a thread; *total for all.
__device__ __forceinline__ int block_scan(int v, int* sh /* [33] */, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, off);
    if (lane >= off) s += u;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = lane < static_cast<int>(blockDim.x >> 5) ? sh[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += u;
    }
    sh[lane] = w;
  }
  __syncthreads();
  *total = sh[(blockDim.x >> 5) - 1];
  return (warp > 0 ? sh[warp - 1] : 0) + s - v;
}

// list[] = the pages whose count is 0 (want_free) in ascending order, *n their number.
__global__ void __launch_bounds__(kScanThreads) free_list_kernel(const int32_t* ref, int64_t pages,
                                                                int32_t* list, int32_t* n) {
  __shared__ int sh[33];
  int base = 0;
  for (int64_t p0 = 0; p0 < pages; p0 += kScanThreads) {
    const int64_t p = p0 + threadIdx.x;
    const int is = (p < pages && ref[p] == 0) ? 1 : 0;
    int total;
    const int at = base + block_scan(is, sh, &total);
    if (is) list[at] = static_cast<int32_t>(p);
    base += total;
  }
  if (threadIdx.x == 0) *n = base;
}

__device__ __forceinline__ bool listed_before(const int32_t* list, int i) {
  for (int j = 0; j < i; ++j)
    if (list[j] == list[i]) return true;
  return false;
}

__device__ __forceinline__ bool good_len(const CacheView& c, int64_t len) {
  return len >= 0 && len <= (static_cast<int64_t>(c.width) << c.ps_log2);
}

__global__ void __launch_bounds__(kMaxList) extend_plan_kernel(CacheView c, int n,
                                                              const int32_t* rows,
                                                              const int32_t* add, Plan* plan,
                                                              uint32_t* status) {
  __shared__ int sh[33];
  const int i = threadIdx.x;
  bool ok = false;
  int row = -1, need = 0, first = 0;
  int64_t len = 0, grown = 0;
  if (i < n) {
    row = rows[i];
    if (row >= 0 && row < c.num_rows && add[i] >= 0 && !listed_before(rows, i)) {
      len = c.len[row];
      grown = len + add[i];
      if (good_len(c, len) && good_len(c, grown)) {
        ok = true;
        const int64_t ps1 = (1 << c.ps_log2) - 1;
        first = static_cast<int>((len + ps1) >> c.ps_log2);
        need = static_cast<int>((grown + ps1) >> c.ps_log2) - first;
      }
    }
    if (!ok) set_device_status(status, DEV_BAD_INDEX);
  }
  int total;
  const int rank = block_scan(ok ? need : 0, sh, &total);
  if (i >= n) return;
  if (ok && rank + need > plan->n_free) {
    set_device_status(status, DEV_NO_PAGES);
    ok = false;
  }
  plan->row[i] = ok ? row : -1;
  plan->first[i] = first;
  plan->count[i] = need;
  plan->rank[i] = rank;
  if (ok) c.len[row] = static_cast<int32_t>(grown);
}

__global__ void __launch_bounds__(kCopyThreads) extend_kernel(CacheView c, const Plan* plan,
                                                             const int32_t* list) {
  const int i = blockIdx.x;
  const int row = plan->row[i];
  if (row < 0) return;
  const int first = plan->first[i], count = plan->count[i], rank = plan->rank[i];
  for (int j = threadIdx.x; j < count; j += kCopyThreads) {
    const int page = list[rank + j];
    c.table[static_cast<int64_t>(row) * c.width + first + j] = page;
    c.ref[page] = 1;
  }
}

__global__ void __launch_bounds__(kMaxList) fork_plan_kernel(CacheView c, int n,
                                                            const int32_t* parents,
                                                            const int32_t* children, Plan* plan,
                                                            uint32_t* status) {
  __shared__ int sh[33];
  const int i = threadIdx.x;
  bool ok = false;
  int child = -1, parent = -1;
  int64_t len = 0;
  if (i < n) {
    child = children[i];
    parent = parents[i];
    ok = child >= 0 && child < c.num_rows && parent >= 0 && parent < c.num_rows &&
         !listed_before(children, i);
    if (ok) {
      len = c.len[parent];
      ok = c.len[child] == 0 && good_len(c, len) && child != parent;
    }
    if (!ok) set_device_status(status, DEV_BAD_INDEX);
  }
  const int full = static_cast<int>(len >> c.ps_log2);
  const int part = static_cast<int>(len & ((1 << c.ps_log2) - 1));
  int total;
  // every length above is read before the first one is written below
  const int rank = block_scan(ok && part > 0 ? 1 : 0, sh, &total);
  if (i >= n) return;
  if (ok && part > 0 && rank >= plan->n_free) {
    set_device_status(status, DEV_NO_PAGES);
    ok = false;
  }
  plan->row[i] = ok ? child : -1;
  plan->from[i] = parent;
  plan->first[i] = full;
  plan->count[i] = part;
  plan->rank[i] = rank;
  if (ok) c.len[child] = static_cast<int32_t>(len);
}

// The first `tokens` tokens of a page's keys and values, page src to page dst (16-byte units).
__device__ __forceinline__ void copy_page(const CacheView& sc, const CacheView& dc, int64_t src,
                                          int64_t dst, int tokens) {
  const int d8 = sc.D / 8;
  const int units = tokens * sc.Hkv * d8;
  const uint4* sk = reinterpret_cast<const uint4*>(sc.k + src * sc.page_stride);
  const uint4* sv = reinterpret_cast<const uint4*>(sc.v + src * sc.page_stride);
  uint4* dk = reinterpret_cast<uint4*>(dc.k + dst * dc.page_stride);
  uint4* dv = reinterpret_cast<uint4*>(dc.v + dst * dc.page_stride);
  const int per_head = tokens * d8;
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    int64_t at = u;
    if (sc.head_stride > sc.tok_stride) {     // [Hkv, page_size, D]: a run a head
      const int h = u / per_head;
      at = h * (sc.head_stride / 8) + (u - h * per_head);
    }
    dk[at] = sk[at];
    dv[at] = sv[at];
  }
}

__global__ void __launch_bounds__(kCopyThreads) fork_kernel(CacheView c, const Plan* plan,
                                                           const int32_t* list, uint32_t* status) {
  const int i = blockIdx.x;
  const int row = plan->row[i];
  if (row < 0) return;
  const int32_t* src = c.table + static_cast<int64_t>(plan->from[i]) * c.width;
  int32_t* dst = c.table + static_cast<int64_t>(row) * c.width;
  const int full = plan->first[i], part = plan->count[i];
  for (int j = threadIdx.x; j < full; j += kCopyThreads) {
    const int page = src[j];
    dst[j] = page;
    if (page >= 0 && page < c.num_pages)
      atomicAdd(c.ref + page, 1);
    else
      set_device_status(status, DEV_BAD_INDEX);
  }
  if (part > 0) {
    const int page = list[plan->rank[i]], from = src[full];
    if (threadIdx.x == 0) {
      dst[full] = page;
      c.ref[page] = 1;
    }
    if (from >= 0 && from < c.num_pages)
      copy_page(c, c, from, page, part);
    else if (threadIdx.x == 0)
      set_device_status(status, DEV_BAD_INDEX);
  }
}

__global__ void __launch_bounds__(kCopyThreads) free_kernel(CacheView c, int n, const int32_t* rows,
                                                           uint32_t* status) {
  const int i = blockIdx.x;
  const int row = rows[i];
  int dup = 0;
  for (int j = threadIdx.x; j < i; j += kCopyThreads) dup |= rows[j] == row;
  dup = __syncthreads_or(dup);
  if (row < 0 || row >= c.num_rows || dup) {
    if (threadIdx.x == 0) set_device_status(status, DEV_BAD_INDEX);
    return;
  }
  const int64_t len = c.len[row];
  if (!good_len(c, len)) {
    if (threadIdx.x == 0) set_device_status(status, DEV_BAD_INDEX);
    return;
  }
  int32_t* t = c.table + static_cast<int64_t>(row) * c.width;
  const int pages = static_cast<int>((len + (1 << c.ps_log2) - 1) >> c.ps_log2);
  for (int j = threadIdx.x; j < pages; j += kCopyThreads) {
    const int page = t[j];
    t[j] = -1;
    if (page >= 0 && page < c.num_pages)
      atomicSub(c.ref + page, 1);
    else
      set_device_status(status, DEV_BAD_INDEX);
  }
  __syncthreads();
  if (threadIdx.x == 0) c.len[row] = 0;
}

// to[p] = the page that p moves to (-1: not live); *n_live the number of live pages.
// Out of place: its rank among the live pages.  In place: p itself below n_live, else the hole
// of p's rank among the live pages from n_live on.
__global__ void __launch_bounds__(kScanThreads) compact_plan_kernel(const int32_t* ref, int64_t pages,
                                                                   int inplace, int32_t* to,
                                                                   int32_t* n_ws, int32_t* n_live) {
  __shared__ int sh[33];
  int base = 0;
  for (int64_t p0 = 0; p0 < pages; p0 += kScanThreads) {
    const int64_t p = p0 + threadIdx.x;
    const int is = (p < pages && ref[p] > 0) ? 1 : 0;
    int total;
    const int at = base + block_scan(is, sh, &total);
    if (p < pages) to[p] = is ? at : -1;
    base += total;
  }
  const int live = base;
  if (threadIdx.x == 0) {
    *n_ws = live;
    if (n_live != nullptr) *n_live = live;
  }
  if (!inplace) return;
  __syncthreads();
  // A live page q >= live of rank r is mover number r - (live pages below `live`).  The hole
  // of number m is the m-th page below `live` that is not live; walk both in order, holes
  // kept as to[hole] = -2 - m until the movers have looked them up.
  int holes = 0;
  for (int64_t p0 = 0; p0 < live; p0 += kScanThreads) {
    const int64_t p = p0 + threadIdx.x;
    const int is = (p < live && to[p] < 0) ? 1 : 0;
    int total;
    const int at = holes + block_scan(is, sh, &total);
    // hole number `at` is kept in the entry of free slot `at` behind the table
    if (is) to[pages + at] = static_cast<int32_t>(p);
    holes += total;
    if (p < live && !is) to[p] = static_cast<int32_t>(p);
  }
  __syncthreads();
  const int stay = live - holes;          // live pages below `live`
  for (int64_t p = live + threadIdx.x; p < pages; p += kScanThreads)
    if (to[p] >= 0) to[p] = to[pages + (to[p] - stay)];
}

// A block a source page (grid-stride): its keys and values and its count.
__global__ void __launch_bounds__(kCopyThreads) compact_copy_kernel(CacheView sc, CacheView dc,
                                                                   int inplace, const int32_t* to,
                                                                   const int32_t* n_ws,
                                                                   uint32_t* status) {
  const int n = *n_ws;
  for (int64_t p = blockIdx.x; p < sc.num_pages; p += gridDim.x) {
    const int d = to[p];
    if (d < 0 || (inplace && d == p)) continue;
    if (d >= dc.num_pages) {
      if (threadIdx.x == 0) set_device_status(status, DEV_NO_PAGES);
      continue;
    }
    copy_page(sc, dc, p, d, 1 << sc.ps_log2);
    if (threadIdx.x == 0) {
      dc.ref[d] = sc.ref[p];
      if (inplace) sc.ref[p] = 0;
    }
  }
  if (!inplace)
    for (int64_t p = n + blockIdx.x * static_cast<int64_t>(kCopyThreads) + threadIdx.x; p < dc.num_pages;
         p += static_cast<int64_t>(gridDim.x) * kCopyThreads)
      dc.ref[p] = 0;
}

__global__ void __launch_bounds__(kCopyThreads) compact_table_kernel(CacheView sc, CacheView dc,
                                                                    const int32_t* to,
                                                                    uint32_t* status) {
  const int64_t total = static_cast<int64_t>(sc.num_rows) * sc.width;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kCopyThreads;
  const int64_t i0 = blockIdx.x * static_cast<int64_t>(kCopyThreads) + threadIdx.x;
  for (int64_t i = i0; i < total; i += stride) {
    const int page = sc.table[i];
    int d = -1;
    if (page >= 0 && page < sc.num_pages) {
      d = to[page];
      if (d >= dc.num_pages) d = -1;
    } else if (page >= sc.num_pages) {
      set_device_status(status, DEV_BAD_INDEX);
    }
    dc.table[i] = d;
  }
  for (int64_t i = i0; i < sc.num_rows; i += stride) dc.len[i] = sc.len[i];
}

__global__ void __launch_bounds__(kCopyThreads) reset_kernel(CacheView c) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kCopyThreads;
  const int64_t i0 = blockIdx.x * static_cast<int64_t>(kCopyThreads) + threadIdx.x;
  for (int64_t i = i0; i < static_cast<int64_t>(c.num_rows) * c.width; i += stride) c.table[i] = -1;
  for (int64_t i = i0; i < c.num_rows; i += stride) c.len[i] = 0;
  for (int64_t i = i0; i < c.num_pages; i += stride) c.ref[i] = 0;
}

unsigned wide_grid(int64_t items) {
  int64_t g = static_cast<int64_t>(num_sms()) * 8;
  if (g > items) g = items;
  return static_cast<unsigned>(g < 1 ? 1 : g);
}

}  // namespace

// The page list doubles as the compaction's map (num_pages) and its holes (num_pages).
size_t cache_pages_ws_bytes(int64_t num_pages) {
  return sizeof(Plan) + static_cast<size_t>(num_pages) * 2 * sizeof(int32_t);
}

cudaError_t launch_cache_reset(const CacheView& c, cudaStream_t s) {
  const int64_t n = static_cast<int64_t>(c.num_rows) * c.width;
  reset_kernel<<<wide_grid(((n > c.num_pages ? n : c.num_pages) + kCopyThreads - 1) / kCopyThreads),
                 kCopyThreads, 0, s>>>(c);
  return cudaGetLastError();
}

cudaError_t launch_cache_extend(const CacheView& c, int n, const int32_t* rows, const int32_t* add,
                                void* ws, uint32_t* status, cudaStream_t s) {
  Plan* plan = static_cast<Plan*>(ws);
  free_list_kernel<<<1, kScanThreads, 0, s>>>(c.ref, c.num_pages, page_list(ws), &plan->n_free);
  extend_plan_kernel<<<1, kMaxList, 0, s>>>(c, n, rows, add, plan, status);
  extend_kernel<<<static_cast<unsigned>(n), kCopyThreads, 0, s>>>(c, plan, page_list(ws));
  return cudaGetLastError();
}

cudaError_t launch_cache_fork(const CacheView& c, int n, const int32_t* parents,
                              const int32_t* children, void* ws, uint32_t* status, cudaStream_t s) {
  Plan* plan = static_cast<Plan*>(ws);
  free_list_kernel<<<1, kScanThreads, 0, s>>>(c.ref, c.num_pages, page_list(ws), &plan->n_free);
  fork_plan_kernel<<<1, kMaxList, 0, s>>>(c, n, parents, children, plan, status);
  fork_kernel<<<static_cast<unsigned>(n), kCopyThreads, 0, s>>>(c, plan, page_list(ws), status);
  return cudaGetLastError();
}

cudaError_t launch_cache_free(const CacheView& c, int n, const int32_t* rows, uint32_t* status,
                              cudaStream_t s) {
  free_kernel<<<static_cast<unsigned>(n), kCopyThreads, 0, s>>>(c, n, rows, status);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CacheView& src, const CacheView& dst, bool inplace,
                                 int32_t* n_live, void* ws, uint32_t* status, cudaStream_t s) {
  Plan* plan = static_cast<Plan*>(ws);
  int32_t* to = page_list(ws);
  compact_plan_kernel<<<1, kScanThreads, 0, s>>>(src.ref, src.num_pages, inplace ? 1 : 0, to,
                                                 &plan->n_free, n_live);
  compact_copy_kernel<<<wide_grid(src.num_pages), kCopyThreads, 0, s>>>(src, dst, inplace ? 1 : 0, to,
                                                                        &plan->n_free, status);
  const int64_t n = static_cast<int64_t>(src.num_rows) * src.width;
  compact_table_kernel<<<wide_grid((n + kCopyThreads - 1) / kCopyThreads), kCopyThreads, 0, s>>>(
      src, dst, to, status);
  return cudaGetLastError();
}

}  // namespace ls
