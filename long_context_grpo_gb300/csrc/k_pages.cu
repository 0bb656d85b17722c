// Page management of the cache: extend, fork, free, compact, reset.
//
// Free pages are those with count 0.  Allocation takes the lowest ones in list order, so the
// result is a function of the arrays alone: one block decides on every entry of the list (sizes,
// ranks among the free pages, refusals) and scans the counts for as many free pages as that
// takes; then the entries' table rows, counts and page copies run on the whole grid.  Counts
// change by integer atomics, whose order cannot change them.
//
// Few rows: bound by launches and by rounds of dependent loads (0.6 us each; 128 rows freed and
// forked from 8 of 33,000 tokens: 12.3-14.4 us for 18 MB).  Compaction: bound by HBM (4.2 GB moved
// between pools in 646 us, 6.5 TB/s).
#include <climits>

#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"

namespace ls {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kCopyThreads = 256;

// Workspace: a header, the list's plan, one int32 a page.
struct Plan {
  int32_t n_moves;                    // compact
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

// Exclusive sum over the block of one number a thread; *total for all.
template <class N>
__device__ __forceinline__ N block_scan(N v, N* sh /* [33] */, N* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  N s = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const N u = __shfl_up_sync(0xffffffffu, s, off);
    if (lane >= off) s += u;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = s;
  __syncthreads();
  if (warp == 0) {
    N w = lane < static_cast<int>(blockDim.x >> 5) ? sh[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const N u = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += u;
    }
    sh[lane] = w;
  }
  __syncthreads();
  *total = sh[(blockDim.x >> 5) - 1];
  return (warp > 0 ? sh[warp - 1] : 0) + s - v;
}

constexpr int kScanPer = 8;          // pages of a thread in one step of a scan

// The counts of a thread's pages in one step of a scan.
struct Counts {
  int r[kScanPer];
};
__device__ __forceinline__ Counts load_counts(const int32_t* ref, int64_t pages, int64_t p0) {
  const int64_t p = p0 + threadIdx.x * kScanPer;
  Counts c;
#pragma unroll
  for (int k = 0; k < kScanPer; ++k) c.r[k] = p + k < pages ? __ldcg(ref + p + k) : 1;
  return c;
}

// list[] = the lowest pages whose count is 0, in ascending order, at least `want` of them if there
// are as many (the scan stops there); returns how many are listed.  Whole block; c: the first
// step's counts (loaded while the list is read).
__device__ int scan_free(Counts c, const int32_t* ref, int64_t pages, int want, int32_t* list, int* sh) {
  int base = 0;
  for (int64_t p0 = 0; p0 < pages && base < want; p0 += kScanThreads * kScanPer) {
    if (p0 > 0) c = load_counts(ref, pages, p0);
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < kScanPer; ++k) bits |= c.r[k] == 0 ? 1u << k : 0u;
    int total;
    int at = base + block_scan(__popc(bits), sh, &total);
#pragma unroll
    for (int k = 0; k < kScanPer; ++k)
      if (bits & (1u << k)) list[at++] = static_cast<int32_t>(p0 + threadIdx.x * kScanPer + k);
    base += total;
  }
  __syncthreads();
  return base;
}

// The first position of every row of a list: a hash table of twice as many slots as entries, so
// that an entry costs a few probes instead of a comparison with every earlier one.  (This, the first
// counts loaded ahead and the entries' plan read at once save 4 us of a fork of 128 rows.)
// clear, sync, put, sync, first.
struct FirstAt {
  int32_t key[2 * kMaxList], at[2 * kMaxList];
  __device__ __forceinline__ void clear() {
    for (int i = threadIdx.x; i < 2 * kMaxList; i += blockDim.x) {
      key[i] = -1;
      at[i] = kMaxList;
    }
  }
  static __device__ __forceinline__ uint32_t slot_of(int32_t row) {
    return (static_cast<uint32_t>(row) * 2654435761u >> 16) % (2 * kMaxList);
  }
  // (rows are not negative)
  __device__ __forceinline__ void put(int32_t row, int i) {
    uint32_t x = slot_of(row);
    for (int n = 0; n < 2 * kMaxList; ++n, x = (x + 1) % (2 * kMaxList)) {
      const int32_t k = atomicCAS(&key[x], -1, row);
      if (k != -1 && k != row) continue;
      atomicMin(&at[x], i);
      return;
    }
  }
  __device__ __forceinline__ int first(int32_t row) const {
    uint32_t x = slot_of(row);
    for (int n = 0; n < 2 * kMaxList && key[x] != row; ++n) x = (x + 1) % (2 * kMaxList);
    return at[x];
  }
};

__device__ __forceinline__ bool good_len(const CacheView& c, int64_t len) {
  return len >= 0 && len <= (static_cast<int64_t>(c.width) << c.ps_log2);
}

__global__ void __launch_bounds__(kMaxList) extend_plan_kernel(CacheView c, int n,
                                                              const int32_t* rows,
                                                              const int32_t* add, Plan* plan,
                                                              int32_t* list, uint32_t* status) {
  __shared__ int sh[33];
  __shared__ int64_t sums[33];
  __shared__ FirstAt listed;
  const int i = threadIdx.x;
  pdl_launch_dependents();
  const Counts counts = load_counts(c.ref, c.num_pages, 0);
  listed.clear();
  bool ok = false;
  int row = -1, more = 0, need = 0, first = 0;
  int64_t len = 0, grown = 0;
  if (i < n) {
    row = rows[i];
    more = add[i];
    if (row < 0 || row >= c.num_rows) row = -1;
    if (row >= 0) len = c.len[row];
  }
  __syncthreads();
  if (row >= 0) listed.put(row, i);
  __syncthreads();
  if (i < n) {
    if (row >= 0 && more >= 0 && listed.first(row) == i) {
      grown = len + more;
      if (good_len(c, len) && good_len(c, grown)) {
        ok = true;
        const int64_t ps1 = (1 << c.ps_log2) - 1;
        first = static_cast<int>((len + ps1) >> c.ps_log2);
        need = static_cast<int>((grown + ps1) >> c.ps_log2) - first;
      }
    }
    if (!ok) set_device_status(status, DEV_BAD_INDEX);
  }
  // (an entry may ask for 2^27 pages: the sum of a list passes 32 bits)
  int64_t total;
  const int64_t rank = block_scan<int64_t>(ok ? need : 0, sums, &total);
  const int n_free = scan_free(counts, c.ref, c.num_pages, static_cast<int>(total < INT_MAX ? total : INT_MAX), list, sh);
  if (i >= n) return;
  if (ok && need > 0 && rank + need > n_free) {
    set_device_status(status, DEV_NO_PAGES);
    ok = false;
  }
  plan->row[i] = ok ? row : -1;
  plan->first[i] = first;
  plan->count[i] = need;
  plan->rank[i] = static_cast<int32_t>(rank);     // (fits if the entry is not left out)
  if (ok) c.len[row] = static_cast<int32_t>(grown);
}

__global__ void __launch_bounds__(kCopyThreads) extend_kernel(CacheView c, const Plan* plan,
                                                             const int32_t* list) {
  const int i = blockIdx.x;
  pdl_wait();
  const int row = plan->row[i], first = plan->first[i], count = plan->count[i], rank = plan->rank[i];
  if (row < 0) return;
  for (int j = threadIdx.x; j < count; j += kCopyThreads) {
    const int page = list[rank + j];
    c.table[static_cast<int64_t>(row) * c.width + first + j] = page;
    c.ref[page] = 1;
  }
}

__global__ void __launch_bounds__(kMaxList) fork_plan_kernel(CacheView c, int n,
                                                            const int32_t* parents,
                                                            const int32_t* children, Plan* plan,
                                                            int32_t* list, uint32_t* status) {
  __shared__ int sh[33];
  __shared__ FirstAt listed;
  const int i = threadIdx.x;
  pdl_launch_dependents();
  const Counts counts = load_counts(c.ref, c.num_pages, 0);
  listed.clear();
  bool ok = false;
  int child = -1, parent = -1;
  int64_t len = 0;
  if (i < n) {
    child = children[i];
    parent = parents[i];
    ok = child >= 0 && child < c.num_rows && parent >= 0 && parent < c.num_rows;
    if (ok) {
      len = c.len[parent];
      ok = c.len[child] == 0 && good_len(c, len) && child != parent;
    }
  }
  __syncthreads();
  const bool row = child >= 0 && child < c.num_rows;
  if (row) listed.put(child, i);
  __syncthreads();
  if (i < n) {
    ok = ok && row && listed.first(child) == i;
    if (!ok) set_device_status(status, DEV_BAD_INDEX);
  }
  const int full = static_cast<int>(len >> c.ps_log2);
  const int part = static_cast<int>(len & ((1 << c.ps_log2) - 1));
  int total;
  // every length above is read before the first one is written below
  const int rank = block_scan(ok && part > 0 ? 1 : 0, sh, &total);
  const int n_free = scan_free(counts, c.ref, c.num_pages, total, list, sh);
  if (i >= n) return;
  if (ok && part > 0 && rank >= n_free) {
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

// The first `tokens` tokens of a page's keys and values, page src to page dst, in 16-byte units,
// four of each in flight a thread; this block's share of them is number y of ny.
__device__ __forceinline__ void copy_tokens(const CacheView& c, int64_t src, int64_t dst, int tokens, int y,
                                            int ny) {
  const int d8 = c.D / 8;
  const int units = tokens * c.Hkv * d8;
  const uint4* sk = reinterpret_cast<const uint4*>(c.k + src * c.page_stride);
  const uint4* sv = reinterpret_cast<const uint4*>(c.v + src * c.page_stride);
  uint4* dk = reinterpret_cast<uint4*>(c.k + dst * c.page_stride);
  uint4* dv = reinterpret_cast<uint4*>(c.v + dst * c.page_stride);
  const int per_head = tokens * d8;
  const bool runs = c.head_stride > c.tok_stride;     // [Hkv, page_size, D]: a run a head
  const int step = ny * kCopyThreads;
  for (int u0 = y * kCopyThreads + threadIdx.x; u0 < units; u0 += 4 * step) {
    uint4 k[4], v[4];
    int64_t at[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int u = u0 + x * step;
      at[x] = u;
      if (runs) {
        const int h = u / per_head;
        at[x] = h * (c.head_stride / 8) + (u - h * per_head);
      }
      if (u < units) {
        k[x] = __ldcs(sk + at[x]);
        v[x] = __ldcs(sv + at[x]);
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (u0 + x * step < units) {
        dk[at[x]] = k[x];
        dv[at[x]] = v[x];
      }
  }
}

// Blocks (pair, y): the pair's table columns and page units are shared out over gridDim.y.
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(CacheView c, const Plan* plan,
                                                           const int32_t* list, uint32_t* status) {
  const int i = blockIdx.x, y = blockIdx.y, ny = gridDim.y;
  pdl_wait();
  // (in one round of loads: each costs 0.6 us here)
  const int row = plan->row[i], parent = plan->from[i], full = plan->first[i], part = plan->count[i];
  const int rank = plan->rank[i];
  if (row < 0) return;
  const int32_t* src = c.table + static_cast<int64_t>(parent) * c.width;
  int32_t* dst = c.table + static_cast<int64_t>(row) * c.width;
  const int page = part > 0 ? list[rank] : -1, from = part > 0 ? src[full] : -1;
  for (int j = y * kCopyThreads + threadIdx.x; j < full; j += ny * kCopyThreads) {
    const int p = src[j];
    dst[j] = p;
    if (p >= 0 && p < c.num_pages)
      atomicAdd(c.ref + p, 1);
    else
      set_device_status(status, DEV_BAD_INDEX);
  }
  if (part > 0) {
    if (y == 0 && threadIdx.x == 0) {
      dst[full] = page;
      c.ref[page] = 1;
    }
    if (from >= 0 && from < c.num_pages)
      copy_tokens(c, from, page, part, y, ny);
    else if (y == 0 && threadIdx.x == 0)
      set_device_status(status, DEV_BAD_INDEX);
  }
}

__global__ void __launch_bounds__(kCopyThreads) free_kernel(CacheView c, int n, const int32_t* rows,
                                                           uint32_t* status) {
  const int i = blockIdx.x;
  const int row = rows[i];
  int dup = 0;
  for (int j = threadIdx.x; j < i; j += kCopyThreads) dup |= rows[j] == row;
  const bool in = row >= 0 && row < c.num_rows;
  int32_t* t = c.table + static_cast<int64_t>(in ? row : 0) * c.width;
  // the length and the first pages in one round of loads
  const int64_t len = in ? c.len[row] : -1;
  int next = in && threadIdx.x < c.width ? t[threadIdx.x] : -1;
  dup = __syncthreads_or(dup);
  if (!in || dup || !good_len(c, len)) {
    if (threadIdx.x == 0) set_device_status(status, DEV_BAD_INDEX);
    return;
  }
  const int pages = static_cast<int>((len + (1 << c.ps_log2) - 1) >> c.ps_log2);
  for (int j = threadIdx.x; j < pages; j += kCopyThreads) {
    const int page = next;
    t[j] = -1;
    if (j + kCopyThreads < pages) next = t[j + kCopyThreads];
    if (page >= 0 && page < c.num_pages)
      atomicSub(c.ref + page, 1);
    else
      set_device_status(status, DEV_BAD_INDEX);
  }
  __syncthreads();
  if (threadIdx.x == 0) c.len[row] = 0;
}

// The compaction's workspace behind the plan, int32 [pages] each: to[p], the page that p moves to
// (-1: not live), and from[m], the source of move m.  Out of place every live page moves, to its
// rank among them (move m is to page m).  In place the live pages from n_live on move
// into the holes below, both in ascending order; hole[m], a third list, is move m's target.
struct Moves {
  int32_t *to, *from, *hole;
};
__host__ __device__ inline Moves moves_of(void* ws, int64_t pages) {
  int32_t* l = page_list(ws);
  return {l, l + pages, l + 2 * pages};
}

__global__ void __launch_bounds__(kScanThreads) compact_plan_kernel(const int32_t* ref, int64_t pages,
                                                                   int inplace, Moves mv, Plan* plan,
                                                                   int32_t* n_live) {
  __shared__ int sh[33];
  pdl_launch_dependents();
  // ranks among the live pages
  int live = 0;
  for (int64_t p0 = 0; p0 < pages; p0 += kScanThreads * kScanPer) {
    const int64_t p = p0 + threadIdx.x * kScanPer;
    uint32_t bits = 0;
    int r[kScanPer];
#pragma unroll
    for (int k = 0; k < kScanPer; ++k) r[k] = p + k < pages ? __ldcg(ref + p + k) : 0;
#pragma unroll
    for (int k = 0; k < kScanPer; ++k) bits |= r[k] > 0 ? 1u << k : 0u;
    int total;
    int at = live + block_scan(__popc(bits), sh, &total);
#pragma unroll
    for (int k = 0; k < kScanPer; ++k)
      if (p + k < pages) {
        const bool is = bits & (1u << k);
        mv.to[p + k] = is ? at : -1;
        if (is) mv.from[at++] = static_cast<int32_t>(p + k);
      }
    live += total;
  }
  if (threadIdx.x == 0) {
    if (n_live != nullptr) *n_live = live;
    if (!inplace) plan->n_moves = live;
  }
  if (!inplace) return;
  __syncthreads();
  // pages below n_live that are not live: the holes; the live ones there stay
  int holes = 0;
  for (int64_t p0 = 0; p0 < live; p0 += kScanThreads) {
    const int64_t p = p0 + threadIdx.x;
    const int is = (p < live && mv.to[p] < 0) ? 1 : 0;
    int total;
    const int at = holes + block_scan(is, sh, &total);
    if (is) mv.hole[at] = static_cast<int32_t>(p);
    holes += total;
  }
  __syncthreads();
  const int stay = live - holes;          // live pages below n_live: moves are from[stay ...]
  for (int64_t p = threadIdx.x; p < pages; p += kScanThreads) {
    const int rank = mv.to[p];
    if (rank >= 0) mv.to[p] = rank < stay ? static_cast<int32_t>(p) : mv.hole[rank - stay];
  }
  __syncthreads();
  // the movers to the front, in their order
  for (int m0 = 0; m0 < holes; m0 += kScanThreads) {
    const int m = m0 + threadIdx.x;
    const int f = m < holes ? mv.from[stay + m] : 0;
    __syncthreads();
    if (m < holes) mv.from[m] = f;
    __syncthreads();
  }
  if (threadIdx.x == 0) plan->n_moves = holes;
}

// Copies the moves' keys and values through shared memory by bulk copies (one thread, six
// 32 KB stages, four loads ahead of the stores: bound by HBM, 2 x the moved bytes), while the
// block's other threads write the tables, lengths and counts.
constexpr int kPieces = 32768, kStages = 6, kAhead = 4;
constexpr int kMoveThreads = 288;

__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(CacheView sc, CacheView dc, int inplace,
                                                                   Moves mv, const Plan* plan,
                                                                   uint32_t* status) {
  extern __shared__ __align__(128) uint8_t stage[];
  __shared__ __align__(8) uint64_t full[kStages];
  const int tid = threadIdx.x;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
    // the barriers are used by the bulk copies
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait();
  const int n = plan->n_moves;
  if (tid >= 256) {
    if (tid > 256) return;
    // ---------------------------------------------------------------- the copies
    const int64_t page_bytes = 2ll * sc.Hkv * sc.D << sc.ps_log2;
    const int pieces = static_cast<int>((page_bytes + kPieces - 1) / kPieces);
    const int64_t units = static_cast<int64_t>(n) * 2 * pieces;
    auto unit = [&](int64_t u, const uint8_t** src, uint8_t** dst) -> uint32_t {
      const int64_t m = u / (2 * pieces);
      const int x = static_cast<int>(u - m * 2 * pieces), half = x / pieces, piece = x - half * pieces;
      const int64_t from = mv.from[m], to = inplace ? mv.hole[m] : m;
      const int64_t off = static_cast<int64_t>(piece) * kPieces;
      *src = reinterpret_cast<const uint8_t*>((half ? sc.v : sc.k) + from * sc.page_stride) + off;
      *dst = to < dc.num_pages ? reinterpret_cast<uint8_t*>((half ? dc.v : dc.k) + to * dc.page_stride) + off : nullptr;
      const int64_t left = page_bytes - off;
      return static_cast<uint32_t>(left < kPieces ? left : kPieces);
    };
    const int64_t mine = units > blockIdx.x ? (units - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    auto load = [&](int64_t k) {
      const uint8_t* src;
      uint8_t* dst;
      const uint32_t bytes = unit(blockIdx.x + k * gridDim.x, &src, &dst);
      const int s = static_cast<int>(k % kStages);
      mbar_arrive_expect_tx(&full[s], bytes);
      bulk_load(stage + s * kPieces, src, bytes, &full[s]);
    };
    for (int64_t k = 0; k < kAhead && k < mine; ++k) load(k);
    int64_t k = 0;
    for (; k < mine; ++k) {
      const int s = static_cast<int>(k % kStages);
      if (!mbar_wait(&full[s], static_cast<uint32_t>(k / kStages) & 1u, status)) break;
      const uint8_t* src;
      uint8_t* dst;
      const uint32_t bytes = unit(blockIdx.x + k * gridDim.x, &src, &dst);
      fence_proxy_async_smem();
      if (dst != nullptr) bulk_store(dst, stage + s * kPieces, bytes);
      bulk_commit();
      if (k + kAhead < mine) {
        // its stage was stored kStages - kAhead groups ago
        bulk_wait_read<kStages - kAhead>();
        load(k + kAhead);
      }
    }
    // every copy has landed before the block ends (after a wait that gave up: the loads, bounded)
    if (k < mine)
      for (int64_t j = k; j < mine && j < k + kAhead; ++j)
        mbar_wait_ns(&full[j % kStages], static_cast<uint32_t>(j / kStages) & 1u, 200000000ull);
    bulk_wait_all();
    return;
  }
  // ------------------------------------------------------- tables, lengths and counts
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  const int64_t i0 = blockIdx.x * 256ll + tid;
  const int64_t total = static_cast<int64_t>(sc.num_rows) * sc.width;
  for (int64_t i = i0; i < total; i += stride) {
    const int page = sc.table[i];
    int d = -1;
    if (page >= 0 && page < sc.num_pages) {
      d = mv.to[page];
      if (d >= dc.num_pages) d = -1;
    } else {
      // no page: reported where the row's length makes it one that is listed
      const int64_t row = i <= UINT_MAX ? static_cast<unsigned>(i) / static_cast<unsigned>(sc.width) : i / sc.width;
      const int64_t len = sc.len[row];
      if (good_len(sc, len) && (i - row * sc.width) << sc.ps_log2 < len) set_device_status(status, DEV_BAD_INDEX);
    }
    dc.table[i] = d;
  }
  for (int64_t i = i0; i < sc.num_rows; i += stride)
    if (!good_len(sc, sc.len[i])) set_device_status(status, DEV_BAD_INDEX);
  if (!inplace) {
    for (int64_t i = i0; i < sc.num_rows; i += stride) dc.len[i] = sc.len[i];
    for (int64_t p = i0; p < dc.num_pages; p += stride) dc.ref[p] = p < n ? sc.ref[mv.from[p]] : 0;
    if (i0 == 0 && n > dc.num_pages) set_device_status(status, DEV_NO_PAGES);
  } else {
    for (int64_t m = i0; m < n; m += stride) {
      const int from = mv.from[m];
      sc.ref[mv.hole[m]] = sc.ref[from];
      sc.ref[from] = 0;
    }
  }
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

// Behind the plan: the list of free pages, or the compaction's three lists.
size_t cache_pages_ws_bytes(int64_t num_pages) {
  return sizeof(Plan) + static_cast<size_t>(num_pages) * 3 * sizeof(int32_t);
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
  extend_plan_kernel<<<1, kMaxList, 0, s>>>(c, n, rows, add, plan, page_list(ws), status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(extend_kernel, dim3(static_cast<unsigned>(n)), kCopyThreads, 0, s, c,
                      static_cast<const Plan*>(plan), static_cast<const int32_t*>(page_list(ws)));
}

cudaError_t launch_cache_fork(const CacheView& c, int n, const int32_t* parents,
                              const int32_t* children, void* ws, uint32_t* status, cudaStream_t s) {
  Plan* plan = static_cast<Plan*>(ws);
  fork_plan_kernel<<<1, kMaxList, 0, s>>>(c, n, parents, children, plan, page_list(ws), status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // enough blocks to fill the GPU, while each has a few hundred units (128 rows freed and forked:
  // 12.3 us; with half as many blocks 14.1, with twice as many 12.4)
  int ny = 4 * num_sms() / n;
  ny = ny < 1 ? 1 : (ny > 16 ? 16 : ny);
  return launch_after(fork_kernel, dim3(static_cast<unsigned>(n), static_cast<unsigned>(ny)), kCopyThreads, 0, s, c,
                      static_cast<const Plan*>(plan), static_cast<const int32_t*>(page_list(ws)), status);
}

cudaError_t launch_cache_free(const CacheView& c, int n, const int32_t* rows, uint32_t* status,
                              cudaStream_t s) {
  free_kernel<<<static_cast<unsigned>(n), kCopyThreads, 0, s>>>(c, n, rows, status);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CacheView& src, const CacheView& dst, bool inplace,
                                 int32_t* n_live, void* ws, uint32_t* status, cudaStream_t s) {
  static bool attr_set[kMaxDeviceCache] = {};
  const int dev = cached_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(compact_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kStages * kPieces);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  Plan* plan = static_cast<Plan*>(ws);
  const Moves mv = moves_of(ws, src.num_pages);
  compact_plan_kernel<<<1, kScanThreads, 0, s>>>(src.ref, src.num_pages, inplace ? 1 : 0, mv, plan, n_live);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(compact_move_kernel, dim3(static_cast<unsigned>(num_sms())), kMoveThreads, kStages * kPieces, s,
                      src, dst, inplace ? 1 : 0, mv, static_cast<const Plan*>(plan), status);
}

}  // namespace ls
