// Attention of packed new tokens over the cache's pages.
//
//   o = softmax(s q K^T) V over the keys 0 .. position of the token's own sequence,
//   lse = log sum exp(s q k)
//
// Three kernels, each started while the one before drains (programmatic launch):
//
// cache_plan_kernel (one block).  The lengths live on the device, so the work is cut there.  A
//   segment is a run of packed tokens and a run of 128-key tiles of one table row: a sequence's
//   tokens over its keys, or, for a group with shared pages, all the group's tokens over the
//   shared keys (read once) and each sequence's over the rest.  Key runs are split into
//   chunks so that the tile counts of all SMs come out even (the chunk length with the least
//   estimated makespan of 16 candidates); a segment of more than one chunk, or a token in two
//   segments, leaves partial results.  Output: lists of jobs.
//
// cache_attn_kernel<D, wide> (persistent, 384 threads).  Warp 0 feeds Q, K and V by TMA (pages
//   of 16 .. 256 tokens: a 128-key tile is 128 / page_size boxes), warp 1 issues tcgen05.mma,
//   warps 4-7 and 8-11 are the softmax of two streams (thread = TMEM lane = (token, head)
//   row; running maximum and sum in fp32, O rescaled in TMEM only when the maximum grows by
//   more than 2^8).
//   wide: segments of more than 64 rows.  The two streams are two 128-row Q tiles that use
//     the same K and V tiles; bound by the softmax's latency between a tile's two products and,
//     on long calls, by the power limit (1,024 tokens of 40 heads over 131,072 keys: 1.87-1.93 ms
//     in a graph, 1.96 a call: 1,400-1,460 TFLOP/s of 1,930 measured; over 16,384 keys 308 us,
//     1,080 TFLOP/s).
//   narrow: at most 64 rows (a token or a few per sequence).  The two streams are two
//     independent jobs with K/V tiles of their own, so one's softmax hides the other's loads;
//     Q takes 16 KB instead of 32, which leaves room for three K and three V tiles in flight
//     (192 KB an SM).  M = 128 MMAs with most rows idle still take less than half the time that
//     the tile's 64 KB take from HBM; bound by HBM (40 sequences of up to 65,000 keys: 829 us for
//     5.7 GB, 94 % of the 7.35 TB/s of a kernel that only reads; 8 responses that share 32,768 of 34,000 keys: 46 us
//     for 173 MB, of which the plan and the join, latency both, are about ten).
//
// cache_join_kernel.  Combines a token's partial results in chunk order (deterministic), and
//   writes zeros for tokens that see no key.
//
// V rows behind a sequence's end are cleared in shared memory before the MMA (0 x NaN); pages
// outside the pool read as zeros (the TMA's fill).  P is rounded to bf16, the type of V, for the
// tensor cores (one kind of operand a product; P in two parts would double that product); the sum is
// taken before that rounding.  The outputs' error against float64 is 0.0023 relative, that of fp32
// probabilities 0.0017, most of both the output's own rounding.  Every wait is bounded as in the replay kernels.
#include <climits>

#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"

namespace ls {
namespace {

constexpr int kThreads = 384;
// Registers of a thread: the launch gives all 168 a thread (checked); the softmax warpgroups, which hold a row of
// 128 scores, take what the control warpgroup leaves (without the split 108 bytes of a softmax
// thread spill: 1,024 tokens over 131,072 keys 1,966 us instead of 1,915, 12 sequences' groups
// 51.3 instead of 47.4).
constexpr int kRegsLaunch = 168, kRegsControl = 112, kRegsSoftmax = 192;
static_assert(kRegsControl + 2 * kRegsSoftmax <= 3 * kRegsLaunch, "more than the launch gives");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kNarrowRows = 64;
constexpr int kMaxTiles = 1 << 24;     // 128-key tiles of the longest sequence

// A run of packed tokens over a run of key tiles of one table row.
struct Seg {
  int t0, n_tok;
  int row;
  int lim;          // token t sees lim + t keys; INT_MIN: lims[t]
  int tile0, tiles; // first 128-key tile, tiles in all
  int key_end;      // keys from here on are not read
  int chunk, chunks;
  int part;         // first row of its partial results; -1: written to the output
  int jobs, rows;   // jobs and partial rows of it (planning); a group's shared length before that
};
// One (key head, chunk) of a segment, for one Q tile (narrow) or two (wide).
struct Job {
  int t0, n_tok, row, lim;
  int tile0, n_tiles, key_end, kv;
  int part;         // row of its first token's first head among the partial rows; -1: output
  int pad[3];
};
struct Info {
  int n_jobs[2];    // narrow, wide
  int grouped;
};

__device__ __forceinline__ int qt_of(int g, bool wide) { return (wide ? 128 : kNarrowRows) / g; }
__device__ __forceinline__ bool is_wide(const Seg& s, int g) { return s.n_tok > kNarrowRows / g; }

// Key tiles that tokens t0 .. t0 + n - 1 of a segment need at most.
__device__ __forceinline__ int tiles_of(const Seg& s, int t_end) {
  if (s.lim == INT_MIN) return s.tiles;
  const int keys = s.lim + t_end - 1 - 128 * s.tile0;
  const int n = keys <= 0 ? 0 : (keys + 127) / 128;
  return n < s.tiles ? n : s.tiles;
}

// x / d for 0 <= x < 2^24, inv = 1 / d (an integer division takes a hundred cycles).
__device__ __forceinline__ int quick_div(int x, int d, float inv) {
  int q = static_cast<int>(static_cast<float>(x) * inv);
  const int r = x - q * d;
  q += r >= d ? 1 : 0;
  return r < 0 ? q - 1 : q;
}

// ceil(x / d), x and d counts of tiles or tokens.
__device__ __forceinline__ int ceil_div(int x, int d) {
  if (x >= 1 << 20) return static_cast<int>((static_cast<int64_t>(x) + d - 1) / d);
  return quick_div(x + d - 1, d, __fdividef(1.0f, static_cast<float>(d)));
}

constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;
constexpr int kCandidates = 16;      // of each class: one warp's lanes for both

struct PlanArgs {
  CacheView c;
  int S;
  int64_t T;
  const int32_t* rows;
  const int32_t* cu;
  int max_new;
  int64_t max_len;
  int group;
  const int32_t* shared;
  uint8_t* ws;
  CacheAttnLayout l;
  int sms;
  uint32_t* status;
};

__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const __grid_constant__ PlanArgs a) {
  // the segments, and the jobs of each class before a segment
  extern __shared__ __align__(16) uint8_t dyn[];
  const int cap = a.S + (a.group > 1 ? a.S / a.group : 0);
  Seg* segs = reinterpret_cast<Seg*>(dyn);
  int* first[2] = {reinterpret_cast<int*>(dyn + cap * sizeof(Seg)),
                   reinterpret_cast<int*>(dyn + cap * sizeof(Seg)) + cap};
  __shared__ int sh_max[2], sh_c[2], sh_grouped, sh_bad;
  __shared__ int sh_base[2];
  __shared__ float sh_work[2][kPlanWarps];
  __shared__ unsigned long long cost_of[2 * kCandidates];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = a.c.Hq / a.c.Hkv;
  Info* info = reinterpret_cast<Info*>(a.ws + a.l.info);
  int* lims = reinterpret_cast<int*>(a.ws + a.l.lims);
  pdl_launch_dependents();

  if (tid < 2) sh_max[tid] = 0;
  if (tid == 0) sh_bad = 0;
  __syncthreads();

  // the entries: tokens, table row, length
  for (int b = tid; b < a.S; b += kPlanThreads) {
    Seg s;
    const int c0 = a.cu[b], c1 = a.cu[b + 1];
    const int row = a.rows != nullptr ? a.rows[b] : b;
    // (loaded beside the offsets)
    const int64_t held = row >= 0 && row < a.c.num_rows ? a.c.len[row] : -1;
    const int shared = a.group > 1 && b % a.group == 0 ? a.shared[b / a.group] : 0;
    const bool run = c0 >= 0 && c1 >= c0 && c1 <= a.T;
    if (!run) sh_bad = 1;
    s.t0 = run ? c0 : 0;
    s.n_tok = run ? c1 - c0 : 0;
    s.row = row;
    bool ok = run && (s.n_tok == 0 || (s.row >= 0 && s.row < a.c.num_rows && s.n_tok <= a.max_new));
    int64_t len = 0;
    if (run && s.n_tok == 0) {
      s.row = -1;              // nothing new: not looked at
    } else if (ok) {
      len = held;
      ok = len >= 0 && len <= a.max_len && len <= (static_cast<int64_t>(a.c.width) << a.c.ps_log2);
    }
    if (!ok) {
      set_device_status(a.status, DEV_BAD_INDEX);
      len = 0;
      s.row = -1;
    }
    s.key_end = static_cast<int>(len);
    s.lim = s.key_end - (run ? c1 : 0) + 1;
    s.tile0 = 0;
    s.tiles = s.n_tok > 0 ? static_cast<int>((len + 127) / 128) : 0;
    s.chunk = s.chunks = 0;
    s.part = -1;
    s.jobs = 0;
    s.rows = shared;
    segs[b] = s;
  }
  // groups: the shared keys as one segment, if the partial rows of both parts fit
  const int n_groups = a.group > 1 ? a.S / a.group : 0;
  if (tid == 0)
    sh_grouped = n_groups > 0 && 2 * a.T * a.c.Hq <= a.l.rows_narrow &&
                 (a.l.rows_wide == 0 || 2 * a.T * a.c.Hq <= a.l.rows_wide);
  __syncthreads();
  const bool grouped = sh_grouped != 0 && sh_bad == 0;
  if (sh_bad != 0) {
    // offsets that fall: the runs may overlap, and their jobs pass the lists; no entry is done
    for (int b = tid; b < a.S; b += kPlanThreads) segs[b].n_tok = segs[b].tiles = 0;
    __syncthreads();
  }
  const int n_segs = a.S + (grouped ? n_groups : 0);
  // whether segment i's tokens are in two segments
  const float inv_group = __fdividef(1.0f, static_cast<float>(a.group));
  auto in_two = [&](int i) {
    return grouped && segs[a.S + (i < a.S ? quick_div(i, a.group, inv_group) : i - a.S)].tiles > 0;
  };
  if (grouped) {
    for (int i = tid; i < n_groups; i += kPlanThreads) {
      int lead = -1;
      for (int b = i * a.group; b < (i + 1) * a.group && lead < 0; ++b)
        if (segs[b].row >= 0) lead = b;
      int sh_len = lead < 0 ? 0 : segs[i * a.group].rows;
      if (sh_len < 0) sh_len = 0;
      if (lead >= 0 && sh_len > segs[lead].key_end) sh_len = segs[lead].key_end;
      const int tiles = sh_len / 128;
      Seg s;
      const Seg& tail = segs[(i + 1) * a.group - 1];
      s.t0 = segs[i * a.group].t0;
      const int t1 = tail.t0 + tail.n_tok;
      // (an entry above max_new is refused but its tokens are among these: more of them than the
      // bounds allow could be wide where the host, by the bounds, launches no wide kernel; the
      // group's entries then read their keys for themselves)
      const bool run = t1 >= s.t0 && t1 - s.t0 <= static_cast<int64_t>(a.max_new) * a.group;
      s.n_tok = run ? t1 - s.t0 : 0;
      s.row = lead < 0 ? 0 : segs[lead].row;
      s.lim = INT_MIN;
      s.tile0 = 0;
      s.tiles = run && s.n_tok > 0 ? tiles : 0;
      s.key_end = tiles * 128;
      s.chunk = s.chunks = 0;
      s.part = -1;
      s.jobs = s.rows = 0;
      segs[a.S + i] = s;
    }
    __syncthreads();
    for (int b = warp; b < a.S; b += kPlanThreads / 32) {
      const Seg s = segs[b];
      const int shared = segs[a.S + quick_div(b, a.group, inv_group)].tiles;
      __syncwarp();
      if (lane == 0 && shared > 0) {
        segs[b].tile0 = shared;
        segs[b].tiles = s.tiles > shared ? s.tiles - shared : 0;
      }
      for (int i = lane; i < s.n_tok; i += 32) {
        const int n = s.row < 0 ? 0 : s.lim + s.t0 + i;
        lims[s.t0 + i] = n < 0 ? 0 : n;
      }
    }
  }
  __syncthreads();

  // work of each class, in key tiles of one Q tile (narrow) or pair of them (wide); the estimates
  // are in fp32 (64-bit integers take microseconds here)
  const int qn = qt_of(g, false), per_pair = 2 * qt_of(g, true);
  {
    float work[2] = {0.0f, 0.0f};
    int longest[2] = {0, 0};
    for (int i = tid; i < n_segs; i += kPlanThreads) {
      const int tiles = segs[i].tiles, n = segs[i].n_tok;
      const int w = n > qn ? 1 : 0;
      const float x = static_cast<float>(w ? ceil_div(n, per_pair) : 1) * static_cast<float>(a.c.Hkv * tiles);
      work[0] += w ? 0.0f : x;
      work[1] += w ? x : 0.0f;
      if (w) longest[1] = max(longest[1], tiles); else longest[0] = max(longest[0], tiles);
      segs[i].jobs = in_two(i) ? 1 : 0;      // (until the jobs are counted)
    }
    if (warp * 32 < n_segs) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) work[c] += __shfl_xor_sync(0xffffffffu, work[c], off);
        longest[c] = __reduce_max_sync(0xffffffffu, longest[c]);
        if (lane == 0) {
          sh_work[c][warp] = work[c];
          atomicMax(&sh_max[c], longest[c]);
        }
      }
    }
  }
  __syncthreads();
  // candidates, a warp each: chunks that make k rounds of jobs over all streams
#pragma unroll 1
  for (int x = warp; x < 2 * kCandidates; x += kPlanWarps) {
    const int cls = x / kCandidates, v = x % kCandidates;
    const int longest = sh_max[cls];
    if (lane == 0) cost_of[x] = ~0ull;
    if (longest == 0) continue;
    // wide: 15 round counts; narrow: five, each with chunks an eighth and a quarter longer too (a
    // few short sequences then stay whole); and no split
    const float round = static_cast<float>(cls ? a.sms : 2 * a.sms);
    const float rounds = static_cast<float>(cls ? v + 1 : v / 3 + 1), more = cls ? 1.0f : 1.0f + 0.125f * (v % 3);
    float W = 0.0f;
    for (int w = 0; w < kPlanWarps && w * 32 < n_segs; ++w) W += sh_work[cls][w];
    const float Cf = ceilf(__fdividef(W * more, round * rounds));
    int C = v == kCandidates - 1 || Cf >= static_cast<float>(longest) ? longest : static_cast<int>(Cf);
    const int least = cls ? 8 : 2;
    C = C < least ? least : C;
    C = C > longest ? longest : C;
    // the longest segment's chunks all alike
    C = ceil_div(longest, ceil_div(longest, C));
    // (fp32 quotients of up to 2^20 tiles are on the right side of an integer, or above it; more
    // tiles than that are rounded up by a millionth, so that the capacities hold)
    const float inv = __fdividef(longest < 1 << 20 ? 1.0f : 1.000001f, static_cast<float>(C));
    float jobs = 0.0f, rows = 0.0f;
    for (int i = lane; i < n_segs; i += 32) {
      const int tiles = segs[i].tiles, n = segs[i].n_tok;
      if (tiles == 0 || (n > qn) != (cls == 1)) continue;
      const float chunks = ceilf(static_cast<float>(tiles) * inv);
      const float pairs = static_cast<float>(cls ? ceil_div(n, per_pair) : 1);
      jobs += static_cast<float>(a.c.Hkv) * pairs * chunks;
      if (chunks > 1.0f || segs[i].jobs != 0) rows += static_cast<float>(a.c.Hq) * chunks * static_cast<float>(n);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      jobs += __shfl_xor_sync(0xffffffffu, jobs, off);
      rows += __shfl_xor_sync(0xffffffffu, rows, off);
    }
    // (the capacities with the estimates' rounding to spare; without a split they suffice exactly)
    const float cap = 0.999f * static_cast<float>(cls ? a.l.max_wide : a.l.max_narrow);
    const float most = 0.999f * static_cast<float>(cls ? a.l.rows_wide : a.l.rows_narrow);
    if (lane == 0 && (v == kCandidates - 1 || (jobs <= cap && rows <= most))) {
      // makespan in tiles (3 us of the whole GPU's narrow streams, 1.8 us of wide ones): whole rounds,
      // what a job costs beside its tiles, and the partial rows, written and read at 5 TB/s
      // (without those 1,024 tokens over 16,384 keys take 323 us, so 308); equal ones: the longer
      // chunks
      const float cost = ceilf(__fdividef(jobs, round)) * (static_cast<float>(C) + (cls ? 4.5f : 3.0f)) +
                         rows * (cls ? 1.1e-4f : 7e-5f);
      cost_of[x] = (static_cast<unsigned long long>(__float_as_uint(cost)) << 25) |
                   static_cast<unsigned long long>(kMaxTiles - C);
    }
  }
  __syncthreads();
  if (warp == 0) {
    unsigned long long best = cost_of[lane];
#pragma unroll
    for (int off = kCandidates / 2; off > 0; off >>= 1) {
      const unsigned long long u = __shfl_xor_sync(0xffffffffu, best, off);
      best = u < best ? u : best;
    }
    if (lane % kCandidates == 0)
      sh_c[lane / kCandidates] = best == ~0ull ? kMaxTiles : kMaxTiles - static_cast<int>(best & 0x1FFFFFF);
  }
  __syncthreads();

  // chunks, jobs and partial rows of every segment
  for (int i = tid; i < n_segs; i += kPlanThreads) {
    Seg& s = segs[i];
    const int w = s.n_tok > qn ? 1 : 0;
    const bool two = s.jobs != 0;
    s.jobs = s.rows = 0;
    if (s.tiles == 0) continue;
    s.chunks = ceil_div(s.tiles, sh_c[w]);
    s.chunk = ceil_div(s.tiles, s.chunks);
    s.chunks = ceil_div(s.tiles, s.chunk);
    s.jobs = a.c.Hkv * (w ? ceil_div(s.n_tok, per_pair) : 1) * s.chunks;
    if (s.chunks > 1 || two) s.rows = a.c.Hq * s.chunks * s.n_tok;
  }
  __syncthreads();
  // their exclusive sums: a warp each for the jobs and the rows of the two classes
  if (warp < 4) {
    const int cls = warp & 1;
    const bool of_rows = warp >= 2;
    int base = of_rows && cls ? static_cast<int>(a.l.rows_narrow) : 0;
#pragma unroll 1
    for (int i0 = 0; i0 < n_segs; i0 += 32) {
      const int i = i0 + lane;
      int v = 0;
      if (i < n_segs && (segs[i].n_tok > qn) == (cls == 1)) v = of_rows ? segs[i].rows : segs[i].jobs;
      int s = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += u;
      }
      if (i < n_segs) {
        if (!of_rows)
          first[cls][i] = base + s - v;
        else if (v > 0)
          segs[i].part = base + s - v;
      }
      base += __shfl_sync(0xffffffffu, s, 31);
    }
    if (!of_rows && lane == 0) sh_base[cls] = base;
  }
  __syncthreads();
  if (tid == 0) {
    info->n_jobs[0] = sh_base[0];
    info->n_jobs[1] = sh_base[1];
    info->grouped = grouped ? 1 : 0;
  }

  // for the join
  {
    const int4* from = reinterpret_cast<const int4*>(segs);
    int4* to = reinterpret_cast<int4*>(a.ws + a.l.segs);
    for (int i = tid; i < n_segs * static_cast<int>(sizeof(Seg) / 16); i += kPlanThreads) to[i] = from[i];
  }
  // the job lists
#pragma unroll 1
  for (int cls = 0; cls < 2; ++cls) {
    Job* jobs = reinterpret_cast<Job*>(a.ws + (cls ? a.l.wide : a.l.narrow));
    const int* f = first[cls];
    const int n_jobs = sh_base[cls];
    const float inv_kv = 1.0f / static_cast<float>(a.c.Hkv);
    const bool quick = n_jobs < 1 << 24;
    for (int x = tid; x < n_jobs; x += kPlanThreads) {
      int lo = 0, hi = n_segs - 1;           // the last segment that starts at or before x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (f[mid] <= x) lo = mid; else hi = mid - 1;
      }
      const Seg s = segs[lo];
      int y = x - f[lo];
      Job j;
      j.row = s.row;
      j.lim = s.lim;
      j.key_end = s.key_end;
      int chunk;
      if (cls == 0) {
        // key heads of one chunk side by side: neighbours in memory
        chunk = quick ? quick_div(y, a.c.Hkv, inv_kv) : y / a.c.Hkv;
        j.kv = y - chunk * a.c.Hkv;
        j.t0 = s.t0;
        j.n_tok = s.n_tok;
      } else {
        // Q tiles of one (chunk, key head) side by side: they share its K and V through L2;
        // the last tokens, which see most keys, first
        const int pairs = (s.n_tok + per_pair - 1) / per_pair;
        const int p = pairs - 1 - y % pairs;
        y /= pairs;
        chunk = quick ? quick_div(y, a.c.Hkv, inv_kv) : y / a.c.Hkv;
        j.kv = y - chunk * a.c.Hkv;
        j.t0 = s.t0 + p * per_pair;
        j.n_tok = s.n_tok - p * per_pair < per_pair ? s.n_tok - p * per_pair : per_pair;
      }
      const int tiles = tiles_of(s, j.t0 + j.n_tok);
      j.tile0 = s.tile0 + chunk * s.chunk;
      j.n_tiles = tiles - chunk * s.chunk;
      j.n_tiles = j.n_tiles < 0 ? 0 : (j.n_tiles > s.chunk ? s.chunk : j.n_tiles);
      // rows of the partial results: [kv][chunk][token][head of the group]
      j.part = s.part < 0 ? -1 : s.part + ((j.kv * s.chunks + chunk) * s.n_tok + (j.t0 - s.t0)) * g;
      int4* out = reinterpret_cast<int4*>(jobs + x);
      out[0] = make_int4(j.t0, j.n_tok, j.row, j.lim);
      out[1] = make_int4(j.tile0, j.n_tiles, j.key_end, j.kv);
      out[2] = make_int4(j.part, 0, 0, 0);
    }
  }
}

// --------------------------------------------------------------------------------------
template <int D, bool kWide>
struct Cfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kQRows = kWide ? 128 : kNarrowRows;
  static constexpr int kQBox = kQRows * 128;               // bytes of one 64-column box of Q
  static constexpr int kQTile = kQBox * kBoxes;
  static constexpr int kN = (kWide ? 2 : 3) * (D == 128 ? 1 : 2);   // K (and V) ring stages
  static constexpr int kOffK = 2 * kQTile;
  static constexpr int kOffV = kOffK + kN * kTile;
  static constexpr int kOffBar = kOffV + kN * kTile;
  static constexpr int kBarQFull = 0, kBarQEmpty = 1, kBarKFull = 2;
  static constexpr int kBarKEmpty = kBarKFull + kN;
  static constexpr int kBarVFull = kBarKEmpty + kN;
  static constexpr int kBarVEmpty = kBarVFull + kN;
  static constexpr int kBarSFull = kBarVEmpty + kN;
  static constexpr int kBarPFull = kBarSFull + 2;          // [stream][half]
  static constexpr int kBarODone = kBarPFull + 4;
  static constexpr int kBarOFree = kBarODone + 2;
  static constexpr int kBarDrain = kBarOFree + 2;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kSmem = kOffBar + kNumBars * 8 + 16 + 1024;
  __host__ __device__ static constexpr uint32_t col_s(int q) { return 128u * q; }
  __host__ __device__ static constexpr uint32_t col_o(int q) { return 256u + D * q; }
};

struct AttnArgs {
  CacheView c;
  float scale;
  int layout;
  const Job* jobs;
  const int* n_jobs;
  const int* lims;
  float* part_o;
  float* part_lse;
  uint16_t* o;
  float* lse;
  uint32_t* status;
  // o starts on a 32-byte boundary: stores of whole sectors (8 x 1,000 tokens without a past 224 us,
  // 234 with halves; a 16-byte boundary is enough for the halves)
  bool o_whole;
};

// The two streams of an item: narrow, jobs 2 i and 2 i + 1; wide, the Q tiles of job i.
struct Streams {
  Job j[2];
  int n[2];         // key tiles of each stream
};
// (through L1: the producer loads a job one item ahead, the other warps of the SM then find it there)
__device__ __forceinline__ Job load_job(const Job* p) {
  Job j;
  const int4* v = reinterpret_cast<const int4*>(p);
  const int4 x = v[0], y = v[1], z = v[2];
  j.t0 = x.x; j.n_tok = x.y; j.row = x.z; j.lim = x.w;
  j.tile0 = y.x; j.n_tiles = y.y; j.key_end = y.z; j.kv = y.w;
  j.part = z.x;
  return j;
}
template <bool kWide>
__device__ __forceinline__ Streams load_streams(const AttnArgs& a, int item, int n_jobs, int qt, int g) {
  Streams s;
  s.n[0] = s.n[1] = 0;
  if (item >= (kWide ? n_jobs : (n_jobs + 1) / 2)) return s;
  if constexpr (kWide) {
    s.j[0] = load_job(a.jobs + item);
    s.j[1] = s.j[0];
    s.n[0] = s.j[0].n_tiles;
    s.n[1] = s.j[0].n_tok > qt ? s.j[0].n_tiles : 0;
    s.j[1].t0 += qt;
    s.j[1].n_tok -= qt;
    if (s.j[1].part >= 0) s.j[1].part += qt * g;
    if (s.j[0].n_tok > qt) s.j[0].n_tok = qt;
  } else {
    s.j[0] = load_job(a.jobs + 2 * item);
    s.n[0] = s.j[0].n_tiles;
    if (2 * item + 1 < n_jobs) {
      s.j[1] = load_job(a.jobs + 2 * item + 1);
      s.n[1] = s.j[1].n_tiles;
    }
  }
  return s;
}

// Stream q of an item (n_tiles = 0: none).
template <bool kWide>
__device__ __forceinline__ Job load_stream(const AttnArgs& a, int item, int q, int n_jobs, int qt, int g) {
  const int at = kWide ? item : 2 * item + q;
  Job j;
  j.n_tiles = 0;
  if (at >= n_jobs) return j;
  j = load_job(a.jobs + at);
  if (kWide && q == 1) {
    if (j.n_tok <= qt) j.n_tiles = 0;
    j.t0 += qt;
    j.n_tok -= qt;
    if (j.part >= 0) j.part += qt * g;
  } else if (kWide && j.n_tok > qt) {
    j.n_tok = qt;
  }
  return j;
}
// What the MMA warp needs of an item: the key tiles of its streams, and their keys from the first
// tile's first key on.
struct Runs {
  int n[2], keys[2];
};
template <bool kWide>
__device__ __forceinline__ Runs load_runs(const AttnArgs& a, int item, int n_jobs, int qt) {
  Runs r;
  r.n[0] = r.n[1] = r.keys[0] = r.keys[1] = 0;
#pragma unroll
  for (int q = 0; q < (kWide ? 1 : 2); ++q) {
    const int at = kWide ? item : 2 * item + q;
    if (at >= n_jobs) continue;
    const int4 y = reinterpret_cast<const int4*>(a.jobs + at)[1];
    r.n[q] = y.y;
    r.keys[q] = y.z - 128 * y.x;
    if (kWide) {
      r.n[1] = reinterpret_cast<const int4*>(a.jobs + at)[0].y > qt ? y.y : 0;
      r.keys[1] = r.keys[0];
    }
  }
  return r;
}

// The page indices of one stream: 64 table entries ahead in the producer warp's lanes.
struct PageWindow {
  const int32_t* row;
  int end;           // pages that hold keys
  int base, cur, next;
  __device__ __forceinline__ int fetch(int i, int lane) const {
    return i + lane < end ? __ldg(row + i + lane) : -1;
  }
  __device__ __forceinline__ void start(const CacheView& c, const Job& j, int lane) {
    row = c.table + static_cast<int64_t>(j.row) * c.width;
    end = (j.key_end + (1 << c.ps_log2) - 1) >> c.ps_log2;
    base = (j.tile0 * 128) >> c.ps_log2;
    cur = fetch(base, lane);
    next = fetch(base + 32, lane);
  }
  // Table entry i + mine of every lane; i is warp-uniform and never falls, mine < 32.
  __device__ __forceinline__ int get(int i, int mine, int lane) {
    if (i >= base + 32) {
      base += 32;
      cur = next;
      next = fetch(base + 32, lane);
    }
    const int at = i - base + mine;
    const int x = __shfl_sync(0xffffffffu, cur, at & 31), y = __shfl_sync(0xffffffffu, next, at & 31);
    return at < 32 ? x : y;
  }
};

template <int D, bool kWide>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ AttnArgs a) {
  using C = Cfg<D, kWide>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = a.c.Hq / a.c.Hkv;
  const int qt = C::kQRows / g;
  constexpr int kRowThreads = kWide ? 128 : kNarrowRows;   // softmax threads of a stream

  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(&bars[C::kBarQFull], 1);
    mbar_init(&bars[C::kBarQEmpty], 1);
    for (int i = 0; i < C::kN; ++i) {
      mbar_init(&bars[C::kBarKFull + i], 1);
      mbar_init(&bars[C::kBarKEmpty + i], 1);
      mbar_init(&bars[C::kBarVFull + i], 1);
      mbar_init(&bars[C::kBarVEmpty + i], 1);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&bars[C::kBarSFull + q], 1);
      mbar_init(&bars[C::kBarPFull + 2 * q], kRowThreads);
      mbar_init(&bars[C::kBarPFull + 2 * q + 1], kRowThreads);
      mbar_init(&bars[C::kBarODone + q], 1);
      mbar_init(&bars[C::kBarOFree + q], kRowThreads);
    }
    mbar_init(&bars[C::kBarDrain], 1);
    fence_mbar_init();
  }
  if (warp == 2) {
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  volatile int* vabort = &abort_flag;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_q);
  }
  pdl_launch_dependents();
  pdl_wait();                 // the job lists
  const int n_jobs = __ldcg(a.n_jobs);
  const int n_items = kWide ? n_jobs : (n_jobs + 1) / 2;

  if (warp < 4) {
    setreg_dec<kRegsControl>();
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer (whole warp)
      uint32_t kit = 0, vit = 0, uc = 0;
      bool ok = true;
      const int ps = 1 << a.c.ps_log2;
      const int boxes = ps < 128 ? 128 / ps : 1;
      const int box_tok = ps < 128 ? ps : 128;
      // One 128-key tile: a lane issues one box (64 columns of the tokens of one page); one
      // lane after the other took 185 clocks a box and held 16-token pages to half the rate.
      const int my_box = lane / C::kBoxes, my_half = lane % C::kBoxes;
      auto load_tile = [&](int page, const Job& j, int tile, const CUtensorMap* tm, uint8_t* dst, uint64_t* bar) {
        if (lane == 0) mbar_arrive_expect_tx(bar, C::kTile);
        __syncwarp();
        if (my_box < boxes) {
          const int slot = (128 * tile + my_box * box_tok) & (ps - 1);
          tma_load_4d(dst + my_half * 16384 + my_box * box_tok * 128, tm, bar, 64 * my_half,
                      a.layout == 0 ? j.kv : slot, a.layout == 0 ? slot : j.kv, page);
        }
        __syncwarp();
      };
      // The page of this lane's box of a tile; one past the pool (the map's fill: zeros) if it
      // lies behind the sequence or the entry is none.
      auto page_of = [&](PageWindow& w, int tile) {
        const int i = (128 * tile) >> a.c.ps_log2;
        const int page = w.get(i, my_box, lane);
        if (page >= 0 && page < a.c.num_pages) return page;
        if (my_box < boxes && i + my_box < w.end) set_device_status(a.status, DEV_BAD_INDEX);
        return static_cast<int>(a.c.num_pages);
      };
      // the next item's jobs and first pages are loaded while this one's tiles are
      Streams next = load_streams<kWide>(a, blockIdx.x, n_jobs, qt, g);
      PageWindow next_w[2];
      auto start_windows = [&]() {
        if (next.n[0] > 0) next_w[0].start(a.c, next.j[0], lane);
        if (!kWide && next.n[1] > 0) next_w[1].start(a.c, next.j[1], lane);
      };
      start_windows();
      for (int it = blockIdx.x; it < n_items && ok; it += gridDim.x) {
        const Streams s = next;
        PageWindow w[2] = {next_w[0], next_w[1]};
        next = load_streams<kWide>(a, it + static_cast<int>(gridDim.x), n_jobs, qt, g);
        start_windows();
        const int most = s.n[0] > s.n[1] ? s.n[0] : s.n[1];
        if (most == 0) continue;
        bool q_sent = false;
        for (int j = 0; j < most && ok; ++j) {
#pragma unroll
          for (int q = 0; q < (kWide ? 1 : 2); ++q) {
            if (!ok || j >= s.n[q]) continue;
            const uint32_t ks = kit % C::kN;
            if (kit >= static_cast<uint32_t>(C::kN))
              ok = __all_sync(0xffffffffu, mbar_wait(&bars[C::kBarKEmpty + ks], ((kit / C::kN) - 1) & 1u, a.status, vabort));
            if (!ok) break;
            const int page = page_of(w[q], s.j[q].tile0 + j);
            load_tile(page, s.j[q], s.j[q].tile0 + j, &tm_k, smem + C::kOffK + ks * C::kTile, &bars[C::kBarKFull + ks]);
            ++kit;
            if (!q_sent) {
              // Q goes behind the first K tile: its buffer is free once the last item's scores are done
              q_sent = true;
              if (uc > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars[C::kBarQEmpty], (uc - 1) & 1u, a.status, vabort));
              if (!ok) break;
              ++uc;
              const int nq = (s.n[0] > 0 ? 1 : 0) + (s.n[1] > 0 ? 1 : 0);
              if (lane == 0) mbar_arrive_expect_tx(&bars[C::kBarQFull], static_cast<uint32_t>(nq * C::kBoxes * 128 * g * qt));
              __syncwarp();
              if (lane < 2 * C::kBoxes) {
                const int qq = lane / C::kBoxes, b = lane % C::kBoxes;
                if ((qq ? s.n[1] : s.n[0]) > 0)
                  tma_load_3d(smem + qq * C::kQTile + b * C::kQBox, &tm_q, &bars[C::kBarQFull], 64 * b,
                              (qq ? s.j[1].kv : s.j[0].kv) * g, qq ? s.j[1].t0 : s.j[0].t0);
              }
            }
            const uint32_t vs = vit % C::kN;
            if (vit >= static_cast<uint32_t>(C::kN))
              ok = __all_sync(0xffffffffu, mbar_wait(&bars[C::kBarVEmpty + vs], ((vit / C::kN) - 1) & 1u, a.status, vabort));
            if (!ok) break;
            load_tile(page, s.j[q], s.j[q].tile0 + j, &tm_v, smem + C::kOffV + vs * C::kTile, &bars[C::kBarVFull + vs]);
            ++vit;
          }
        }
      }
      if (!ok) *vabort = 1;
      // This warp's own copies still in flight land before the CTA may exit: also where all are
      // sent, since another warp may give up while the last are on their way.
#pragma unroll 1
      for (uint32_t i = kit > static_cast<uint32_t>(C::kN) ? kit - C::kN : 0u; i < kit; ++i)
        mbar_wait_ns(&bars[C::kBarKFull + i % C::kN], (i / C::kN) & 1u, 200000000ull);
#pragma unroll 1
      for (uint32_t i = vit > static_cast<uint32_t>(C::kN) ? vit - C::kN : 0u; i < vit; ++i)
        mbar_wait_ns(&bars[C::kBarVFull + i % C::kN], (i / C::kN) & 1u, 200000000ull);
      if (uc > 0) mbar_wait_ns(&bars[C::kBarQFull], (uc - 1) & 1u, 200000000ull);
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer (converged warp)
      constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
      constexpr uint32_t kIdPV = idesc_bf16(128, D, false, true);
      const uint64_t dQ0 = smem_desc(smem_u32(smem), 16, 1024);
      const uint64_t dK0 = smem_desc(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t dV0 = smem_desc(smem_u32(smem + C::kOffV), 16384, 1024);
      uint32_t kit = 0, vit = 0, uc = 0;
      uint32_t pph = 0u;               // bit q: parity of the next p_full waits of stream q
      uint32_t uq[2] = {0u, 0u};       // jobs done per stream
      bool ok = true;
      auto wait = [&](int bar, uint32_t parity) {
        return mbar_wait_warp<20u>(&bars[bar], parity, a.status, vabort);
      };
      auto issue_s = [&](int q, uint32_t kstage) {
        const uint64_t qa = dQ0 + static_cast<uint64_t>((q * C::kQTile) >> 4);
        const uint64_t ka = dK0 + static_cast<uint64_t>((kstage * C::kTile) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t qo = static_cast<uint64_t>(((kk >> 2) * C::kQBox + (kk & 3) * 32) >> 4);
          const uint64_t ko = static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
          mma_bf16_ss_w(tmem + C::col_s(q), qa + qo, ka + ko, kIdS, kk > 0 ? 1u : 0u);
        }
      };
      auto issue_pv = [&](int q, uint32_t vstage, int h, bool acc) {
        const uint64_t va = dV0 + static_cast<uint64_t>((vstage * C::kTile) >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kk = 4 * h + i;
          mma_bf16_ts_w(tmem + C::col_o(q), tmem + C::col_s(q) + kk * 8,
                        va + static_cast<uint64_t>((kk * 2048) >> 4), kIdPV, (acc || i > 0) ? 1u : 0u);
        }
      };
      // Clear the V rows from `from` on (behind the sequence's end; whatever they hold must not
      // meet a probability of zero).
      auto clear_v = [&](uint32_t vstage, int from) {
        uint8_t* v = smem + C::kOffV + vstage * C::kTile;
        for (int i = lane; i < (128 - from) * 8; i += 32)
#pragma unroll
          for (int b = 0; b < C::kBoxes; ++b)
            *reinterpret_cast<uint4*>(v + b * 16384 + from * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
      };
      Runs next = load_runs<kWide>(a, blockIdx.x, n_jobs, qt);
      for (int it = blockIdx.x; it < n_items && ok; it += gridDim.x) {
        const Runs s = next;
        next = load_runs<kWide>(a, it + static_cast<int>(gridDim.x), n_jobs, qt);
        const int most = s.n[0] > s.n[1] ? s.n[0] : s.n[1];
        if (most == 0) continue;
        ok = wait(C::kBarQFull, uc & 1u);
        if (!ok) break;
        tc_fence_after();
        // Q is free for the next item once the last scores are taken
        int scores = s.n[0] + s.n[1];
        // first scores
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (!ok || s.n[q] == 0) continue;
          const uint32_t ks = kit % C::kN;
          if (!kWide || q == 0) {
            ok = wait(C::kBarKFull + ks, (kit / C::kN) & 1u);
            if (!ok) break;
            tc_fence_after();
          }
          issue_s(q, ks);
          mma_commit_w(&bars[C::kBarSFull + q]);
          if (--scores == 0) mma_commit_w(&bars[C::kBarQEmpty]);
          if (!kWide || q == 1 || s.n[1] == 0) {
            mma_commit_w(&bars[C::kBarKEmpty + ks]);
            ++kit;
          }
        }
        for (int j = 0; j < most && ok; ++j) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (!ok || j >= s.n[q]) continue;
            const uint32_t vs = vit % C::kN;
            if (!kWide || q == 0) {
              ok = wait(C::kBarVFull + vs, (vit / C::kN) & 1u);
              if (!ok) break;
              const int left = s.keys[q] - 128 * j;
              if (left < 128) clear_v(vs, left < 0 ? 0 : left);
            }
            ok = wait(C::kBarPFull + 2 * q, (pph >> q) & 1u);
            if (!ok) break;
            if (j == 0 && uq[q] > 0) {
              ok = wait(C::kBarOFree + q, (uq[q] - 1) & 1u);
              if (!ok) break;
            }
            tc_fence_after();
            issue_pv(q, vs, 0, j > 0);
            ok = wait(C::kBarPFull + 2 * q + 1, (pph >> q) & 1u);
            if (!ok) break;
            pph ^= 1u << q;
            tc_fence_after();
            issue_pv(q, vs, 1, true);
            if (j + 1 == s.n[q]) mma_commit_w(&bars[C::kBarODone + q]);
            if (!kWide || q == 1 || s.n[1] == 0) {
              mma_commit_w(&bars[C::kBarVEmpty + vs]);
              ++vit;
            }
            if (j + 1 < s.n[q]) {
              const uint32_t ks = kit % C::kN;
              if (!kWide || q == 0) {
                ok = wait(C::kBarKFull + ks, (kit / C::kN) & 1u);
                if (!ok) break;
                tc_fence_after();
              }
              issue_s(q, ks);
              mma_commit_w(&bars[C::kBarSFull + q]);
              if (--scores == 0) mma_commit_w(&bars[C::kBarQEmpty]);
              if (!kWide || q == 1 || s.n[1] == 0) {
                mma_commit_w(&bars[C::kBarKEmpty + ks]);
                ++kit;
              }
            }
          }
        }
        if (!ok) break;
        if (s.n[0] > 0) ++uq[0];
        if (s.n[1] > 0) ++uq[1];
        ++uc;
      }
      if (!ok) *vabort = 1;
      // every MMA (and the arrivals committed behind it) has landed before exit
      mma_commit_w(&bars[C::kBarDrain]);
      mbar_wait_ns(&bars[C::kBarDrain], 0u, ok ? 4000000000ull : 200000000ull);
    }
  } else {
    setreg_inc<kRegsSoftmax>();
    if (kWide || (warp & 3) < kNarrowRows / 32) {
      // ------------------------------------------------------------ softmax of stream q
      const int q = (warp - 4) >> 2;
      const int quarter = warp & 3;
      const int row = quarter * 32 + lane;
      const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      const uint32_t colS = C::col_s(q), colO = C::col_o(q);
      const float c2 = a.scale * kLog2e;
      const int tok = row / g;
      uint32_t sph = 0u, uq = 0u;
      bool ok = true;
      for (int it = blockIdx.x; it < n_items && ok; it += gridDim.x) {
        const Job w = load_stream<kWide>(a, it, q, n_jobs, qt, g);
        const int n = w.n_tiles;
        if (n == 0) continue;
        const bool valid = tok < w.n_tok && row < g * qt;
        const bool any = __any_sync(0xffffffffu, valid);
        const int t = w.t0 + tok;
        // rows that are not used need no mask: what they hold reaches no other row
        int limit = INT_MAX;
        if (valid) limit = w.lim == INT_MIN ? __ldcg(a.lims + t) : w.lim + t;
        limit -= 128 * w.tile0;
        float m_run = -INFINITY, l = 0.0f;
        for (int j = 0; j < n; ++j) {
          ok = mbar_wait_hint<20u>(&bars[C::kBarSFull + q], sph, a.status, vabort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          sph ^= 1u;
          if (!any) {               // no row of this warp is used: what it leaves in P reaches none
            tc_fence_after();
            tc_fence_before();
            mbar_arrive(&bars[C::kBarPFull + 2 * q]);
            mbar_arrive(&bars[C::kBarPFull + 2 * q + 1]);
            continue;
          }
          tc_fence_after();
          uint32_t sv[4][32];
          tmem_ld32(lane_base + colS + 0, sv[0]);
          tmem_ld32(lane_base + colS + 32, sv[1]);
          tmem_ld32(lane_base + colS + 64, sv[2]);
          tmem_ld32(lane_base + colS + 96, sv[3]);
          tmem_ld_wait();
          const int lim = limit - 128 * j;
          if (lim < 128) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c >= lim) sv[c >> 5][c & 31] = __float_as_uint(-INFINITY);
          }
          float mxa = -INFINITY, mxb = -INFINITY, mxc = -INFINITY, mxd = -INFINITY;
#pragma unroll
          for (int c = 0; c < 128; c += 8) {
            mxa = fmax3(mxa, __uint_as_float(sv[c >> 5][c & 31]), __uint_as_float(sv[c >> 5][(c + 1) & 31]));
            mxb = fmax3(mxb, __uint_as_float(sv[c >> 5][(c + 2) & 31]), __uint_as_float(sv[c >> 5][(c + 3) & 31]));
            mxc = fmax3(mxc, __uint_as_float(sv[c >> 5][(c + 4) & 31]), __uint_as_float(sv[c >> 5][(c + 5) & 31]));
            mxd = fmax3(mxd, __uint_as_float(sv[c >> 5][(c + 6) & 31]), __uint_as_float(sv[c >> 5][(c + 7) & 31]));
          }
          const float mt = fmax3(mxa, mxb, fmaxf(mxc, mxd)) * c2;
          float factor = 1.0f;
          bool resc = false;
          if (m_run == -INFINITY) {
            m_run = mt;
          } else if (mt > m_run + kRescaleLog2) {
            factor = ex2_approx(m_run - mt);
            l *= factor;
            m_run = mt;
            resc = true;
          }
          const float neg_m = (m_run == -INFINITY) ? 0.0f : -m_run;
          const bool any_resc = __any_sync(0xffffffffu, resc);
          const uint64_t c2x2 = f2_pack(c2, c2), nm2 = f2_pack(neg_m, neg_m);
          uint64_t rs2[4] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f),
                             f2_pack(0.0f, 0.0f)};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pw[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int c = half * 64 + 2 * i;
              const uint64_t e = f2_fma(f2_pack(__uint_as_float(sv[c >> 5][c & 31]),
                                                __uint_as_float(sv[(c + 1) >> 5][(c + 1) & 31])),
                                        c2x2, nm2);
              float x0, x1;
              f2_unpack(e, x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              rs2[i & 3] = f2_add(rs2[i & 3], f2_pack(p0, p1));
              pw[i] = pack_bf16x2(p0, p1);
            }
            tmem_st32(lane_base + colS + half * 32, pw);
            if (!any_resc) {
              tmem_st_wait();
              tc_fence_before();
              mbar_arrive(&bars[C::kBarPFull + 2 * q + half]);
            }
          }
          float r0, r1, r2, r3;
          f2_unpack(f2_add(rs2[0], rs2[1]), r0, r1);
          f2_unpack(f2_add(rs2[2], rs2[3]), r2, r3);
          l += (r0 + r1) + (r2 + r3);
          if (any_resc) {
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t ov[32];
              tmem_ld32(lane_base + colO + cc * 32, ov);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * factor);
              tmem_st32(lane_base + colO + cc * 32, ov);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bars[C::kBarPFull + 2 * q]);
            mbar_arrive(&bars[C::kBarPFull + 2 * q + 1]);
          }
        }
        if (!ok) break;
        ok = mbar_wait_hint<20u>(&bars[C::kBarODone + q], uq & 1u, a.status, vabort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int hh = row - tok * g;
        // (only a sum of zero is of no key; a NaN one is of a NaN score, and stays)
        const float inv_l = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t out = static_cast<int64_t>(t) * a.c.Hq + w.kv * g + hh;
        const int64_t prow = static_cast<int64_t>(w.part) + row;
#pragma unroll
        for (int cc = 0; cc < D / 64; ++cc) {
          uint32_t ov[2][32];
          tmem_ld32(lane_base + colO + cc * 64, ov[0]);
          tmem_ld32(lane_base + colO + cc * 64 + 32, ov[1]);
          tmem_ld_wait();
          if (cc + 1 == D / 64) {       // the next job's products may go to TMEM during the stores
            tc_fence_before();
            mbar_arrive(&bars[C::kBarOFree + q]);
          }
          if (!valid) continue;
          if (w.part < 0) {
            uint16_t* dst = a.o + out * D + cc * 64;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t p[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                p[e] = pack_bf16x2(__uint_as_float(ov[i >> 1][16 * (i & 1) + 2 * e]) * inv_l,
                                   __uint_as_float(ov[i >> 1][16 * (i & 1) + 2 * e + 1]) * inv_l);
              if (a.o_whole) {
                st_global_v8(dst + 16 * i, p);
              } else {
                reinterpret_cast<uint4*>(dst + 16 * i)[0] = make_uint4(p[0], p[1], p[2], p[3]);
                reinterpret_cast<uint4*>(dst + 16 * i)[1] = make_uint4(p[4], p[5], p[6], p[7]);
              }
            }
          } else {
            float* dst = a.part_o + prow * D + cc * 64;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(__uint_as_float(ov[i >> 2][8 * (i & 3) + e]) * inv_l);
              st_global_v8(dst + 8 * i, v);
            }
          }
        }
        if (valid) {
          const float lse2 = l == 0.0f ? -INFINITY : m_run + __log2f(l);
          if (w.part < 0)
            a.lse[out] = lse2 * kLn2;
          else
            a.part_lse[prow] = lse2;
        }
        ++uq;
      }
      if (!ok) *vabort = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// --------------------------------------------------------------------------------------
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

struct JoinArgs {
  int S, group, Hq, Hkv;
  int64_t T;
  const int32_t* cu;
  const Info* info;
  const Seg* segs;
  const float* part_o;
  const float* part_lse;
  uint16_t* o;
  float* lse;
};

// kPer warps join one (token, head) row: 1 with many rows, all of the block's with few rows of many
// parts.  32 parts at a time: a lane loads one part's log-sum-exp, the warp sets the weights
// (every warp of the row the same), then adds every kPer-th part's row, loads independent.
template <int D, int kPer>
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const __grid_constant__ JoinArgs a) {
  constexpr int kV = D / 32;          // values of a lane
  __shared__ float so[kPer > 1 ? kJoinWarps : 1][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = a.Hq / a.Hkv;
  const int64_t out = (static_cast<int64_t>(blockIdx.x) * kJoinWarps + warp) / kPer;
  const int t = static_cast<int>(out / a.Hq), h = static_cast<int>(out - static_cast<int64_t>(t) * a.Hq);
  // the entry of token t: the last one that starts at or before it and is not empty (the offsets
  // are the caller's: found while the kernel before drains)
  int lo = 0, hi = t < a.T ? a.S : 0; // entries [0, lo) end at or before t, [hi, S) do not
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid + 1] <= t) lo = mid + 1; else hi = mid;
  }
  const int b = lo;
  const bool mine = t < a.T && b < a.S && t >= a.cu[b];
  pdl_wait();
  if (!mine) return;                  // (with kPer > 1 for the whole block)
  // the row's part lists: its own segment's, and its group's
  const int grouped = a.info->grouped;
  const int kv = h / g, hh = h - kv * g;
  int n[2] = {0, 0};
  int64_t first[2] = {0, 0}, step[2] = {0, 0};
  bool direct = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k == 1 && !grouped) continue;
    const Seg s = a.segs[k == 0 ? b : a.S + b / a.group];
    if (s.tiles == 0) continue;
    int tiles = s.tiles;
    if (is_wide(s, g)) {      // the keys of the token's pair of Q tiles
      const int per = 2 * qt_of(g, true);
      int end = s.t0 + ((t - s.t0) / per + 1) * per;
      if (end > s.t0 + s.n_tok) end = s.t0 + s.n_tok;
      tiles = tiles_of(s, end);
    }
    n[k] = (tiles + s.chunk - 1) / s.chunk;
    step[k] = static_cast<int64_t>(s.n_tok) * g;
    first[k] = s.part + static_cast<int64_t>(kv) * s.chunks * step[k] + static_cast<int64_t>(t - s.t0) * g + hh;
    if (s.part < 0) direct = n[k] > 0;
  }
  if (direct) return;
  const int total = n[0] + n[1];
  float m = -INFINITY, l = 0.0f, acc[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = 0.0f;
  for (int p0 = 0; p0 < total; p0 += 32) {
    const int p = p0 + lane;
    const int64_t row = p < n[0] ? first[0] + p * step[0] : first[1] + (p - n[0]) * step[1];
    const float x = p < total ? __ldcg(a.part_lse + row) : -INFINITY;
    float mx = x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    // (the maximum drops a NaN part, its weight does not)
    if (mx == -INFINITY && !__any_sync(0xffffffffu, x != x)) continue;
    const float mn = fmaxf(m, mx);
    const float f = ex2_approx(m - mn);
    const float w = ex2_approx(x - mn);
    float ws = w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, off);
    m = mn;
    l = l * f + ws;
#pragma unroll
    for (int i = 0; i < kV; ++i) acc[i] *= f;
    const int cnt = total - p0 < 32 ? total - p0 : 32;
#pragma unroll 4
    for (int k = warp % kPer; k < cnt; k += kPer) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const float* src = a.part_o + __shfl_sync(0xffffffffu, row, k) * D + lane * kV;
      if constexpr (kV == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
        acc[0] = fmaf(wk, v.x, acc[0]);
        acc[1] = fmaf(wk, v.y, acc[1]);
        acc[2] = fmaf(wk, v.z, acc[2]);
        acc[3] = fmaf(wk, v.w, acc[3]);
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
        acc[0] = fmaf(wk, v.x, acc[0]);
        acc[1] = fmaf(wk, v.y, acc[1]);
      }
    }
  }
  if constexpr (kPer > 1) {
#pragma unroll
    for (int i = 0; i < kV; ++i) so[warp][lane * kV + i] = acc[i];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < kPer; ++w)
#pragma unroll
      for (int i = 0; i < kV; ++i) acc[i] += so[w][lane * kV + i];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + out * D) + lane * (kV / 2);
#pragma unroll
  for (int i = 0; i < kV / 2; ++i) dst[i] = pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  if (lane == 0) a.lse[out] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
}

template <int D, bool kWide>
cudaError_t launch_attn(const CacheAttnArgs& a, const AttnArgs& p, cudaStream_t s) {
  using C = Cfg<D, kWide>;
  static bool attr_set[kMaxDeviceCache] = {};
  const int dev = cached_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<D, kWide>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    // the register split is of what the launch gives
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, cache_attn_kernel<D, kWide>);
    if (e != cudaSuccess) return e;
    if (f.numRegs < kRegsLaunch) return cudaErrorLaunchOutOfResources;
    attr_set[dev] = true;
  }
  return launch_after(cache_attn_kernel<D, kWide>, dim3(static_cast<unsigned>(num_sms())), kThreads,
                      C::kSmem, s, *a.tm_k, *a.tm_v, kWide ? a.tm_q : a.tm_qn, p);
}

constexpr int kPlanSeg = sizeof(Seg) + 2 * sizeof(int);   // shared memory of a segment

}  // namespace

CacheAttnLayout cache_attn_layout(const CacheView& c, int S, int64_t T) {
  CacheAttnLayout l{};
  const int g = c.Hq / c.Hkv;
  const int64_t sms = num_sms();
  // Partial rows: a token in two segments (groups) a few times over, and twelve chunks of a
  // narrow job, eight of a wide one, a SM.
  const int64_t tok = T < kMaxSeqs ? T : kMaxSeqs;
  const bool wide = T > kNarrowRows / g;
  l.rows_narrow = 3 * tok * c.Hq + sms * 12 * (T * g < kNarrowRows ? T * g : kNarrowRows);
  l.rows_wide = wide ? 3 * tok * c.Hq + sms * 8 * 256 : 0;
  // jobs: one a (segment, key head) at least, and the chunks
  const int64_t segs = S + S / 2;
  l.max_narrow = segs * c.Hkv + 2 * 16 * sms;
  // (every token is in one segment or two, each with a last pair of Q tiles that is not full)
  l.max_wide = wide ? (T / (128 / g) + 2 * segs) * c.Hkv + 16 * sms : 0;
  auto put = [&](size_t* at, size_t bytes) {
    *at = l.total;
    l.total += (bytes + 255) / 256 * 256;
  };
  put(&l.info, sizeof(Info));
  put(&l.segs, sizeof(Seg) * static_cast<size_t>(segs));
  put(&l.lims, sizeof(int) * static_cast<size_t>(T));
  put(&l.narrow, sizeof(Job) * static_cast<size_t>(l.max_narrow));
  put(&l.wide, sizeof(Job) * static_cast<size_t>(l.max_wide));
  put(&l.lse, sizeof(float) * static_cast<size_t>(l.rows_narrow + l.rows_wide));
  put(&l.o, sizeof(float) * static_cast<size_t>(l.rows_narrow + l.rows_wide) * c.D);
  l.total += 256;      // offsets are from the workspace's first 256-byte boundary
  return l;
}

// Whether the bounds allow more than 64 rows in a segment.
bool cache_attn_wide(const CacheView& c, int64_t T, int max_new, int group) {
  const int tokens = kNarrowRows / (c.Hq / c.Hkv);
  return static_cast<int64_t>(max_new) * group > tokens && T > tokens;
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t s) {
  // (the layout has room for the alignment)
  uint8_t* ws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(a.ws) + 255) & ~static_cast<uintptr_t>(255));
  PlanArgs p{};
  p.c = a.c;
  p.S = a.S;
  p.T = a.T;
  p.rows = a.rows;
  p.cu = a.cu;
  p.max_new = a.max_new;
  p.max_len = a.max_len;
  p.group = a.group;
  p.shared = a.shared;
  p.ws = ws;
  p.l = cache_attn_layout(a.c, a.S, a.T);
  p.sms = num_sms();
  p.status = a.status;
  static bool attr_set[kMaxDeviceCache] = {};
  const int dev = cached_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (kMaxSeqs + kMaxSeqs / 2) * kPlanSeg);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int segs = a.S + (a.group > 1 ? a.S / a.group : 0);
  cache_plan_kernel<<<1, kPlanThreads, static_cast<size_t>(segs) * kPlanSeg, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  const Info* info = reinterpret_cast<const Info*>(ws + p.l.info);
  AttnArgs k{};
  k.c = a.c;
  k.scale = a.scale;
  k.layout = a.layout;
  k.lims = reinterpret_cast<const int*>(ws + p.l.lims);
  k.part_lse = reinterpret_cast<float*>(ws + p.l.lse);
  k.part_o = reinterpret_cast<float*>(ws + p.l.o);
  k.o = a.o;
  k.o_whole = reinterpret_cast<uintptr_t>(a.o) % 32 == 0;
  k.lse = a.lse;
  k.status = a.status;
  k.jobs = reinterpret_cast<const Job*>(ws + p.l.narrow);
  k.n_jobs = info->n_jobs;
  e = a.c.D == 128 ? launch_attn<128, false>(a, k, s) : launch_attn<64, false>(a, k, s);
  if (e != cudaSuccess) return e;
  if (a.wide) {
    k.jobs = reinterpret_cast<const Job*>(ws + p.l.wide);
    k.n_jobs = info->n_jobs + 1;
    e = a.c.D == 128 ? launch_attn<128, true>(a, k, s) : launch_attn<64, true>(a, k, s);
    if (e != cudaSuccess) return e;
  }
  JoinArgs j{};
  j.S = a.S;
  j.group = a.group;
  j.Hq = a.c.Hq;
  j.Hkv = a.c.Hkv;
  j.cu = a.cu;
  j.info = info;
  j.segs = reinterpret_cast<const Seg*>(ws + p.l.segs);
  j.part_o = k.part_o;
  j.part_lse = k.part_lse;
  j.o = a.o;
  j.lse = a.lse;
  // few rows have many parts each: a block a row; else a warp a row (2,048 rows of a group of 8 over
  // 34,000 keys 48.1 against 49.3 us for the call; 3,200 rows of 20 sequences 96.1 against 93.7)
  j.T = a.T;
  const int64_t rows = a.T * a.c.Hq;
  if (rows <= 16 * num_sms()) {
    const dim3 grid(static_cast<unsigned>(rows));
    return a.c.D == 128 ? launch_after(cache_join_kernel<128, kJoinWarps>, grid, kJoinThreads, 0, s, j)
                        : launch_after(cache_join_kernel<64, kJoinWarps>, grid, kJoinThreads, 0, s, j);
  }
  const dim3 grid(static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps));
  return a.c.D == 128 ? launch_after(cache_join_kernel<128, 1>, grid, kJoinThreads, 0, s, j)
                      : launch_after(cache_join_kernel<64, 1>, grid, kJoinThreads, 0, s, j);
}

}  // namespace ls
