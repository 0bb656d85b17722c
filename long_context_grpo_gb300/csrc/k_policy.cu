// Clipped policy loss with a KL term over packed tokens, forward and backward.
//
//   p = softmax(x), logp = log p_y, d = logp - old, rho = e^d,
//   term = w (beta kl - min(rho A, clip(rho) A)),  g = d term / d logp,
//   dlogits = g (onehot_y - p)
//
// Rows are read from HBM once and gradients written once (4 bytes a logit; bound by HBM).
//
// policy_warp<n>: V <= 256 n.  A warp a row, the row in registers: no block-wide step at all.
// policy_cluster: larger rows stay in shared memory between the two passes.  A cluster of 1, 2, 4
//   or 8 CTAs owns one row at a time, each a slice of at most 76 KB, in three or four buffers: one
//   row (or two) waits for its gradient while its sums are exchanged, the next row's sums are taken,
//   and the last arrives by bulk copy.  The exchange takes about 4 us whatever the slice, so the fewest
//   CTAs a row are the fastest (slices of 76 KB against 38 KB with two CTAs an SM:
//   4,096 x 151,936 388 against 457 us), and two rows' exchanges overlap (5,341 x 50,256 184
//   against 260 us).
//   4 or 8 streaming warps: the sum of exp(x - m) in fp32, m the maximum of a thread's first eight
//     logits (the true one if that overflows), joined across lanes in fp32 pairs; later p g
//     rounded to bf16 and stored.  One exponential a logit and pass.
//   2 scalar warps, every other row each: join the partials, exchange them with the other CTAs (distributed
//     shared memory, remote mbarrier arrivals, bounded waits), join those in rank order and decide
//     the clip.  They also own the up to 7 + 7 logits of a row outside its 16-byte granules.
//   1 copy warp: requests a row's slice as soon as a buffer is free.
//   A row whose gradient has another alignment than its logits goes through shared memory once
//   more and is shifted there.
// policy_rows: one CTA a row from global memory, for vocabularies beyond eight slices (304,000).
// policy_finish: a thread a token: its outputs and its loss term in fp64 (an fp64 instruction of one
//   lane costs as much as one of 32 tokens), and their sum in a fixed order, rounded once.
#include <atomic>
#include <type_traits>

#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"

namespace ls {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float bf16_bits(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ float bf16_at(const uint16_t* x, int64_t i) {
  return bf16_bits(__ldcg(reinterpret_cast<const unsigned short*>(x) + i));
}
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint16_t to_bf16(float x) {
  return static_cast<uint16_t>(pack_bf16x2(x, 0.0f) & 0xFFFFu);
}

// The inputs of one token, its outcome.
struct Token {
  int y;
  float old, ref, A, w;
  // (derived where they are needed, so that a token loaded ahead is not waited for)
  __device__ __forceinline__ bool bad(int64_t V) const { return w != 0.0f && (y < 0 || y >= V); }
  __device__ __forceinline__ bool used(int64_t V) const { return w != 0.0f && y >= 0 && y < V; }
};
__device__ __forceinline__ Token load_token(const PolicyArgs& a, int64_t row) {
  Token t;
  t.w = a.weight[row];
  t.y = a.ids[row];
  t.old = a.old[row];
  t.ref = a.ref != nullptr ? a.ref[row] : 0.0f;
  t.A = a.adv[row];
  return t;
}

// Unevaluated sums of two fp32 values, about 48 bits: an fp64 instruction holds its pipe for
// tens of cycles here, and a dozen of them in a row's critical path cost more than all the rest.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = a + b, bb = s - a;
  return {s, (a - (s - bb)) + (b - bb)};
}
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return {s.hi, s.lo + (a.lo + b.lo)};
}
// log(s), s >= 0: the exponent apart, so that the fp32 logarithm sees [1/2, 1) (absolute error
// below 2^-24); exponent x log 2 is exact in its upper part (16 bits of log 2).
__device__ __forceinline__ Pair log_pair(Pair s) {
  constexpr float kLn2Hi = 0.693145751953125f, kLn2Lo = 1.4286068203094172e-06f;
  int e = 0;
  const float f = frexpf(s.hi, &e);
  const float rest = logf(f) + s.lo / s.hi;
  const float k = static_cast<float>(e);
  Pair r = two_sum(k * kLn2Hi, rest);
  r.lo = fmaf(k, kLn2Lo, r.lo);
  return r;
}
// The sum of two log-probabilities, which may be infinite: an infinite sum has no rounding error
// (its parts' differences are infinity - infinity: a sampled token whose logit is -inf, or an
// infinite logp_old, would turn into NaN).
__device__ __forceinline__ Pair log_add(Pair a, Pair b) {
  Pair s = pair_add(a, b);
  if (fabsf(s.hi) == INFINITY) s.lo = 0.0f;
  return s;
}
// Whether a > b.
__device__ __forceinline__ bool above(Pair a, Pair b) {
  const Pair d = log_add(a, {-b.hi, -b.lo});
  return d.hi + d.lo > 0.0f;
}

struct TokenLoss {
  float g;           // d term / d logp
  bool clipped;
};
// The clip is decided on the pair d; ratio and gradient follow in fp32 (relative error ~2^-22).
__device__ __forceinline__ TokenLoss token_grad(const PolicyArgs& a, const Token& t, Pair logp) {
  TokenLoss o;
  const Pair d = log_add(logp, {-t.old, 0.0f});
  o.clipped = (t.A > 0.0f && above(d, {a.log_hi[0], a.log_hi[1]})) || (t.A < 0.0f && above({a.log_lo[0], a.log_lo[1]}, d));
  float slope = 0.0f;
  if (a.ref != nullptr) {
    const Pair r = log_add(logp, {-t.ref, 0.0f});
    slope = a.kl == 1 ? 1.0f : (a.kl == 2 ? r.hi + r.lo : -expm1f(-(r.hi + r.lo)));
  }
  o.g = t.w * (static_cast<float>(a.beta) * slope - (o.clipped ? 0.0f : expf(d.hi + d.lo) * t.A));
  return o;
}
// What the row kernels leave for policy_finish.
__device__ __forceinline__ void leave_logp(const PolicyArgs& a, int64_t row, Pair logp) {
  a.logp_pair[row] = make_float2(logp.hi, logp.lo);
}
__device__ __forceinline__ void reset_counter(const PolicyArgs& a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.counter = 0u;
}

// ======================================================================================
// One CTA a row
// ======================================================================================
constexpr int kRowThreads = 512;

__global__ void __launch_bounds__(kRowThreads) policy_rows(const __grid_constant__ PolicyArgs a) {
  __shared__ float sh_m[kRowThreads / 32];
  __shared__ double sh_s[kRowThreads / 32];
  __shared__ float sh_g, sh_ls;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  reset_counter(a);
  pdl_launch_dependents();
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const uint16_t* x = a.logits + row * a.ldx;
    uint16_t* d = a.dlogits + row * a.ldd;
    const Token tok = load_token(a, row);
    if (!tok.used(a.V)) {
      for (int64_t i = tid; i < a.V; i += kRowThreads) d[i] = 0;
      continue;
    }
    float m = -INFINITY;
    for (int64_t i = tid; i < a.V; i += kRowThreads) m = fmaxf(m, bf16_at(x, i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) sh_m[warp] = m;
    __syncthreads();
    m = sh_m[0];
    for (int w = 1; w < kRowThreads / 32; ++w) m = fmaxf(m, sh_m[w]);
    double s = 0.0;
    for (int64_t i = tid; i < a.V; i += kRowThreads)
      s += static_cast<double>(ex2_approx((bf16_at(x, i) - m) * kLog2e));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) sh_s[warp] = s;
    __syncthreads();
    if (warp == 0) {
      s = 0.0;
      for (int w = 0; w < kRowThreads / 32; ++w) s += sh_s[w];
      const float s_hi = static_cast<float>(s);
      const Pair ls = log_pair({s_hi, static_cast<float>(s - static_cast<double>(s_hi))});
      const Pair lp = log_add(two_sum(bf16_at(x, tok.y), -m), {-ls.hi, -ls.lo});
      const TokenLoss o = token_grad(a, tok, lp);
      if (lane == 0) {
        leave_logp(a, row, lp);
        sh_g = o.g;
        sh_ls = ls.hi + ls.lo;
      }
    }
    __syncthreads();
    const float g = sh_g, ls = sh_ls;
    for (int64_t i = tid; i < a.V; i += kRowThreads) {
      const float p = ex2_approx((bf16_at(x, i) - m - ls) * kLog2e);
      d[i] = to_bf16(g * ((i == tok.y ? 1.0f : 0.0f) - p));
    }
    __syncthreads();
  }
}

// ======================================================================================
// A cluster a row, the row in shared memory
// ======================================================================================
// Rows whose log-sum-exp is at most this far from zero fold it into one constant of the gradient's
// exponent: rounded to fp32 (twice) it costs the probability 2^-14 at most.  Farther ones subtract
// the row's maximum from each logit first, as the sums do, or the rounding would pass bf16's half
// step at 1e5 (4,096 x 151,936: 389 us near zero, 394 with the subtraction).
constexpr float kNear = 512.0f;
constexpr int kMaxCluster = 8;
constexpr int kMaxBufs = 4;                    // slices in shared memory (three or four)
constexpr int kSliceMax = 76000;               // bytes: three slices in one CTA's shared memory
constexpr int kSlice4 = 57000;                 // four
constexpr int kSlice2 = 38000;                 // three, and two such CTAs on an SM
constexpr int kSliceSmall = 26000;             // up to here: 128 streaming threads; four CTAs an SM to
                                               // 18,700 bytes, three to 25,200

// How a row lies in memory: `head` logits before its first 16-byte granule, `nv` whole granules, then
// the tail; granules [g0, g0 + n) are this CTA's.
struct RowSpan {
  int head, tail, nv, g0, n;
};
__device__ __forceinline__ RowSpan row_span(const PolicyArgs& a, int64_t row, int per, int rank) {
  RowSpan s;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits + row * a.ldx);
  s.head = static_cast<int>((16 - (at & 15)) & 15) / 2;
  if (s.head > a.V) s.head = static_cast<int>(a.V);
  s.nv = static_cast<int>(a.V - s.head) >> 3;
  s.tail = static_cast<int>(a.V) - s.head - 8 * s.nv;
  s.g0 = rank * per;
  s.n = s.nv - s.g0;
  s.n = s.n < 0 ? 0 : (s.n > per ? per : s.n);
  return s;
}

// The logit outside the granules that a lane owns, or -1.
__device__ __forceinline__ int64_t edge_index(const RowSpan& s, int64_t V, int lane) {
  if (lane >= 16 && lane - 16 < s.head) return lane - 16;
  if (lane >= 24 && lane - 24 < s.tail) return V - s.tail + lane - 24;
  return -1;
}

// Over the lanes that differ in the bits below kLanes: the maximum of m, and the sum of the parts
// s relative to it (each given relative to its own m; m a logit, not scaled).  -INF with 0
// is an empty part.
template <int kLanes>
__device__ __forceinline__ void join_lanes(float& m, Pair& s) {
  float M = m;
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float f = m == -INFINITY ? 1.0f : ex2_approx((m - M) * kLog2e);
  s.hi *= f;
  s.lo *= f;
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) {
    const Pair o = {__shfl_xor_sync(0xffffffffu, s.hi, off), __shfl_xor_sync(0xffffffffu, s.lo, off)};
    s = pair_add(s, o);
  }
  m = M;
}

// Named barriers.  With nb buffers the streaming warps take the sums of row r + nb - 2 before they
// wait for the gradient of row r, so at most nb - 1 <= 3 rows' parts are waiting for the scalar
// warps, and as many gradients for the streaming warps.  Row r uses id r modulo 4: an even
// number, so that an id belongs to one of the two scalar warps (of three ids the warp that
// is ahead could take the parts that the other one has not come to yet).  Nothing holds the
// streaming warps back from running ahead of the copy warp but the copies that it issues: row
// r + nb is requested behind its wait for row r, and the rows at the end, which wait for no
// copy, are at most nb: nb <= 4 ids.
enum : uint32_t { kBarParts = 1, kBarG = 5, kBarEmpty = 9, kBarCopy = 13 };
constexpr int kRing = 4;            // rows whose parts and gradients are kept apart

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float granule_max(const uint4& v) {
  const uint32_t m = max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w));
  return fmaxf(lo_bf16(m), hi_bf16(m));
}

// Eight logits from word kFirst (and a half, if odd) of two granules on.
template <int kFirst>
__device__ __forceinline__ void cut_words(const uint32_t (&w)[8], bool odd, uint32_t (&o)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
    o[u] = odd ? __byte_perm(w[kFirst + u], w[kFirst + u + 1], 0x5432) : w[kFirst + u];
}

// n granules of a buffer to a row that does not start on a 16-byte boundary: its whole granules
// are cut from two of the buffer's, its ends written one by one.  Threads tid of threads.
__device__ __forceinline__ void shift_row(uint16_t* d, const uint4* buf, int n, int tid, int threads) {
  if (n == 0) return;
  const int off = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(d) & 15)) & 15) / 2;   // 1 .. 7
  const int nd = n - 1;
  uint4* to = reinterpret_cast<uint4*>(d + off);
  for (int i = tid; i < nd; i += threads) {
    const uint4 p = buf[i], q = buf[i + 1];
    const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
    uint32_t o[4];
    switch (off >> 1) {
      case 0: cut_words<0>(w, off & 1, o); break;
      case 1: cut_words<1>(w, off & 1, o); break;
      case 2: cut_words<2>(w, off & 1, o); break;
      default: cut_words<3>(w, off & 1, o); break;
    }
    to[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  const uint16_t* h = reinterpret_cast<const uint16_t*>(buf);
  if (tid < off) d[tid] = h[tid];
  if (tid < 8 - off) d[off + 8 * nd + tid] = h[off + 8 * nd + tid];
}

// Zeros to n granules of a row that does not start on a 16-byte boundary.
__device__ __forceinline__ void zero_row(uint16_t* d, int n, int tid, int threads) {
  if (n == 0) return;
  const int off = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(d) & 15)) & 15) / 2;   // 1 .. 7
  uint4* to = reinterpret_cast<uint4*>(d + off);
  for (int i = tid; i < n - 1; i += threads) to[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid < off) d[tid] = 0;
  if (tid < 8 - off) d[off + 8 * (n - 1) + tid] = 0;
}

template <int kStream>
__global__ void __launch_bounds__(kStream + 96, kStream == 128 ? 4 : 3)
    policy_cluster(const __grid_constant__ PolicyArgs a, int cl, int per, int nb) {
  constexpr int kWarps = kStream / 32;
  static_assert(kWarps <= 8, "a scalar warp joins the warps' parts over eight lanes");
  constexpr int kThreads = kStream + 32;        // streaming warps and one other
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ __align__(8) uint64_t full[kMaxBufs], xbar[4];
  __shared__ float part[kRing][kWarps][3];         // a warp's maximum and sum (pair)
  __shared__ float slot[4][kMaxCluster][3];    // a CTA's, by rank
  __shared__ __align__(16) float4 sh_turn[kRing];   // g, -base, c, g (1 - p) of a row
  __shared__ int sh_used[kMaxBufs], sh_y[kRing];
  // Set when a bounded wait of this CTA or of a peer gave up: rows are only walked through from
  // then on, barrier by barrier, with gradients of zero, and nothing is copied any more.  Every
  // decision on it is a vote of the warp (its lanes may see it at different times).
  __shared__ int cl_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = cl > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t cid = cl > 1 ? cluster_id_x() : blockIdx.x;
  const int64_t ncl = cl > 1 ? cluster_count_x() : gridDim.x;
  const int slice = per * 16;
  volatile int* vabort = &cl_abort;
  // rows that all lie alike are looked at once
  const bool alike = a.ldx % 8 == 0;

  if (tid == 0) {
    cl_abort = 0;
    for (int i = 0; i < nb; ++i) mbar_init(&full[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&xbar[i], static_cast<uint32_t>(cl));
    fence_mbar_init();
  }
  __syncthreads();
  if (cl > 1) cluster_sync_all();     // peers' barriers are ready before any remote arrival
  reset_counter(a);
  pdl_launch_dependents();

  RowSpan sp = row_span(a, cid, per, rank);
  if (warp == kWarps || warp == kWarps + 1) {
    // ----------------------------------------------------------------- scalar warps
    // Each takes every other row, so that two rows' exchanges overlap (one alone takes 3.7 us a
    // row).  What belongs to the next rows is loaded ahead: a token two rows, its logit and the
    // logits outside the granules (lanes 16-22 the head's, 24-30 the tail's, on rank 0) one.
    const int who = warp - kWarps;
    const int64_t first = cid + who * ncl, step = 2 * ncl;
    struct Ahead {
      Token tok;
      float xy, edge;
    };
    auto token = [&](int64_t row) {
      Token t = {0, 0.0f, 0.0f, 0.0f, 0.0f};
      if (row < a.T) t = load_token(a, row);
      return t;
    };
    auto logits = [&](int64_t row, const Token& t) {
      Ahead r = {t, 0.0f, -INFINITY};
      if (row < a.T && t.used(a.V)) {
        const uint16_t* x = a.logits + row * a.ldx;
        r.xy = bf16_at(x, t.y);
        if (rank == 0) {
          const int64_t e = edge_index(alike ? sp : row_span(a, row, per, rank), a.V, lane);
          if (e >= 0) r.edge = bf16_at(x, e);
        }
      }
      return r;
    };
    Ahead now = logits(first, token(first));
    Token next = token(first + step);
    uint32_t ux = 0;                   // rows exchanged
    int par = who;                     // row modulo kRing
    for (int64_t row = first; row < a.T; row += step, par = (par + 2) % kRing) {
      const Token t = now.tok;
      const float xv = now.xy, ev = now.edge;
      now = logits(row + step, next);
      next = token(row + 2 * step);
      if (!alike) sp = row_span(a, row, per, rank);
      TokenLoss o;
      o.g = 0.0f;
      o.clipped = false;
      Pair logp = {0.0f, 0.0f};
      float base = 0.0f, rest = 0.0f;      // their sum is the row's log-sum-exp
      bool aborted = false;
      named_barrier_sync(kBarParts + par, kThreads);
      if (t.used(a.V)) {
        float m = -INFINITY;
        Pair s = {0.0f, 0.0f};
        if (lane < kWarps) {
          m = part[par][lane][0];
          s = {part[par][lane][1], part[par][lane][2]};
        } else if (lane >= 16) {
          m = ev;                        // a logit outside the granules
          s.hi = ev == -INFINITY ? 0.0f : 1.0f;
        }
        if (rank == 0) join_lanes<32>(m, s); else join_lanes<8>(m, s);
        // (the shuffles also make sure that xv has arrived: the row may be overwritten in place
        // once the partials are out)
        const float x_y = __shfl_sync(0xffffffffu, xv, 0);
        aborted = __any_sync(0xffffffffu, *vabort != 0);
        if (cl > 1 && !aborted) {
          const int sl = 2 * who + (ux & 1);
          if (lane < cl) {
            const uint32_t dst = cluster_map(&slot[sl][rank][0], lane);
            st_cluster_f32(dst, m);
            st_cluster_f32(dst + 4, s.hi);
            st_cluster_f32(dst + 8, s.lo);
            mbar_arrive_remote(cluster_map(&xbar[sl], lane));
          }
          __syncwarp();
          aborted = __any_sync(0xffffffffu, !mbar_wait_limit<true>(&xbar[sl], (ux >> 1) & 1u, a.status, vabort, a.wait_ns));
          if (!aborted) {
            // every CTA joins the same parts the same way
            const bool in = lane < cl;
            m = in ? slot[sl][lane][0] : -INFINITY;
            s = {in ? slot[sl][lane][1] : 0.0f, in ? slot[sl][lane][2] : 0.0f};
            join_lanes<8>(m, s);
            m = __shfl_sync(0xffffffffu, m, 0);
            s = {__shfl_sync(0xffffffffu, s.hi, 0), __shfl_sync(0xffffffffu, s.lo, 0)};
          }
        }
        // the peers' own waits poll their flag
        if (cl > 1 && aborted && lane < cl) st_cluster_u32(cluster_map(&cl_abort, lane), 1u);
        ++ux;
        const Pair ls = log_pair(s);
        logp = log_add(two_sum(x_y, -m), {-ls.hi, -ls.lo});
        rest = m + (ls.hi + ls.lo);
        if (!(fabsf(rest) <= kNear)) {
          base = m;
          rest = ls.hi + ls.lo;
        }
        if (!aborted) o = token_grad(a, t, logp);
      }
      // -g p = -sign(g) 2^((x - base) log2 e - rest log2 e + log2 |g|), base = 0 for rows near zero
      const float c = fmaf(-rest, kLog2e, log2f(fabsf(o.g)));
      const float gy = o.g * (1.0f - ex2_approx((logp.hi + logp.lo) * kLog2e));
      if (lane == 0) {
        sh_turn[par] = make_float4(o.g, -base, c, gy);
        sh_y[par] = t.used(a.V) ? t.y - sp.head : -1;
      }
      __syncwarp();
      named_barrier_arrive(kBarG + par, kThreads);
      if (rank == 0) {
        if (lane == 0 && t.used(a.V)) leave_logp(a, row, logp);
        const int64_t e = edge_index(sp, a.V, lane);
        if (e >= 0) {
          float v = 0.0f;
          if (o.g != 0.0f) v = e == t.y ? gy : copysignf(ex2_approx(fmaf(ev - base, kLog2e, c)), -o.g);
          if (o.g != o.g) v = o.g;
          a.dlogits[row * a.ldd + e] = to_bf16(v);
        }
      }
    }
  } else if (warp == kWarps + 2) {
    // -------------------------------------------------------------------- copy warp
    // Requests a row's slice as soon as a buffer is free.  After an abort nothing more is requested:
    // the buffer's last phase may not be complete, and nobody waits for another one.  (A streaming
    // warp that gave up on a row's phase has set the flag before it let the row's buffer go.)
    int sent = 0;                        // rows requested
    auto request = [&](int64_t row, int b, const Token& t) {
      if (row >= a.T || __any_sync(0xffffffffu, *vabort != 0)) return;
      ++sent;
      const bool used = t.used(a.V);
      const RowSpan rs = alike ? sp : row_span(a, row, per, rank);
      if (lane == 0) {
        sh_used[b] = used ? 1 : 0;
        if (used && rs.n > 0) {
          mbar_arrive_expect_tx(&full[b], static_cast<uint32_t>(rs.n) * 16u);
          bulk_load(dyn + b * slice, a.logits + row * a.ldx + rs.head + 8 * static_cast<int64_t>(rs.g0),
                    static_cast<uint32_t>(rs.n) * 16u, &full[b]);
        } else {
          mbar_arrive(&full[b]);
        }
      }
      __syncwarp();
    };
    auto token = [&](int64_t row) {
      Token t = {0, 0.0f, 0.0f, 0.0f, 0.0f};
      if (row < a.T) t = load_token(a, row);
      return t;
    };
    for (int i = 0; i < nb; ++i) request(cid + i * ncl, i, token(cid + i * ncl));
    Token next = token(cid + nb * ncl);
    int b = 0;
    for (int64_t row = cid; row < a.T; row += ncl, b = b == nb - 1 ? 0 : b + 1) {
      named_barrier_sync(kBarEmpty + b, kThreads);
      request(row + nb * ncl, b, next);
      next = token(row + (nb + 1) * ncl);
    }
    if (*vabort) {
      // copies still in flight land before the CTA may exit: the last request of each buffer
      for (int i = 0; i < nb; ++i)
        if (sent > i) mbar_wait_ns(&full[i], static_cast<uint32_t>((sent - 1 - i) / nb) & 1u, 200000000ull);
    }
  } else {
    // -------------------------------------------------------------- streaming warps
    const uint64_t l2 = f2_pack(kLog2e, kLog2e);
    auto slice_sum = [&](const uint4* buf, int n, int from, float m) {
      const float base = m == -INFINITY ? 0.0f : -m;
      const uint64_t nb = f2_pack(base, base);
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 4
      for (int j = from; j < n; j += kStream) {
        const uint4 v = buf[j];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float e0, e1;
          f2_unpack(f2_mul(f2_add(f2_pack(lo_bf16(w[u]), hi_bf16(w[u])), nb), l2), e0, e1);
          acc[u] = f2_add(acc[u], f2_pack(ex2_approx(e0), ex2_approx(e1)));
        }
      }
      float s0, s1;
      f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), s0, s1);
      return s0 + s1;
    };
    // Sum of exponentials of this CTA's slice of its i-th row.
    int sum_buf = 0, sum_par = 0;      // of the next row to be summed
    uint32_t sum_phase = 0u;
    bool dead = false;                 // this warp has given up on the copies
    auto pass1 = [&](int64_t row) {
      const int bi = sum_buf, par = sum_par;
      const int n = alike ? sp.n : row_span(a, row, per, rank).n;
      const uint4* buf = reinterpret_cast<const uint4*>(dyn + bi * slice);
      if (!dead && !__all_sync(0xffffffffu, mbar_wait_limit<false>(&full[bi], sum_phase, a.status, vabort, a.wait_ns))) {
        dead = true;
        *vabort = 1;
      }
      float m = -INFINITY;
      Pair s = {0.0f, 0.0f};
      if (!dead && sh_used[bi] != 0) {
        // Relative to the maximum of the thread's first granule; if a later logit is so much
        // larger that the sum leaves [0, 2^100), or nothing in it is finite, once more relative
        // to the warp's true maximum.
        m = tid < n ? granule_max(buf[tid]) : -INFINITY;
        float sum = slice_sum(buf, n, tid, m);
        const bool odd = tid < n && (m == -INFINITY || !(sum < 1.2676506e30f));
        if (__any_sync(0xffffffffu, odd)) {
          m = -INFINITY;
          for (int j = tid; j < n; j += kStream) m = fmaxf(m, granule_max(buf[j]));
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
          sum = slice_sum(buf, n, tid, m);
        }
        s.hi = sum;
        join_lanes<32>(m, s);
      }
      if (lane == 0) {
        part[par][warp][0] = m;
        part[par][warp][1] = s.hi;
        part[par][warp][2] = s.lo;
      }
      __syncwarp();
      named_barrier_arrive(kBarParts + par, kThreads);
      sum_par = (par + 1) % kRing;
      sum_buf = bi == nb - 1 ? 0 : bi + 1;
      sum_phase ^= bi == nb - 1 ? 1u : 0u;
    };
    int b = 0, par = 0;
    const int64_t ahead = (nb - 2) * ncl;
    for (int64_t row = cid; row < cid + ahead && row < a.T; row += ncl) pass1(row);
    for (int64_t row = cid; row < a.T; row += ncl, b = b == nb - 1 ? 0 : b + 1, par = (par + 1) % kRing) {
      uint4* buf = reinterpret_cast<uint4*>(dyn + b * slice);
      // later rows' sums while this row's are exchanged
      if (row + ahead < a.T) pass1(row + ahead);
      named_barrier_sync(kBarG + par, kThreads);
      const float4 tn = sh_turn[par];
      const float g = tn.x, nm = tn.y, c = tn.z, gy = tn.w;
      const int y = sh_y[par];
      if (!alike) sp = row_span(a, row, per, rank);
      uint16_t* d = a.dlogits + row * a.ldd + sp.head + 8 * static_cast<int64_t>(sp.g0);
      const bool direct = (reinterpret_cast<uintptr_t>(d) & 15) == 0;
      uint4* d4 = direct ? reinterpret_cast<uint4*>(d) : buf;
      // (a row with g != 0 has its slice in the buffer, whoever gave up on a later one)
      const uint32_t sign = g > 0.0f ? 0x80008000u : 0u;
      const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(nm, nm);
      if (g == 0.0f) {
        if (direct) {
          for (int i = tid; i < sp.n; i += kStream) d4[i] = make_uint4(0u, 0u, 0u, 0u);
        } else {
          zero_row(d, sp.n, tid, kStream);     // (a copy given up on may still be landing in the buffer)
        }
      } else {
        const auto turn = [&](auto far) {
#pragma unroll 4
          for (int i = tid; i < sp.n; i += kStream) {
            const uint4 v = buf[i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              float e0, e1;
              uint64_t x = f2_pack(lo_bf16(w[u]), hi_bf16(w[u]));
              if constexpr (decltype(far)::value) x = f2_add(x, nm2);
              f2_unpack(f2_fma(x, l2, c2), e0, e1);
              o[u] = pack_bf16x2(ex2_approx(e0), ex2_approx(e1)) ^ sign;
            }
            d4[i] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        };
        if (nm == 0.0f)
          turn(std::false_type{});
        else
          turn(std::true_type{});
      }
      // the sampled token's column, by the thread that wrote its granule
      const int yl = y - 8 * sp.g0;
      if (y >= 0 && yl >= 0 && yl < 8 * sp.n && (yl >> 3) % kStream == tid && g != 0.0f)
        reinterpret_cast<uint16_t*>(d4)[yl] = to_bf16(gy);
      if (!direct && sp.n > 0 && g != 0.0f) {
        // the gradient row lies at another offset from a 16-byte boundary: its granules are cut
        // from two of the buffer's
        named_barrier_sync(kBarCopy, kStream);
        shift_row(d, buf, sp.n, tid, kStream);
        // the next copy into this buffer comes behind the writes above
        fence_proxy_async_smem();
      }
      // (a warp that waits for no copies any more would run ahead of the copy warp: it waits for it here)
      if (dead)
        named_barrier_sync(kBarEmpty + b, kThreads);
      else
        named_barrier_arrive(kBarEmpty + b, kThreads);
    }
  }
  __syncwarp();
  __syncthreads();
  if (cl > 1) {
    // a wait that gave up behind the last exchange is known to the whole cluster too
    if (tid < cl && *vabort) st_cluster_u32(cluster_map(&cl_abort, tid), 1u);
    __syncwarp();
    // no CTA leaves while a peer may still write its shared memory; every wait above is bounded
    cluster_sync_all();
  }
  // Which of the cluster's rows are whole is not known then: none of them counts, and the loss is NaN.
  if (rank == 0 && *vabort) {
    const float nan = __int_as_float(0x7fc00000);
    for (int64_t row = cid + tid * ncl; row < a.T; row += (kStream + 96) * ncl) leave_logp(a, row, {nan, nan});
  }
}

// ======================================================================================
// A warp a row, the row in registers
// ======================================================================================
constexpr int kWarpThreads = 256;

// n granules of 16 bytes from registers (granule i in v[i / 32] of lane i % 32) to a row that is
// aligned, or through the warp's shared memory to one that is not.
template <int kG>
__device__ __forceinline__ void store_row(uint16_t* d, const uint4 (&v)[kG], int n, uint4* buf, int lane) {
  if ((reinterpret_cast<uintptr_t>(d) & 15) == 0) {
#pragma unroll
    for (int k = 0; k < kG; ++k)
      if (lane + 32 * k < n) __stcs(reinterpret_cast<uint4*>(d) + lane + 32 * k, v[k]);
    return;
  }
#pragma unroll
  for (int k = 0; k < kG; ++k)
    if (lane + 32 * k < n) buf[lane + 32 * k] = v[k];
  __syncwarp();
  shift_row(d, buf, n, lane, 32);
  __syncwarp();
}

template <int kG>
__global__ void __launch_bounds__(kWarpThreads, kG > 4 ? 2 : 4) policy_warp(const __grid_constant__ PolicyArgs a) {
  extern __shared__ __align__(128) uint8_t dyn[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint4* buf = reinterpret_cast<uint4*>(dyn) + warp * 32 * kG;     // only for unaligned gradients
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kWarpThreads / 32);
  const int64_t first = blockIdx.x * static_cast<int64_t>(kWarpThreads / 32) + warp;
  reset_counter(a);
  pdl_launch_dependents();
  Token next = {0, 0.0f, 0.0f, 0.0f, 0.0f};
  if (first < a.T) next = load_token(a, first);
  const uint64_t l2 = f2_pack(kLog2e, kLog2e);
  for (int64_t row = first; row < a.T; row += stride) {
    const Token t = next;
    if (row + stride < a.T) next = load_token(a, row + stride);
    const RowSpan sp = row_span(a, row, 32 * kG, 0);
    const uint16_t* x = a.logits + row * a.ldx;
    uint16_t* d = a.dlogits + row * a.ldd;
    const int64_t e = edge_index(sp, a.V, lane);
    uint4 v[kG];
    if (!t.used(a.V)) {
#pragma unroll
      for (int k = 0; k < kG; ++k) v[k] = make_uint4(0u, 0u, 0u, 0u);
      store_row(d + sp.head, v, sp.n, buf, lane);
      if (e >= 0) d[e] = 0;
      continue;
    }
    const uint4* x4 = reinterpret_cast<const uint4*>(x + sp.head);
#pragma unroll
    for (int k = 0; k < kG; ++k)
      v[k] = lane + 32 * k < sp.n ? __ldcs(x4 + lane + 32 * k)
                                  : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
    const float xy = bf16_at(x, t.y);
    const float ev = e >= 0 ? bf16_at(x, e) : -INFINITY;
    float m = ev;
#pragma unroll
    for (int k = 0; k < kG; ++k) m = fmaxf(m, granule_max(v[k]));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float base = m == -INFINITY ? 0.0f : -m;
    const uint64_t nb = f2_pack(base, base);
    uint64_t acc[4] = {f2_pack(ex2_approx((ev + base) * kLog2e), 0.0f), 0ull, 0ull, 0ull};
#pragma unroll
    for (int k = 0; k < kG; ++k) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float e0, e1;
        f2_unpack(f2_mul(f2_add(f2_pack(lo_bf16(w[u]), hi_bf16(w[u])), nb), l2), e0, e1);
        acc[u] = f2_add(acc[u], f2_pack(ex2_approx(e0), ex2_approx(e1)));
      }
    }
    float s0, s1;
    f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), s0, s1);
    Pair s = two_sum(s0, s1);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      s = pair_add(s, {__shfl_xor_sync(0xffffffffu, s.hi, off), __shfl_xor_sync(0xffffffffu, s.lo, off)});
    const Pair ls = log_pair(s);
    const Pair logp = log_add(two_sum(xy, -m), {-ls.hi, -ls.lo});
    const TokenLoss o = token_grad(a, t, logp);
    if (lane == 0) leave_logp(a, row, logp);
    const float c = fmaf(-(ls.hi + ls.lo), kLog2e, log2f(fabsf(o.g)));
    const float gy = o.g * (1.0f - ex2_approx((logp.hi + logp.lo) * kLog2e));
    const uint32_t sign = o.g > 0.0f ? 0x80008000u : 0u;
    const uint64_t c2 = f2_pack(c, c);
#pragma unroll
    for (int k = 0; k < kG; ++k) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      uint32_t r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float e0, e1;
        f2_unpack(f2_fma(f2_add(f2_pack(lo_bf16(w[u]), hi_bf16(w[u])), nb), l2, c2), e0, e1);
        r[u] = o.g == 0.0f ? 0u : pack_bf16x2(ex2_approx(e0), ex2_approx(e1)) ^ sign;
      }
      v[k] = make_uint4(r[0], r[1], r[2], r[3]);
    }
    store_row(d + sp.head, v, sp.n, buf, lane);
    if (e >= 0) {
      float w = 0.0f;
      if (o.g != 0.0f) w = copysignf(ex2_approx(fmaf(ev + base, kLog2e, c)), -o.g);
      if (o.g != o.g) w = o.g;
      d[e] = to_bf16(w);
    }
    // the sampled token's column, behind the lane's own store of its granule
    __syncwarp();
    if (lane == 0 && o.g != 0.0f) d[t.y] = to_bf16(gy);
  }
}

// ======================================================================================
// The tokens' outputs and the loss
// ======================================================================================
constexpr int kFinishThreads = 128;

__global__ void __launch_bounds__(kFinishThreads) policy_finish(const __grid_constant__ PolicyArgs a) {
  __shared__ double sh[kFinishThreads / 32];
  __shared__ unsigned sh_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t first = blockIdx.x * static_cast<int64_t>(kFinishThreads) + tid;
  Token t = {0, 0.0f, 0.0f, 0.0f, 0.0f};
  if (first < a.T) t = load_token(a, first);     // (while the rows are still at work)
  pdl_wait();
  double sum = 0.0;
  for (int64_t row = first; row < a.T; row += static_cast<int64_t>(gridDim.x) * kFinishThreads) {
    if (row != first) t = load_token(a, row);
    float logp_out = 0.0f, kl_out = 0.0f;
    bool clipped = false;
    if (t.bad(a.V)) set_device_status(a.status, DEV_BAD_INDEX);
    if (t.used(a.V)) {
      const float2 p = __ldcg(a.logp_pair + row);
      const Pair lp = {p.x, p.y};
      clipped = token_grad(a, t, lp).clipped;
      const double logp = static_cast<double>(p.x) + static_cast<double>(p.y);
      const double A = t.A, r = logp - static_cast<double>(t.ref);
      const double surr = clipped ? (A > 0.0 ? a.clip_hi : a.clip_lo) * A
                                  : exp(logp - static_cast<double>(t.old)) * A;
      double kl = 0.0;
      if (a.ref != nullptr) kl = a.kl == 1 ? r : (a.kl == 2 ? 0.5 * r * r : expm1(-r) + r);
      sum += static_cast<double>(t.w) * (a.beta * kl - surr);
      logp_out = static_cast<float>(logp);
      kl_out = static_cast<float>(kl);
    }
    a.clip_mask[row] = clipped ? 1 : 0;
    if (a.logp_out != nullptr) a.logp_out[row] = logp_out;
    if (a.kl_out != nullptr) a.kl_out[row] = kl_out;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) sh[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kFinishThreads / 32; ++w) sum += sh[w];
    a.partial[blockIdx.x] = sum;
    __threadfence();
    sh_last = atomicAdd(a.counter, 1u) == gridDim.x - 1 ? 1u : 0u;
  }
  __syncthreads();
  // the last block adds the blocks' sums in their order: the same result whichever block it is
  if (!sh_last || warp > 0) return;
  __threadfence();
  sum = 0.0;
  for (int i = lane; i < static_cast<int>(gridDim.x); i += 32) sum += __ldcg(a.partial + i);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) *a.loss = static_cast<float>(sum);
}

template <int kG>
cudaError_t launch_warp(const PolicyArgs& a, cudaStream_t s) {
  constexpr int kRows = kWarpThreads / 32;
  // the shifting buffer only where some gradient row is not aligned as its logits are
  const bool shift = (a.ldx - a.ldd) % 8 != 0 ||
                     (reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.dlogits)) % 16 != 0;
  const int smem = shift ? kRows * 32 * kG * 16 : 0;
  static bool attr_set[kMaxDeviceCache] = {};
  const int dev = cached_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(policy_warp<kG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kRows * 32 * kG * 16);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  int64_t grid = (a.T + kRows - 1) / kRows;
  const int64_t most = static_cast<int64_t>(num_sms()) * 8;
  if (grid > most) grid = most;
  policy_warp<kG><<<static_cast<unsigned>(grid), kWarpThreads, static_cast<size_t>(smem), s>>>(a);
  return cudaGetLastError();
}

template <int kStream>
cudaError_t launch_cluster(const PolicyArgs& a, int cl, int per, cudaStream_t s) {
  constexpr int kThreads = kStream + 96;
  // four buffers (two rows of sums ahead) where the exchange or the SM's one CTA leaves room for
  // them
  const int nb = per * 16 <= kSlice4 && (cl > 1 || per * 16 > kSlice2) ? 4 : 3;
  const int smem = nb * per * 16;
  static bool attr_set[kMaxDeviceCache] = {};
  const int dev = cached_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(policy_cluster<kStream>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         3 * kSliceMax);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cl);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 1 : 0;
  // how many fit the GPU, asked once for a shape of launch
  static std::atomic<uint64_t> memo[kMaxDeviceCache];
  const uint64_t key = (static_cast<uint64_t>(cl) << 48) | (static_cast<uint64_t>(per) << 24);
  const uint64_t seen = memo[dev].load();
  int n = 0;
  if ((seen & ~0xFFFFFFull) == key) {
    n = static_cast<int>(seen & 0xFFFFFF);
  } else if (cl > 1) {
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms() * cl), 1, 1);
    if (cudaOccupancyMaxActiveClusters(&n, policy_cluster<kStream>, &cfg) != cudaSuccess || n <= 0) {
      (void)cudaGetLastError();
      n = num_sms() / cl;
    }
  } else {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, policy_cluster<kStream>, kThreads,
                                                      static_cast<size_t>(smem)) != cudaSuccess || n <= 0) {
      (void)cudaGetLastError();
      n = 1;
    }
    n *= num_sms();
  }
  memo[dev].store(key | static_cast<uint64_t>(n));
  if (n > a.T) n = static_cast<int>(a.T);
  cfg.gridDim = dim3(static_cast<unsigned>(n * cl), 1, 1);
  return cudaLaunchKernelEx(&cfg, policy_cluster<kStream>, a, cl, per, nb);
}

}  // namespace

cudaError_t launch_policy_loss(const PolicyArgs& a, cudaStream_t s) {
  const int64_t granules = (a.V + 7) / 8;
  cudaError_t e;
  if (a.V <= 1024) {
    e = launch_warp<4>(a, s);
  } else if (a.V <= 2048) {
    e = launch_warp<8>(a, s);
  } else if (a.V <= 4096) {
    e = launch_warp<16>(a, s);
  } else {
    // the fewest CTAs a row
    int cl = 1;
    while (cl < kMaxCluster && (granules + cl - 1) / cl * 16 > kSliceMax) cl *= 2;
    const int64_t per = (granules + cl - 1) / cl;
    if (per * 16 <= kSliceMax) {
      // (33,554 x 8,000: 185 us with 128 streaming threads, 211 with 256; 16,777 x 16,000: 180, 174)
      e = per * 16 <= kSliceSmall ? launch_cluster<128>(a, cl, static_cast<int>(per), s)
                                  : launch_cluster<256>(a, cl, static_cast<int>(per), s);
    } else {
      int64_t grid = static_cast<int64_t>(num_sms()) * 4;
      if (grid > a.T) grid = a.T;
      policy_rows<<<static_cast<unsigned>(grid), kRowThreads, 0, s>>>(a);
      e = cudaGetLastError();
    }
  }
  if (e != cudaSuccess) return e;
  int64_t grid = (a.T + kFinishThreads - 1) / kFinishThreads;
  if (grid > kMaxPartials) grid = kMaxPartials;
  return launch_after(policy_finish, dim3(static_cast<unsigned>(grid)), kFinishThreads, 0, s, a);
}

}  // namespace ls
