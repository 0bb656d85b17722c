// Scores of given tokens (review section 2-1 step 2, old- and reference-policy scoring, with what a
// rollout answers beside it): log-probability, log-sum-exp, entropy and the most likely alternatives of
// every row at a temperature t, and the gradient through the first and the third.
//
//   lse = log sum_v exp(x_v / t),  logp = x_y / t - lse,  p_v = exp(x_v / t - lse)
//   entropy = - sum_v p_v log p_v = log S - (sum_v e_v z_v) / S,  z_v = (x_v - max) / t, e_v = exp(z_v), S = sum e_v
//   d x_v = (d_logp (1[v = y] - p_v) - d_entropy p_v (log p_v + entropy)) / t
//
// scores_kernel: a CTA a row, or a cluster of them where there are few rows, each with a slice; one read
//   of the row.  A thread keeps the sum of exponentials (compensated) and sum e z in fp32, relative to its warp's
//   largest logit, and how many equal it; joined across the CTA, the last logarithm in
//   fp64: a token with nearly all of the probability keeps the digits of what is left.  For the alternatives
//   the largest logit of every 32 neighbours stays in shared memory: the k best logits of a row (ties to the
//   lowest index) lie in the k groups with the largest maxima (ties to the lowest group), so that only these are
//   looked at again.  Proof: were one of them in another group, each of the k groups before that one
//   would hold a logit before it.
//   Bound by HBM without alternatives (4,096 rows of 151,936: 190 us, 6.5 TB/s); with 20 of them (228 us) a row's
//   end, a chain of eight barriers, keeps a ninth of the SM's CTAs from reading.  128 threads and nine CTAs an SM: with
//   256 threads 281 us, one CTA an SM fed by bulk copies, with warps of its own for the alternatives, 291.
// scores_bwd_kernel: one pass, a block 4,096 logits of a row (1,279 rows of 151,936: 108 us, 7.2 TB/s); rows whose lse is
//   far from zero by one block each.
#include <type_traits>

#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"

namespace ls {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kUnroll = 4;                        // 4 x 8 logits a thread and step
constexpr int kStep = kThreads * 8 * kUnroll;
constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.69314718055994530942;
constexpr uint32_t kNegInf2 = 0xFF80FF80u;

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Largest of two pairs; a NaN stays.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// Whole numbers in the order of bf16 values, -0 as 0; +inf is 0xFF80, and NaN (as max2 leaves it) above.
__device__ __forceinline__ uint32_t order(uint32_t bits) {
  bits = bits == 0x8000u ? 0u : bits;
  return bits & 0x8000u ? 0xFFFFu - bits : bits | 0x8000u;
}
__device__ __forceinline__ float value_of(uint32_t ord) {
  return __uint_as_float((ord & 0x8000u ? ord & 0x7FFFu : 0xFFFFu - ord) << 16);
}

// hi + lo += t, with the exact error of the fp32 addition kept in lo.
__device__ __forceinline__ void two_sum_acc(float& hi, float& lo, float t) {
  const float s = hi + t;
  const float b = s - hi;
  lo += (hi - (s - b)) + (t - b);
  hi = s;
}

// Eight logits of a row from index i on (a multiple of 8); -inf past the end.
template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t* x, int64_t i, int64_t end) {
  if (kVec && i + 8 <= end) return __ldg(reinterpret_cast<const uint4*>(x + i));
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = i + 2 * k < end ? x[i + 2 * k] : 0xFF80u, b = i + 2 * k + 1 < end ? x[i + 2 * k + 1] : 0xFF80u;
    w[k] = a | (b << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sums are kept of 2^z, z = x scale2 - r, r = m scale2 rounded, m the largest logit of theirs: one fused
// product and difference an exponent, right to 2^-24 of it.  The logits that equal m are counted instead, 1 each
// (m's own z is only the rounding of r).  Where r is past kFar, or m is -inf, z is (x - m) scale2: any two
// logits there differ by 2^-9 of the larger or more, so z is below -2^13 for all but the counted ones, and the rounding
// of r, half an ulp of it, stays below 1 (past 2^34 it would pass fp32's exponents, whose 2^z is then no correction).
constexpr float kFar = 8388608.0f;       // 2^23
// (a product by itself: fused into the difference of two references it would not be the rounded one that the sums are
// relative to)
__device__ __forceinline__ float reference(float m, float scale2) { return __fmul_rn(m, scale2); }

// Sums with the largest logit m and reference r, for a larger one.
__device__ __forceinline__ void rebase(float to, float scale2, float m, float& r, float& ones, float& hi, float& lo, float& e) {
  const float next = reference(to, scale2);
  const bool near = fabsf(r) < kFar && fabsf(next) < kFar;
  if (near) {                        // the counted ones join the sum
    const float z = fmaf(m, scale2, -r);
    e = fmaf(ones, z, e);
    two_sum_acc(hi, lo, ones * fmaf(z, 0.69314718f, 1.0f));
  }
  // z falls by d for all, 2^z by f, sum 2^z z to f (sum 2^z z + d sum 2^z)
  const float d = near ? fmaxf(r - next, -1000.0f) : -1000.0f, f = ex2_approx(d);
  e = f * fmaf(d, hi, e);
  hi *= f;
  lo *= f;
  ones = 0.0f;
  r = next;
}

// Sum and sum e z of a thread's chunk.  kPeak: without the exponentials of logits that equal m, which are
// counted; kFarOff: r is out of range.
template <bool kPeak, bool kFarOff>
__device__ __forceinline__ void add_chunk(const uint4 (&v)[kUnroll], float m, float r, float scale2, float& ones, float& s,
                                          float& es) {
  const uint64_t c2 = f2_pack(scale2, scale2), r2 = f2_pack(-r, -r);
  uint64_t s2[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)}, e2[2] = {s2[0], s2[0]};
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t x = f2_pack(lo_bf16(w[k]), hi_bf16(w[k]));
      uint64_t z;
      if constexpr (kFarOff) {
        // (below: exponents of nothing, and -inf - -inf)
        z = f2_pack(fmaxf((lo_bf16(w[k]) - m) * scale2, -1000.0f), fmaxf((hi_bf16(w[k]) - m) * scale2, -1000.0f));
      } else {
        z = f2_fma(x, c2, r2);
      }
      float z0, z1;
      f2_unpack(z, z0, z1);
      float p0 = ex2_approx(z0), p1 = ex2_approx(z1);
      if constexpr (kPeak) {
        if (lo_bf16(w[k]) == m) {
          ones += 1.0f;
          p0 = 0.0f;
        }
        if (hi_bf16(w[k]) == m) {
          ones += 1.0f;
          p1 = 0.0f;
        }
      }
      const uint64_t p = f2_pack(p0, p1);
      s2[k & 1] = f2_add(s2[k & 1], p);
      e2[k & 1] = f2_fma(p, z, e2[k & 1]);
    }
  }
  float s0, s1, e0, e1;
  f2_unpack(f2_add(s2[0], s2[1]), s0, s1);
  f2_unpack(f2_add(e2[0], e2[1]), e0, e1);
  s = s0 + s1;
  es = e0 + e1;
}

// Sum e z of a chunk that holds logits of -inf (or so low that their z is): 0 x -1000 is 0 where 0 x -inf is not.
__device__ __forceinline__ float chunk_entropy(const uint4 (&v)[kUnroll], float m, float r, float scale2) {
  float es = 0.0f;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x0 = lo_bf16(w[k]), x1 = hi_bf16(w[k]);
      const float z0 = fmaxf(fmaf(x0, scale2, -r), -1000.0f), z1 = fmaxf(fmaf(x1, scale2, -r), -1000.0f);
      if (x0 != m) es = fmaf(ex2_approx(z0), z0, es);
      if (x1 != m) es = fmaf(ex2_approx(z1), z1, es);
    }
  }
  return es;
}

// A warp's sums of what it has read, relative to its own maximum m (one a warp).
struct Sums {
  float m, r, ones, hi, lo, e;
  uint32_t top2;             // a lane's largest logits of even and odd places, a NaN if there is one
  uint32_t group;            // the largest of the groups that it has stored, as select_best counts them
};

__device__ __forceinline__ Sums no_sums() { return {-INFINITY, -INFINITY, 0.0f, 0.0f, 0.0f, 0.0f, kNegInf2, 0u}; }

// A step of kN threads: thread tid has logits base + 8 kN u + 8 tid .. + 7 of a slice of len in v[u].
template <bool kTop, int kN>
__device__ __forceinline__ void add_step(Sums& s, const uint4 (&v)[kUnroll], float scale2, int base, int tid, int len,
                                         uint16_t* groups) {
  uint32_t g[kUnroll / 2];      // the largest of each eight, two a register
#pragma unroll
  for (int u = 0; u < kUnroll; u += 2) {
    const uint32_t p = max2(max2(v[u].x, v[u].y), max2(v[u].z, v[u].w));
    const uint32_t q = max2(max2(v[u + 1].x, v[u + 1].y), max2(v[u + 1].z, v[u + 1].w));
    g[u / 2] = max2(__byte_perm(p, q, 0x5410), __byte_perm(p, q, 0x7632));
  }
  if constexpr (kTop) {
    // of 32 neighbours: four lanes together
#pragma unroll
    for (int i = 0; i < kUnroll / 2; ++i) {
      g[i] = max2(g[i], __shfl_xor_sync(0xffffffffu, g[i], 1));
      g[i] = max2(g[i], __shfl_xor_sync(0xffffffffu, g[i], 2));
    }
    const int u = tid & 3;
    const uint32_t w = u & 2 ? g[1] : g[0];
    const int at = (base + u * kN * 8 + tid * 8) >> 5;
    if (at * 32 < len) {
      const uint32_t o = order(u & 1 ? w >> 16 : w & 0xFFFFu);
      groups[at] = static_cast<uint16_t>(o);
      s.group = max(s.group, (o << 16) | (0xFFFFu - static_cast<uint32_t>(at)));
    }
  }
  const uint32_t t2 = max2(g[0], g[1]);
  s.top2 = max2(s.top2, t2);
  // (one maximum a warp: a lane's own would grow in most steps of some lane)
  const float cm = warp_max(fmaxf(lo_bf16(t2), hi_bf16(t2)));
  if (cm > s.m) {
    rebase(cm, scale2, s.m, s.r, s.ones, s.hi, s.lo, s.e);
    s.m = cm;
  }
  // peak: the maximum is among these; its exponentials, 1 each, are counted and not added
  const bool peak = cm == s.m;
  float sum, es;
  if (!(fabsf(s.r) < kFar)) {
    add_chunk<true, true>(v, s.m, s.r, scale2, s.ones, sum, es);
  } else if (peak) {
    add_chunk<true, false>(v, s.m, s.r, scale2, s.ones, sum, es);
  } else {
    add_chunk<false, false>(v, s.m, s.r, scale2, s.ones, sum, es);
  }
  if (!(es == es)) es = chunk_entropy(v, s.m, s.r, scale2);     // 0 x -inf
  two_sum_acc(s.hi, s.lo, sum);
  s.e += es;
}

// Logits [begin, end) of a row by kThreads threads, tid of them; groups: the largest logit of every 32, as a whole number.
template <bool kVec, bool kTop>
__device__ __forceinline__ Sums stream(const ScoresArgs& a, const uint16_t* x, int64_t begin, int64_t end, int tid,
                                       uint16_t* groups) {
  const int len = end > begin ? static_cast<int>(end - begin) : 0;
  Sums w = no_sums();
  for (int base = 0; base < len; base += kStep) {
    // the next step on its way to L2 (one step ahead: 231 us with 20 alternatives, two 233, none 251)
    if (kVec && tid == 0 && base + 2 * kStep <= len) bulk_prefetch_l2(x + begin + base + kStep, kStep * 2);
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int at = base + u * kThreads * 8 + tid * 8;
      v[u] = kVec && base + kStep <= len ? __ldg(reinterpret_cast<const uint4*>(x + begin + at)) : load8<kVec>(x, begin + at, end);
    }
    add_step<kTop, kThreads>(w, v, a.scale2, base, tid, len, groups);
  }
  return w;
}

// The warp's sums over its lanes, relative to `peak`.
__device__ __forceinline__ void add_lanes(Sums& w, float peak, float scale2) {
  if (w.m != peak) rebase(peak, scale2, w.m, w.r, w.ones, w.hi, w.lo, w.e);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, w.hi, off);
    w.lo += __shfl_xor_sync(0xffffffffu, w.lo, off);
    two_sum_acc(w.hi, w.lo, h);
    w.e += __shfl_xor_sync(0xffffffffu, w.e, off);
    w.ones += __shfl_xor_sync(0xffffffffu, w.ones, off);
  }
}

// Largest logit of a warp's part as a whole number.
__device__ __forceinline__ uint32_t warp_top(const Sums& w) {
  return __reduce_max_sync(0xffffffffu, max(order(w.top2 & 0xFFFFu), order(w.top2 >> 16)));
}

// What a part of a row has come to: its largest logit (as a whole number), sums relative to it.
struct Slice {
  uint32_t top;
  float ones, hi, lo, e;
};
// A row from its parts, joined in order (one thread).
struct Row {
  uint32_t top;
  bool none;       // a NaN or an infinite logit, or none that is larger than -inf: no distribution
  double lns;      // log of the sum relative to the largest logit
};
__device__ __forceinline__ Row finish_row(const ScoresArgs& a, const Slice* parts, int n_parts, int64_t row, int y, float xy) {
  uint32_t all = 0u;
  for (int i = 0; i < n_parts; ++i) all = max(all, parts[i].top);
  const float peak = value_of(all);
  float n = 0.0f, h = 0.0f, l = 0.0f, w = 0.0f;
  for (int i = 0; i < n_parts; ++i) {
    Slice s = parts[i];
    const float from = value_of(s.top);
    float base = reference(from, a.scale2);
    if (from != peak) rebase(peak, a.scale2, from, base, s.ones, s.hi, s.lo, s.e);
    n += s.ones;
    two_sum_acc(h, l, s.hi);
    l += s.lo;
    w += s.e;
  }
  Row out;
  out.top = all;
  out.none = all >= 0xFF80u || all <= 0x007Fu;
  // the reference's rounding goes out again: z from the peak itself is z + off
  const float base = reference(peak, a.scale2);
  const double off = fabsf(base) < kFar ? static_cast<double>(base) - static_cast<double>(peak) * a.scale2 : 0.0;
  const double back = fabs(off) < 0x1p-12 ? 1.0 + off * kLn2 : exp2(off);
  const double rest = (static_cast<double>(h) + static_cast<double>(l)) * back, S = n + rest;
  out.lns = out.none ? static_cast<double>(NAN) : log1p(n - 1.0 + rest);
  a.logp[row] = y < 0 ? 0.0f : static_cast<float>((static_cast<double>(xy) - peak) * a.scale - out.lns);
  if (a.lse != nullptr) a.lse[row] = static_cast<float>(peak * a.scale + out.lns);
  if (a.entropy != nullptr) {
    const double ent = out.lns - kLn2 * (w * back + off * rest) / S;
    a.entropy[row] = ent < 0.0 ? 0.0f : static_cast<float>(ent);
  }
  return out;
}

// The row's given token (-1: out of range, reported) and its logit.
__device__ __forceinline__ int given_token(const ScoresArgs& a, int64_t row, float* xy) {
  const int y = a.ids[row];
  *xy = 0.0f;
  if (y < 0 || y >= a.V) {
    set_device_status(a.status, DEV_BAD_INDEX);
    return -1;
  }
  *xy = lo_bf16(a.logits[row * a.ldx + y]);
  return y;
}

// The k largest logits of [begin, begin + len) of a row, largest first, equal ones the lowest index first, by kThreads
// threads: keys (order, then the lowest index) to best, 0 where there are fewer.  groups: the largest of every 32.
// mine: the largest group that the thread has stored while it read the row.  scratch: found [32 k], then list [list_size], then chosen [k].
struct Select {
  uint32_t key[kThreads];
  uint32_t low, cut, n[2];
};
__host__ __device__ __forceinline__ int select_list(int64_t len, int k) { return k * static_cast<int>((len / 32 + kThreads) / kThreads); }
__host__ __device__ __forceinline__ size_t select_scratch(int64_t len, int k) {
  return 32 * static_cast<size_t>(k) * 8 + static_cast<size_t>(select_list(len, k)) * 4 + static_cast<size_t>(k) * 4;
}
template <class Sync>
__device__ __forceinline__ void select_best(const uint16_t* x, int64_t begin, int len, const uint16_t* groups, int k,
                                            unsigned long long* best, uint8_t* scratch, int list_size, Select& s, int tid,
                                            uint32_t mine, Sync sync) {
  const int n = (len + 31) >> 5, lane = tid & 31, warp = tid >> 5;
  unsigned long long* found = reinterpret_cast<unsigned long long*>(scratch);
  uint32_t* list = reinterpret_cast<uint32_t*>(found + 32 * k);
  uint32_t* chosen = list + list_size;
  // groups as whole numbers: maximum, then the lowest index; 0: none
  auto key = [&](int g) { return (static_cast<uint32_t>(groups[g]) << 16) | (0xFFFFu - static_cast<uint32_t>(g)); };
  if (tid == 0) {
    s.low = s.cut = 0u;
    s.n[0] = s.n[1] = 0u;
  }
  s.key[tid] = mine;
  if (tid < k) best[tid] = 0ull;
  sync();
  // the k threads with the largest groups hold the k largest groups
  int rank = 0;
#pragma unroll 8
  for (int i = 0; i < kThreads; i += 4) {
    const uint4 o = *reinterpret_cast<const uint4*>(s.key + i);
    rank += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
  }
  if (rank == k - 1) s.low = mine;
  sync();
  if (rank < k && mine > 0u) {
    const uint32_t low = s.low;
    // (the groups that this thread has stored)
#pragma unroll 4
    for (int g = (tid & 3) * (kThreads / 4) + (tid >> 2); g < n; g += kThreads) {
      const uint32_t o = key(g);
      if (o >= low) list[atomicAdd(&s.n[0], 1u)] = o;
    }
  }
  sync();
  const int listed = static_cast<int>(s.n[0]);
  for (int i = tid; i < listed; i += kThreads) {
    const uint32_t o = list[i];
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < listed; ++j) r += list[j] > o;
    if (r < k) chosen[r] = 0xFFFFu - (o & 0xFFFFu);
    if (r == k - 1) s.cut = o >> 16;       // nothing below the last group's maximum is among the best
  }
  sync();
  const int groups_chosen = listed < k ? listed : k;
  const uint32_t cut = s.cut;
  for (int r0 = warp; r0 < groups_chosen; r0 += 8 * kWarps) {
    uint32_t o[8];
    int at[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {      // (eight loads at a time)
      const int r = r0 + q * kWarps;
      at[q] = r < groups_chosen ? static_cast<int>(chosen[r]) * 32 + lane : len;
      o[q] = at[q] < len ? x[begin + at[q]] : 0u;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t key = order(o[q]);
      if (at[q] < len && key >= cut)
        found[atomicAdd(&s.n[1], 1u)] =
            (static_cast<unsigned long long>(key) << 32) | (0xFFFFFFFFull - static_cast<unsigned long long>(begin + at[q]));
    }
  }
  sync();
  const int count = static_cast<int>(s.n[1]);
  for (int i = tid; i < count; i += kThreads) {
    const unsigned long long o = found[i];
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < count; ++j) r += found[j] > o;
    if (r < k) best[r] = o;
  }
}

// Alternative i of a row, given as a key.
__device__ __forceinline__ void put_alternative(const ScoresArgs& a, int64_t row, int i, unsigned long long key, const Row& r) {
  a.top_ids[row * a.top + i] = r.none ? -1 : static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
  a.top_logp[row * a.top + i] =
      r.none ? NAN
             : static_cast<float>((static_cast<double>(value_of(static_cast<uint32_t>(key >> 32))) - value_of(r.top)) * a.scale - r.lns);
}

constexpr int kMaxCluster = 8;

template <bool kVec, bool kTop>
__global__ void __launch_bounds__(kThreads, 9) scores_kernel(const __grid_constant__ ScoresArgs a) {
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ uint32_t sh_max[kWarps];
  __shared__ float sh_sum[kWarps][4];
  __shared__ Slice sh_slice[kMaxCluster];
  __shared__ Select sh_select;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int parts = a.parts;
  const int64_t row = blockIdx.x / parts;
  const int part = parts > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const uint16_t* x = a.logits + row * a.ldx;
  const int64_t begin = part * a.slice;
  const int64_t end = begin + a.slice < a.V ? begin + a.slice : a.V;
  const int len = end > begin ? static_cast<int>(end - begin) : 0;

  if (parts > 1) cluster_arrive();       // (the first CTA has started before the others write to it)

  // the given token's logit is on its way while the row is read
  int y = -1;
  float xy = 0.0f;
  if (tid == 0 && part == 0) y = given_token(a, row, &xy);

  uint16_t* groups = reinterpret_cast<uint16_t*>(dyn);
  Sums w = stream<kVec, kTop>(a, x, begin, end, tid, groups);

  // the slice's maximum, and the sums relative to it
  uint32_t top = warp_top(w);
  if (lane == 0) sh_max[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) top = max(top, sh_max[i]);
  add_lanes(w, value_of(top), a.scale2);
  if (lane == 0) {
    sh_sum[warp][0] = w.hi;
    sh_sum[warp][1] = w.lo;
    sh_sum[warp][2] = w.e;
    sh_sum[warp][3] = w.ones;
  }

  unsigned long long* best = nullptr;        // [parts][top]: the slices' best logits, in order
  if constexpr (kTop) {
    uint8_t* at = dyn + ((static_cast<size_t>(a.slice) + 31) / 32 * 2 + 15) / 16 * 16;
    best = reinterpret_cast<unsigned long long*>(at);
    at += static_cast<size_t>(parts) * a.top * 8;
    select_best(x, begin, len, groups, a.top, best + part * a.top, at, select_list(a.slice, a.top), sh_select, tid, w.group,
                [] { __syncthreads(); });
  }
  __syncwarp();                          // (the cluster's barriers take whole warps; the loops above end lane by lane)
  if (parts > 1) cluster_wait();
  __syncthreads();
  if (tid == 0) {
    Slice s;
    s.top = top;
    s.ones = s.hi = s.lo = s.e = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
      two_sum_acc(s.hi, s.lo, sh_sum[w][0]);
      s.lo += sh_sum[w][1];
      s.e += sh_sum[w][2];
      s.ones += sh_sum[w][3];
    }
    if (part == 0) {
      sh_slice[0] = s;
    } else {
      const uint32_t to = cluster_map(&sh_slice[part], 0);
      st_cluster_u32(to, s.top);
      st_cluster_f32(to + 4, s.ones);
      st_cluster_f32(to + 8, s.hi);
      st_cluster_f32(to + 12, s.lo);
      st_cluster_f32(to + 16, s.e);
    }
  }
  if (parts > 1) {
    if (kTop && part > 0 && tid < a.top) {
      const unsigned long long o = best[part * a.top + tid];
      const uint32_t to = cluster_map(&best[part * a.top + tid], 0);
      st_cluster_u32(to, static_cast<uint32_t>(o));
      st_cluster_u32(to + 4, static_cast<uint32_t>(o >> 32));
    }
    __syncwarp();
    cluster_sync_all();
    if (part > 0) return;
  } else {
    __syncthreads();
  }

  // the row: the slices joined in order
  __shared__ Row sh_row;
  if (tid == 0) sh_row = finish_row(a, sh_slice, parts, row, y, xy);
  if constexpr (kTop) {
    __syncthreads();
    const int k = a.top, all = parts * k;
    const Row r = sh_row;
    if (r.none) {
      if (tid < k) put_alternative(a, row, tid, 0ull, r);
      return;
    }
    for (int i = tid; i < all; i += kThreads) {
      const unsigned long long o = best[i];
      int at = i;
      if (parts > 1) {
        at = 0;
        for (int j = 0; j < all; ++j) at += best[j] > o;
      }
      if (at < k && o != 0ull) put_alternative(a, row, at, o, r);
    }
  }
}

// --------------------------------------------------------------------------------------
// Past this |lse|, p = 2^(x log2 e / t - lse log2 e) from an lse rounded to fp32 would be off by more than 2^-10 (4 x 2^-24
// |lse|: lse, log2 e, 1 / t and their products), half of what the gradient's own rounding is.
constexpr float kFarLse = 4096.0f;

// Eight values of a row's gradient from index i on.
template <bool kVec>
__device__ __forceinline__ void put8(uint16_t* out, int64_t i, int64_t end, const uint32_t (&o)[4]) {
  if (kVec) {
    __stcs(reinterpret_cast<uint4*>(out + i), make_uint4(o[0], o[1], o[2], o[3]));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < end) out[i + k] = static_cast<uint16_t>(k & 1 ? o[k / 2] >> 16 : o[k / 2] & 0xFFFFu);
  }
}
// The given token's value in the chunk that has it.
__device__ __forceinline__ void put_own(uint32_t (&o)[4], int64_t i, int y, float own) {
  if (y < i || y >= i + 8) return;
  const int at = static_cast<int>(y - i);
  const uint32_t b = pack_bf16x2(own, own);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (at == 2 * k) o[k] = __byte_perm(o[k], b, 0x3254);
    if (at == 2 * k + 1) o[k] = __byte_perm(o[k], b, 0x5410);
  }
}

// The gradient of a row with such an lse, by one block (in place no other one may have written any of it): exponents
// relative to the row's maximum and its sum, both found again.  Three reads of the row, two of them from L2 (1,279 such rows
// of 151,936: 276 us).
template <bool kVec>
__device__ __noinline__ void far_row(const ScoresBwdArgs& a, const uint16_t* x, uint16_t* out, int y, float own, float k0,
                                     float k1) {
  __shared__ uint32_t sh_top[kWarps];
  __shared__ double sh_sum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // f(first index, four pairs) for all of the thread's chunks, four loads at a time (-inf behind the row)
  auto all = [&](auto f) {
    for (int64_t first = tid * 8; first < a.V; first += kStep) {
      uint4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = first + u * kThreads * 8;
        v[u] = make_uint4(kNegInf2, kNegInf2, kNegInf2, kNegInf2);
        if (i < a.V) v[u] = kVec ? __ldcg(reinterpret_cast<const uint4*>(x + i)) : load8<false>(x, i, a.V);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        f(first + u * kThreads * 8, w);
      }
    }
  };
  uint32_t top2 = kNegInf2;
  all([&](int64_t, const uint32_t (&w)[4]) { top2 = max2(top2, max2(max2(w[0], w[1]), max2(w[2], w[3]))); });
  uint32_t top = __reduce_max_sync(0xffffffffu, max(order(top2 & 0xFFFFu), order(top2 >> 16)));
  if (lane == 0) sh_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) top = max(top, sh_top[i]);
  const float m = value_of(top);
  float hi = 0.0f, lo = 0.0f;
  all([&](int64_t, const uint32_t (&w)[4]) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      s += ex2_approx((lo_bf16(w[k]) - m) * a.scale2) + ex2_approx((hi_bf16(w[k]) - m) * a.scale2);
    two_sum_acc(hi, lo, s);
  });
  double sum = static_cast<double>(hi) + lo;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) sh_sum[warp] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) sum += sh_sum[i];
  const float base = static_cast<float>(log2(sum)) - a.lift;
  all([&](int64_t i, const uint32_t (&w)[4]) {
    if (i >= a.V) return;
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float z0 = fmaxf(fmaf(lo_bf16(w[k]) - m, a.scale2, -base), -1000.0f);
      const float z1 = fmaxf(fmaf(hi_bf16(w[k]) - m, a.scale2, -base), -1000.0f);
      o[k] = pack_bf16x2(-ex2_approx(z0) * fmaf(k1, z0, k0), -ex2_approx(z1) * fmaf(k1, z1, k0));
    }
    put_own(o, i, y, own);
    put8<kVec>(out, i, a.V, o);
  });
}

template <bool kVec>
__global__ void __launch_bounds__(kThreads) scores_bwd_kernel(const __grid_constant__ ScoresBwdArgs a) {
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.y + static_cast<int64_t>(blockIdx.z) * a.rows_y;
  if (row >= a.T) return;
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * kStep;
  const uint16_t* x = a.logits + row * a.ldx;
  uint16_t* out = a.dlogits + row * a.ldd;
  float dl = a.d_logp != nullptr ? a.d_logp[row] : 0.0f, de = a.d_entropy != nullptr ? a.d_entropy[row] : 0.0f;
  const int y = a.ids[row];
  const float lse = a.lse[row];
  const bool wild = y < 0 || y >= a.V;
  if (wild && begin == 0 && tid == 0) set_device_status(a.status, DEV_BAD_INDEX);
  // a row that nothing is asked of is not looked at
  const bool zero = wild || (dl == 0.0f && de == 0.0f);
  const float base = zero ? 0.0f : fmaf(lse, kLog2e, -a.lift);
  const float ent = zero || a.d_entropy == nullptr ? 0.0f : a.entropy[row];
  dl *= a.scale;
  de *= a.scale;
  // d = -p (dl + de (log p + entropy)) / t = -2^z (k0 + k1 z), z = log2 p + lift (a row without a distribution stays
  // NaN).  1 / t is scale 2^lift, and its second part is the exponentials': dl / t may pass fp32 where p is 0.
  const float k1 = de * static_cast<float>(kLn2);
  float k0 = fmaf(-k1, a.lift, fmaf(de, ent, dl)), own = 0.0f;
  const bool far = !zero && fabsf(lse) > kFarLse;
  if (!zero && (far || (y >= begin && y < begin + kStep))) {
    // 1 - p from the log-probability itself: exact where p is close to 1
    const float lp = a.logp[row];
    own = -expm1f(lp) * dl;
    if (de != 0.0f) own -= de * expf(lp) * (fmaxf(lp, -1000.0f) + ent);
    own *= a.lifted;
  }
  if (far) {
    if (begin == 0) far_row<kVec>(a, x, out, y, own, k0, k1);
    return;
  }
  k0 += base - base;
  uint4 v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = begin + u * kThreads * 8 + tid * 8;
    v[u] = make_uint4(0u, 0u, 0u, 0u);
    if (!zero && i < a.V) v[u] = kVec ? __ldcs(reinterpret_cast<const uint4*>(x + i)) : load8<false>(x, i, a.V);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = begin + u * kThreads * 8 + tid * 8;
    if (i >= a.V) continue;
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    uint32_t o[4] = {0u, 0u, 0u, 0u};
    if (!zero) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float z0 = fmaxf(fmaf(lo_bf16(w[k]), a.scale2, -base), -1000.0f);
        const float z1 = fmaxf(fmaf(hi_bf16(w[k]), a.scale2, -base), -1000.0f);
        o[k] = pack_bf16x2(-ex2_approx(z0) * fmaf(k1, z0, k0), -ex2_approx(z1) * fmaf(k1, z1, k0));
      }
      put_own(o, i, y, own);           // (one chunk of a row has it: no select in the others)
    }
    put8<kVec>(out, i, a.V, o);
  }
}

bool vec_ok(const void* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0; }

template <bool kVec, bool kTop>
cudaError_t launch_scores_t(const ScoresArgs& a, size_t smem, cudaStream_t s) {
  static bool attr_set[kMaxDeviceCache] = {};
  const int dev = cached_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(scores_kernel<kVec, kTop>, cudaFuncAttributeMaxDynamicSharedMemorySize, kScoresSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.parts);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(a.T * a.parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = a.parts > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, scores_kernel<kVec, kTop>, a);
}

}  // namespace

cudaError_t launch_scores(const ScoresArgs& args, cudaStream_t s) {
  ScoresArgs a = args;
  // a cluster a row while the rows alone leave SMs without a CTA, and slices are worth it
  const int64_t sms = num_sms();
  a.parts = 1;
  while (a.parts < kMaxCluster && (a.T * a.parts < 2 * sms || a.V / a.parts > kMaxScoresSlice) && a.V / a.parts > kStep)
    a.parts *= 2;
  a.slice = (a.V + a.parts - 1) / a.parts;
  a.slice = (a.slice + 31) / 32 * 32;
  const bool vec = vec_ok(a.logits, a.ldx);
  const size_t k = static_cast<size_t>(a.top);
  if (a.top == 0) return vec ? launch_scores_t<true, false>(a, 0, s) : launch_scores_t<false, false>(a, 0, s);
  size_t smem = ((static_cast<size_t>(a.slice) + 31) / 32 * 2 + 15) / 16 * 16;
  smem += k * a.parts * 8 + select_scratch(a.slice, a.top);
  if (smem > kScoresSmem) return cudaErrorInvalidValue;
  return vec ? launch_scores_t<true, true>(a, smem, s) : launch_scores_t<false, true>(a, smem, s);
}

cudaError_t launch_scores_bwd(const ScoresBwdArgs& args, cudaStream_t s) {
  ScoresBwdArgs a = args;
  a.rows_y = a.T < 65535 ? static_cast<int>(a.T) : 65535;
  const dim3 grid(static_cast<unsigned>((a.V + kStep - 1) / kStep), static_cast<unsigned>(a.rows_y),
                  static_cast<unsigned>((a.T + a.rows_y - 1) / a.rows_y));
  const bool vec = vec_ok(a.logits, a.ldx) && vec_ok(a.dlogits, a.ldd) && a.V % 8 == 0;
  if (vec)
    scores_bwd_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else
    scores_bwd_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ls
