// Norms of queries and keys, a head each, with the rotation in the same pass; its gradient; and the
// append of new keys and values to a paged cache with both on the way.
//
//   r = 1 / sqrt(mean x^2 + eps),  n_d = x_d r (w_d + offset),  (y_i, y_i') = f (n_i cos a - n_i' sin a, n_i' cos a + n_i sin a)
//   gradient, g = the rotation's transpose of dy, u = g (w + offset):
//     dx = r (u - x r^2 mean(u x)),   dw = sum over tokens and heads of g x r
//
// All in fp32, rounded once to bf16; angles as in k_rope.cu.  Bound by HBM: 2 bytes read (4 for the gradient)
// and 2 written a value.  A warp takes a token, or a part of its heads where there are few tokens: D / 16
// lanes share a head, a lane two 16-byte chunks (in the half layout the two whose values turn together), so
// that a head's sums take three shuffles at D = 128, and the lane's weights stay in its registers over all
// the heads that it walks.  The next head's chunks are on their way while this one's are at work.
// 48 heads of 128: 8,192 tokens 41 us in a graph (201 MB, 4.9 TB/s), 32,768 tokens 139 us (5.8 TB/s; the rotation
// alone 36 and 123); appending 14,000 tokens of 80 heads 101 us (566 MB, 5.6 TB/s; without norms 93).
// Gradient: 3,001 tokens 31 us with its two launches in a graph (25 of them the first one's), 32,768 tokens 222 us
// (5.4 TB/s): 16 warps an SM at 128 registers hold 32 KB in flight.
// Weight gradients: a lane's 16 columns in registers over all heads and tokens that it walks, a row of partial
// sums a block, summed in a fixed order by a second kernel (no atomics).
// Element path (a warp a head) for rows that are not 16-byte aligned, D not a multiple of 16 or rot_dim
// not a multiple of 16 (8 interleaved).
#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"
#include "rope_device.cuh"

namespace ls {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlocks = 4;       // blocks of an SM
constexpr int kBwdBlocks = 2;    // of the gradient (up to 128 registers)

// Weight d of queries (which = 0) or keys (1), with the offset.
__device__ __forceinline__ float weight_of(const NormArgs& a, int which, int d) {
  const void* w = which ? a.wk : a.wq;
  float x = 1.0f;
  if (w != nullptr) {
    x = a.w_fp32 ? static_cast<const float*>(w)[d] : bf(static_cast<const uint16_t*>(w)[d], 0);
    x += a.offset;
  }
  return x;
}

// Sum over kLanes neighbouring lanes, in all of them.
template <int kLanes>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// 1 / sqrt(mean), mean a head's mean square and eps; NaN, not 0, where the squares pass fp32 (done right there, by a branch
// that takes the head's sums again, 8,192 tokens took 47.8 us, so 43.6).
__device__ __forceinline__ float root_of(float mean) { return rsqrtf(mean) + (mean - mean); }

// Eight values as four pairs: the arithmetic goes two values an instruction.
__device__ __forceinline__ void unpack8(const uint4& v, uint64_t (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2_pack(bf(w[i], 0), bf(w[i], 1));
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(x[i], lo, hi);
    w[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float f2_sum(uint64_t x) {
  float lo, hi;
  f2_unpack(x, lo, hi);
  return lo + hi;
}

// The two chunks of lane j of a head, and the first pair of each one's angles (-1: not turned).  In the
// half layout both chunks have the same pairs.
struct Chunks {
  int c0, c1, p0, p1;
};
__device__ __forceinline__ Chunks chunks_of(const RopeArgs& a, int j) {
  Chunks c;
  if (a.interleaved) {
    c.c0 = 16 * j;
    c.c1 = c.c0 + 8;
    c.p0 = c.c0 < a.rot ? c.c0 / 2 : -1;
    c.p1 = c.c1 < a.rot ? c.c1 / 2 : -1;
  } else if (16 * j < a.rot) {
    c.c0 = 8 * j;
    c.c1 = a.rot / 2 + 8 * j;
    c.p0 = c.p1 = 8 * j;
  } else {
    c.c0 = 16 * j;
    c.c1 = c.c0 + 8;
    c.p0 = c.p1 = -1;
  }
  return c;
}

// x0, x1 turned in place.  Lane j's pairs are 8 j .. 8 j + 7 in both layouts; in the warp's part of shared
// memory two of them lie behind one another for all lanes of a head, [4][kLanes] of two cosines and two sines, so
// that a head's lanes read neighbouring 16 bytes.  (volatile: held in registers over the loop they push others out)
template <int kLanes>
__device__ __forceinline__ void turn(const Chunks& c, bool interleaved, const float* cs, int j, uint64_t (&x0)[4], uint64_t (&x1)[4]) {
  if (c.p0 < 0 && c.p1 < 0) return;
  const uint32_t at = smem_u32(cs) + j * 16;
  const uint64_t minus = f2_pack(-1.0f, -1.0f);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float4 r;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(at + u * kLanes * 16) : "memory");
    if (!interleaved) {
      const uint64_t cc = f2_pack(r.x, r.y), ss = f2_pack(r.z, r.w), a = x0[u], b = x1[u];
      x0[u] = f2_fma(b, f2_mul(ss, minus), f2_mul(a, cc));
      x1[u] = f2_fma(a, ss, f2_mul(b, cc));
    } else if (u < 2 || c.p1 >= 0) {
      uint64_t* x = u < 2 ? x0 + 2 * u : x1 + 2 * (u - 2);
      float a, b;
      f2_unpack(x[0], a, b);
      x[0] = f2_pack(a * r.x - b * r.z, b * r.x + a * r.z);
      f2_unpack(x[1], a, b);
      x[1] = f2_pack(a * r.y - b * r.w, b * r.y + a * r.w);
    }
  }
}
// Where the cosine of pair p of a warp's token lies; the sine lies two behind.
template <int kLanes>
__device__ __forceinline__ int angle_place(int p) {
  return (((p & 7) >> 1) * kLanes + (p >> 3)) * 4 + (p & 1);
}

// A lane's weights of queries (0) or keys (1).
__device__ __forceinline__ void load_weights(const NormArgs& n, int which, const Chunks& c, uint64_t (&w0)[4], uint64_t (&w1)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    w0[u] = f2_pack(weight_of(n, which, c.c0 + 2 * u), weight_of(n, which, c.c0 + 2 * u + 1));
    w1[u] = f2_pack(weight_of(n, which, c.c1 + 2 * u), weight_of(n, which, c.c1 + 2 * u + 1));
  }
}

// Where head h of token t lives: 0 query, 1 key, 2 value (append only).
__device__ __forceinline__ const uint16_t* source(const RopeArgs& a, int64_t t, int h) {
  if (h < a.Hq) return a.q + t * a.qs + h * a.D;
  h -= a.Hq;
  if (h < a.Hk) return a.k + t * a.ks + h * a.D;
  return a.v + t * a.vs + (h - a.Hk) * a.D;
}
__device__ __forceinline__ uint16_t* target(const RopeArgs& a, int64_t t, int h, int64_t page) {
  if (h < a.Hq) return a.qo + t * a.qos + h * a.D;
  h -= a.Hq;
  if (!a.append) return a.ko + t * a.kos + h * a.D;
  if (h < a.Hk) return a.c.k + page + h * a.c.head_stride;
  return a.c.v + page + (h - a.Hk) * a.c.head_stride;
}

// A block's one token: its position (an append's place too) and the angles, for the element path.
__device__ __forceinline__ void prepare_token(const RopeArgs& a, int64_t t, Token* tok, float2* cs) {
  const int tid = threadIdx.x, half = a.rot >> 1;
  if (a.append) {
    if (tid < 32) {
      const Token r = locate(a, t, tid);
      if (tid == 0) *tok = r;
    }
  } else if (tid == 0) {
    tok->pos = a.positions != nullptr ? a.positions[t] : a.pos0 + t;
    tok->page = 0;
  }
  __syncthreads();
  for (int p = tid; p < half; p += kThreads) cs[p] = angle_of(a, tok->pos, p);
}

// The place of a warp's token (found by the whole warp).
__device__ __forceinline__ Token warp_token(const RopeArgs& a, int64_t t, int lane) {
  Token r;
  if (a.append) {
    r = locate(a, t, lane);
    r.pos = __shfl_sync(0xffffffffu, r.pos, 0);
    r.page = __shfl_sync(0xffffffffu, r.page, 0);
  } else {
    r.pos = a.positions != nullptr ? a.positions[t] : a.pos0 + t;
    r.page = 0;
  }
  return r;
}
// Its angles in the warp's part of shared memory.
template <int kLanes>
__device__ __forceinline__ void warp_angles(const RopeArgs& a, int64_t pos, int lane, float* cs) {
  __syncwarp();
  for (int p = lane; p < a.rot >> 1; p += 32) {
    const float2 e = angle_of(a, pos, p);
    cs[angle_place<kLanes>(p)] = e.x;
    cs[angle_place<kLanes>(p) + 2] = e.y;
  }
  __syncwarp();
}

// A warp's unit of work: some heads of one token.
struct Split {
  int parts, per;       // units of a token, heads of a unit
};
struct Unit {
  int64_t t;
  int first, end;
};
__device__ __forceinline__ Unit unit_of(int64_t u, const Split& s, int H) {
  Unit w;
  w.t = u / s.parts;
  w.first = static_cast<int>(u - w.t * s.parts) * s.per;
  w.end = w.first + s.per < H ? w.first + s.per : H;
  return w;
}

template <int kLanes>
__global__ void __launch_bounds__(kThreads, kBlocks) norm_rope_kernel(const __grid_constant__ NormArgs n, const Split split) {
  extern __shared__ __align__(16) float angles[];        // [warp][4][kLanes][4]
  constexpr int kSlots = 32 / kLanes;
  const RopeArgs& a = n.r;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (unit >= a.T * split.parts) return;
  const Unit w = unit_of(unit, split, a.Hq + a.Hk + (a.append ? a.Hk : 0));
  const int j = lane % kLanes;
  const bool mine = 16 * j < a.D;
  const Chunks c = chunks_of(a, j);
  float* cs = angles + warp * 16 * kLanes;

  // 0 queries, 1 keys, 2 values: within a kind heads lie at one distance from one another
  auto kind_of = [&](int h) { return h < a.Hq ? 0 : (h < a.Hq + a.Hk ? 1 : 2); };
  int h = w.first + lane / kLanes;
  int from = -1;                   // kind that `in` is of
  const uint16_t* in = nullptr;
  uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
  auto load = [&]() {
    const int kind = kind_of(h);
    if (kind != from) {
      from = kind;
      in = source(a, w.t, h);
    } else {
      in += kSlots * a.D;
    }
    v0 = *reinterpret_cast<const uint4*>(in + c.c0);
    v1 = *reinterpret_cast<const uint4*>(in + c.c1);
  };
  if (h < w.end && mine) load();
  const Token tok = warp_token(a, w.t, lane);
  if (tok.page < 0) return;
  warp_angles<kLanes>(a, tok.pos, lane, cs);
  uint64_t w0[4], w1[4];
  int to = -1;                     // kind that `out` and the weights are of
  uint16_t* out = nullptr;
  const float inv_d = 1.0f / static_cast<float>(a.D);
#pragma unroll 1
  for (int i = w.first; i < w.end; i += kSlots) {
    const uint4 x0v = v0, x1v = v1;
    const int hh = h;
    h += kSlots;
    if (h < w.end && mine) load();
    uint64_t x0[4], x1[4], sq[2] = {0ull, 0ull};
    unpack8(x0v, x0);
    unpack8(x1v, x1);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      sq[0] = f2_fma(x0[u], x0[u], sq[0]);
      sq[1] = f2_fma(x1[u], x1[u], sq[1]);
    }
    const float r = root_of(fmaf(lane_sum<kLanes>(f2_sum(f2_add(sq[0], sq[1]))), inv_d, n.eps));
    if (hh >= w.end || !mine) continue;
    const int kind = kind_of(hh);
    if (kind != to) {
      to = kind;
      out = target(a, w.t, hh, tok.page);
      if (kind < 2) load_weights(n, kind, c, w0, w1);
    } else {
      out += kSlots * (a.append && kind > 0 ? a.c.head_stride : static_cast<int64_t>(a.D));
    }
    if (kind == 2) {                 // a value: as it is
      *reinterpret_cast<uint4*>(out + c.c0) = x0v;
      *reinterpret_cast<uint4*>(out + c.c1) = x1v;
      continue;
    }
    const uint64_t r2 = f2_pack(r, r);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      x0[u] = f2_mul(x0[u], f2_mul(w0[u], r2));
      x1[u] = f2_mul(x1[u], f2_mul(w1[u], r2));
    }
    turn<kLanes>(c, a.interleaved, cs, j, x0, x1);
    *reinterpret_cast<uint4*>(out + c.c0) = pack8(x0);
    *reinterpret_cast<uint4*>(out + c.c1) = pack8(x1);
  }
}

// Element path: a warp a head.
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const __grid_constant__ NormArgs n) {
  extern __shared__ __align__(16) float2 cs[];
  __shared__ Token tok[1];
  __shared__ float row[kWarps][2 * kMaxRot];
  const RopeArgs& a = n.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = a.rot >> 1;
  const int64_t t = blockIdx.x;
  prepare_token(a, t, tok, cs);
  __syncthreads();
  if (tok[0].page < 0) return;
  const int H = a.Hq + a.Hk + (a.append ? a.Hk : 0);
  float* x = row[warp];
  for (int h = warp; h < H; h += kWarps) {
    const uint16_t* p = source(a, t, h);
    uint16_t* out = target(a, t, h, tok[0].page);
    if (h >= a.Hq + a.Hk) {
      for (int d = lane; d < a.D; d += 32) out[d] = p[d];
      continue;
    }
    float ss = 0.0f;
    __syncwarp();
    for (int d = lane; d < a.D; d += 32) {
      const float v = bf(p[d], 0);
      x[d] = v;
      ss = fmaf(v, v, ss);
    }
    const float r = root_of(lane_sum<32>(ss) / static_cast<float>(a.D) + n.eps);
    for (int d = lane; d < a.D; d += 32) x[d] *= r * weight_of(n, h >= a.Hq, d);
    __syncwarp();
    for (int d = lane; d < a.D; d += 32) {
      float y = x[d];
      if (d < a.rot) {
        const bool second = a.interleaved ? (d & 1) != 0 : d >= half;
        const int i = a.interleaved ? d >> 1 : (second ? d - half : d);
        const float2 e = cs[i];
        const float o = x[a.interleaved ? d ^ 1 : (second ? d - half : d + half)];
        y = second ? y * e.x + o * e.y : y * e.x - o * e.y;
      }
      out[d] = to_bf16(y);
    }
  }
}

// --------------------------------------------------------------------------------------
// Gradient.  a.r holds dy (q, k) and dx (qo, ko) and turns back (inverse).
template <int kLanes>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) norm_rope_bwd_kernel(const __grid_constant__ NormArgs n, const Split split_q, const Split split_k) {
  extern __shared__ __align__(16) float angles[];        // [warp][4][kLanes][4], sums [2][warp][D]
  constexpr int kSlots = 32 / kLanes;
  const RopeArgs& a = n.r;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* cs = angles + warp * 16 * kLanes;
  float* sums = angles + kWarps * 16 * kLanes;
  const int j = lane % kLanes;
  const bool mine = 16 * j < a.D;
  const Chunks c = chunks_of(a, j);
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
  pdl_launch_dependents();

  // queries, then keys: a lane's sums are of one weight
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int H = which ? a.Hk : a.Hq;
    if (H == 0) continue;
    const uint16_t* x = which ? n.xk : n.xq;
    const int64_t xs = which ? n.xks : n.xqs;
    const uint16_t* dy = which ? a.k : a.q;
    const int64_t dys = which ? a.ks : a.qs;
    uint16_t* dx = which ? a.ko : a.qo;
    const int64_t dxs = which ? a.kos : a.qos;
    const Split split = which ? split_k : split_q;
    const int64_t units = a.T * split.parts;
    uint64_t w0[4], w1[4], acc0[4], acc1[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) acc0[u] = acc1[u] = w0[u] = w1[u] = 0ull;
    if (mine) load_weights(n, which, c, w0, w1);
    uint4 g0v = make_uint4(0u, 0u, 0u, 0u), g1v = g0v, x0v = g0v, x1v = g0v;
    auto load = [&](int64_t t, int h) {
      const uint16_t* p = dy + t * dys + h * a.D;
      g0v = *reinterpret_cast<const uint4*>(p + c.c0);
      g1v = *reinterpret_cast<const uint4*>(p + c.c1);
      p = x + t * xs + h * a.D;
      x0v = *reinterpret_cast<const uint4*>(p + c.c0);
      x1v = *reinterpret_cast<const uint4*>(p + c.c1);
    };
    // keys from the last warp on: the warps that have a round of queries less than others begin
    // (3,001 tokens of 48 heads 33.6 -> 31.6 us in a graph, one to 64 tokens 10 -> 9)
    int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (which) unit = warps - 1 - unit;
    Unit w = unit_of(unit < units ? unit : 0, split, H);
    int h = w.first + lane / kLanes;
    if (unit < units && h < w.end && mine) load(w.t, h);
    int64_t pos = a.positions != nullptr ? a.positions[w.t] : a.pos0 + w.t;
#pragma unroll 1
    for (; unit < units; unit += warps) {
      const bool more = unit + warps < units;
      Unit next = w;
      int64_t next_pos = 0;
      if (more) {
        next = unit_of(unit + warps, split, H);
        next_pos = a.positions != nullptr ? a.positions[next.t] : a.pos0 + next.t;
      }
      warp_angles<kLanes>(a, pos, lane, cs);
      pos = next_pos;
#pragma unroll 1
      for (int i = w.first; i < w.end; i += kSlots) {
        uint64_t g0[4], g1[4], x0[4], x1[4];
        unpack8(g0v, g0);
        unpack8(g1v, g1);
        unpack8(x0v, x0);
        unpack8(x1v, x1);
        const int hh = h;
        // the next head of this unit, or the first one of the next
        const bool last = i + kSlots >= w.end;
        h = last ? next.first + lane / kLanes : h + kSlots;
        if (mine && (last ? more && h < next.end : h < w.end)) load(last ? next.t : w.t, h);
        turn<kLanes>(c, a.interleaved, cs, j, g0, g1);
        uint64_t sq[2] = {0ull, 0ull}, sx[2] = {0ull, 0ull}, u0[4], u1[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          u0[u] = f2_mul(g0[u], w0[u]);
          u1[u] = f2_mul(g1[u], w1[u]);
          sq[0] = f2_fma(x0[u], x0[u], sq[0]);
          sq[1] = f2_fma(x1[u], x1[u], sq[1]);
          sx[0] = f2_fma(u0[u], x0[u], sx[0]);
          sx[1] = f2_fma(u1[u], x1[u], sx[1]);
        }
        const float ss = lane_sum<kLanes>(f2_sum(f2_add(sq[0], sq[1])));
        const float su = lane_sum<kLanes>(f2_sum(f2_add(sx[0], sx[1])));
        if (hh >= w.end || !mine) continue;
        const float r = root_of(fmaf(ss, inv_d, n.eps));
        const float m = -(r * r * su * inv_d);
        const uint64_t r2 = f2_pack(r, r), m2 = f2_pack(m, m);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          acc0[u] = f2_fma(g0[u], f2_mul(x0[u], r2), acc0[u]);
          acc1[u] = f2_fma(g1[u], f2_mul(x1[u], r2), acc1[u]);
          g0[u] = f2_mul(f2_fma(x0[u], m2, u0[u]), r2);
          g1[u] = f2_mul(f2_fma(x1[u], m2, u1[u]), r2);
        }
        uint16_t* out = dx + w.t * dxs + hh * a.D;
        *reinterpret_cast<uint4*>(out + c.c0) = pack8(g0);
        *reinterpret_cast<uint4*>(out + c.c1) = pack8(g1);
      }
      w = next;
    }
    if (n.partial == nullptr) continue;
    // the lanes of one column: within the warp, then the warps in order
    float col[2][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      f2_unpack(acc0[u], col[0][2 * u], col[0][2 * u + 1]);
      f2_unpack(acc1[u], col[1][2 * u], col[1][2 * u + 1]);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
#pragma unroll
      for (int off = 16; off >= kLanes; off >>= 1) {
        col[0][u] += __shfl_xor_sync(0xffffffffu, col[0][u], off);
        col[1][u] += __shfl_xor_sync(0xffffffffu, col[1][u], off);
      }
    }
    if (lane < kLanes && mine) {
      float* to = sums + (which * kWarps + warp) * a.D;
#pragma unroll
      for (int u = 0; u < 8; u += 4) {
        *reinterpret_cast<float4*>(to + c.c0 + u) = make_float4(col[0][u], col[0][u + 1], col[0][u + 2], col[0][u + 3]);
        *reinterpret_cast<float4*>(to + c.c1 + u) = make_float4(col[1][u], col[1][u + 1], col[1][u + 2], col[1][u + 3]);
      }
    }
  }
  if (n.partial == nullptr) return;
  // (one wait for both kinds: a warp goes from its queries to its keys without the others)
  __syncthreads();
  for (int d = tid; d < 2 * a.D; d += kThreads) {
    const int which = d < a.D ? 0 : 1;
    if ((which ? a.Hk : a.Hq) == 0) continue;
    const float* of = sums + which * (kWarps - 1) * a.D + d;       // (d counts the first kind's columns too)
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += of[w * a.D];
    n.partial[static_cast<int64_t>(blockIdx.x) * 2 * a.D + d] = s;
  }
}

// Element path: a warp a head; its sums in shared memory.
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_any_kernel(const __grid_constant__ NormArgs n) {
  extern __shared__ __align__(16) float2 cs[];
  __shared__ Token tok[1];
  __shared__ float row[kWarps][2 * kMaxRot], acc[kWarps][2 * kMaxRot];
  const RopeArgs& a = n.r;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = a.rot >> 1;
  float* g = row[warp];
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int H = which ? a.Hk : a.Hq;
    if (H == 0) continue;
    for (int d = lane; d < a.D; d += 32) acc[warp][d] = 0.0f;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
      __syncthreads();
      prepare_token(a, t, tok, cs);
      __syncthreads();
      for (int h = warp; h < H; h += kWarps) {
        const uint16_t* dy = which ? a.k + t * a.ks + h * a.D : a.q + t * a.qs + h * a.D;
        const uint16_t* x = which ? n.xk + t * n.xks + h * a.D : n.xq + t * n.xqs + h * a.D;
        uint16_t* out = which ? a.ko + t * a.kos + h * a.D : a.qo + t * a.qos + h * a.D;
        __syncwarp();
        for (int d = lane; d < a.D; d += 32) g[d] = bf(dy[d], 0);
        __syncwarp();
        float back[2 * kMaxRot / 32];
        float ss = 0.0f, su = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * kMaxRot / 32; ++i) {
          const int d = lane + 32 * i;
          back[i] = 0.0f;
          if (d >= a.D) continue;
          float y = g[d];
          if (d < a.rot) {
            const bool second = a.interleaved ? (d & 1) != 0 : d >= half;
            const int p = a.interleaved ? d >> 1 : (second ? d - half : d);
            const float2 e = cs[p];
            const float o = g[a.interleaved ? d ^ 1 : (second ? d - half : d + half)];
            y = second ? y * e.x + o * e.y : y * e.x - o * e.y;
          }
          back[i] = y;
          const float v = bf(x[d], 0);
          ss = fmaf(v, v, ss);
          su = fmaf(y * weight_of(n, which, d), v, su);
        }
        const float r = root_of(lane_sum<32>(ss) / static_cast<float>(a.D) + n.eps);
        const float m = r * r * lane_sum<32>(su) / static_cast<float>(a.D);
#pragma unroll
        for (int i = 0; i < 2 * kMaxRot / 32; ++i) {
          const int d = lane + 32 * i;
          if (d >= a.D) continue;
          const float v = bf(x[d], 0);
          acc[warp][d] += back[i] * v * r;
          out[d] = to_bf16(r * (back[i] * weight_of(n, which, d) - v * m));
        }
      }
    }
    if (n.partial == nullptr) continue;
    __syncthreads();
    for (int d = tid; d < a.D; d += kThreads) {
      float s = 0.0f;
      for (int w = 0; w < kWarps; ++w) s += acc[w][d];
      n.partial[(static_cast<int64_t>(blockIdx.x) * 2 + which) * a.D + d] = s;
    }
    __syncthreads();
  }
}

// The blocks' partial rows summed in order: a block 8 columns, a thread of each every 32nd row.
__global__ void __launch_bounds__(kThreads) norm_rope_sum_kernel(const float* partial, int blocks, int D, float* dwq, float* dwk) {
  __shared__ float s[32][8];
  const int at = threadIdx.x >> 3, col = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x & 7);        // of [2][D]
  const bool want = col < 2 * D && (col < D ? dwq : dwk) != nullptr;
  pdl_wait();
  float x = 0.0f;
  if (want) {
#pragma unroll 10
    for (int b = at; b < blocks; b += 32) x += __ldcg(partial + static_cast<int64_t>(b) * 2 * D + col);
  }
  s[at][threadIdx.x & 7] = x;
  __syncthreads();
  if (at > 0 || !want) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) x += s[i][threadIdx.x & 7];
  if (col < D) dwq[col] = x; else dwk[col - D] = x;
}

bool vec_ok(const void* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0; }

// Lanes of a head: D / 16, rounded up to a power of two; 0: element path.
int lanes_of(const NormArgs& n) {
  const RopeArgs& a = n.r;
  bool vec = a.D % 16 == 0 && (a.interleaved ? a.rot % 8 == 0 : a.rot % 16 == 0);
  if (a.Hq > 0) vec = vec && vec_ok(a.q, a.qs) && vec_ok(a.qo, a.qos) && (n.xq == nullptr || vec_ok(n.xq, n.xqs));
  if (a.Hk > 0) vec = vec && vec_ok(a.k, a.ks) && (n.xk == nullptr || vec_ok(n.xk, n.xks));
  if (a.append)
    vec = vec && vec_ok(a.v, a.vs);    // pages are 16-byte aligned
  else if (a.Hk > 0)
    vec = vec && vec_ok(a.ko, a.kos);
  if (!vec) return 0;
  int l = 1;
  while (16 * l < a.D) l *= 2;
  return l;
}

size_t angles_bytes(int lanes) { return static_cast<size_t>(8) * lanes * kWarps * sizeof(float2); }

// How a token's heads become units: the least rounds of heads on any of the warps, where a unit itself counts as
// `own` of them.  A warp that ends with its unit: 5 (48 heads: 3,001 tokens 17.8 us in a graph, with 1 20.4; 20,000
// 91 and 96); a warp that goes on to the next one, whose loads are on their way: 1 (gradient of 3,001 tokens 31.6 us,
// with 5 34).
Split split_of(int64_t T, int H, int lanes, int64_t warps, double own) {
  const int slots = 32 / lanes, most = (H + slots - 1) / slots;
  Split best = {1, most * slots};
  double least = 0.0;
  for (int p = 1; p <= most; ++p) {
    const int per = ((H + p - 1) / p + slots - 1) / slots * slots;
    const int64_t parts = (H + per - 1) / per;
    const double cost = static_cast<double>((T * parts + warps - 1) / warps) * (per / slots + own);
    if (p == 1 || cost < least) {
      least = cost;
      best = {static_cast<int>(parts), per};
    }
  }
  return best;
}

}  // namespace

cudaError_t launch_norm_rope(const NormArgs& n, cudaStream_t s) {
  const RopeArgs& a = n.r;
  const int lanes = lanes_of(n);
  if (lanes == 0) {
    norm_rope_any_kernel<<<static_cast<unsigned>(a.T), kThreads, (a.rot / 2) * sizeof(float2), s>>>(n);
    return cudaGetLastError();
  }
  const Split sp = split_of(a.T, a.Hq + a.Hk + (a.append ? a.Hk : 0), lanes, static_cast<int64_t>(num_sms()) * kBlocks * kWarps, 5.0);
  const unsigned grid = static_cast<unsigned>((a.T * sp.parts + kWarps - 1) / kWarps);
  const size_t smem = angles_bytes(lanes);
  switch (lanes) {
    case 1: norm_rope_kernel<1><<<grid, kThreads, smem, s>>>(n, sp); break;
    case 2: norm_rope_kernel<2><<<grid, kThreads, smem, s>>>(n, sp); break;
    case 4: norm_rope_kernel<4><<<grid, kThreads, smem, s>>>(n, sp); break;
    case 8: norm_rope_kernel<8><<<grid, kThreads, smem, s>>>(n, sp); break;
    default: norm_rope_kernel<16><<<grid, kThreads, smem, s>>>(n, sp); break;
  }
  return cudaGetLastError();
}

int norm_rope_bwd_blocks(int64_t T) {
  const int64_t most = static_cast<int64_t>(num_sms()) * kBwdBlocks;
  return static_cast<int>(T < most ? T : most);
}

cudaError_t launch_norm_rope_bwd(const NormArgs& n, float* dwq, float* dwk, cudaStream_t s) {
  const RopeArgs& a = n.r;
  const int lanes = lanes_of(n);
  const unsigned grid = static_cast<unsigned>(norm_rope_bwd_blocks(a.T));
  if (lanes == 0) {
    norm_rope_bwd_any_kernel<<<grid, kThreads, (a.rot / 2) * sizeof(float2), s>>>(n);
  } else {
    const size_t smem = angles_bytes(lanes) + 2 * kWarps * static_cast<size_t>(a.D) * sizeof(float);
    const int64_t warps = static_cast<int64_t>(grid) * kWarps;
    const Split q = split_of(a.T, a.Hq > 0 ? a.Hq : 1, lanes, warps, 1.0), k = split_of(a.T, a.Hk > 0 ? a.Hk : 1, lanes, warps, 1.0);
    switch (lanes) {
      case 1: norm_rope_bwd_kernel<1><<<grid, kThreads, smem, s>>>(n, q, k); break;
      case 2: norm_rope_bwd_kernel<2><<<grid, kThreads, smem, s>>>(n, q, k); break;
      case 4: norm_rope_bwd_kernel<4><<<grid, kThreads, smem, s>>>(n, q, k); break;
      case 8: norm_rope_bwd_kernel<8><<<grid, kThreads, smem, s>>>(n, q, k); break;
      default: norm_rope_bwd_kernel<16><<<grid, kThreads, smem, s>>>(n, q, k); break;
    }
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || n.partial == nullptr) return e;
  return launch_after(norm_rope_sum_kernel, dim3(static_cast<unsigned>((2 * a.D + 7) / 8)), kThreads, 0, s,
                      static_cast<const float*>(n.partial), static_cast<int>(grid), a.D, dwq, dwk);
}

}  // namespace ls
