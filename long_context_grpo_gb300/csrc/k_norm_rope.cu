// Norms of queries and keys, a head each, with the rotation in the same pass; its gradient; and the
// append of new keys and values to a paged cache with both on the way.
//
//   r = 1 / sqrt(mean x^2 + eps),  n_d = x_d r (w_d + offset),  (y_i, y_i') = f (n_i cos a - n_i' sin a, n_i' cos a + n_i sin a)
//   gradient, g = the rotation's transpose of dy, u = g (w + offset):
//     dx = r (u - x r^2 mean(u x)),   dw = sum over tokens and heads of g x r
//
// All in fp32, rounded once to bf16; angles as in k_rope.cu.  Bound by HBM: 2 bytes read (4 for the gradient)
// and 2 written a value.  D / 16 lanes share a head, a lane two 16-byte chunks (in the half layout the two
// whose values turn together), so that a head's sums take three shuffles at D = 128; a block's lanes keep
// their chunks and walk the heads of its tokens, the next head's chunks on their way while this one's
// are at work.  Weight gradients: a lane's 16 columns in registers over all heads that it walks, a row of
// partial sums a block, summed in a fixed order by a second kernel (no atomics).
// Element path (a warp a head) for rows that are not 16-byte aligned, D not a multiple of 16 or rot_dim
// not a multiple of 16 (8 interleaved).
#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"
#include "rope_device.cuh"

namespace ls {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTok = 4;       // tokens of a block at a time
constexpr int kBlocks = 4;       // blocks of an SM
constexpr int kBwdBlocks = 2;    // of the gradient (a lane's sums and two heads' chunks: up to 128 registers)

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

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf(w[i], 0);
    x[2 * i + 1] = bf(w[i], 1);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
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

// x0, x1 turned in place by the token's angles.
__device__ __forceinline__ void turn(const Chunks& c, bool interleaved, const float2* cs, float (&x0)[8], float (&x1)[8]) {
  if (interleaved) {
    if (c.p0 >= 0) {
      const float4* t = reinterpret_cast<const float4*>(cs + c.p0);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 r = t[u];
        const float a0 = x0[4 * u], b0 = x0[4 * u + 1], a1 = x0[4 * u + 2], b1 = x0[4 * u + 3];
        x0[4 * u] = a0 * r.x - b0 * r.y;
        x0[4 * u + 1] = b0 * r.x + a0 * r.y;
        x0[4 * u + 2] = a1 * r.z - b1 * r.w;
        x0[4 * u + 3] = b1 * r.z + a1 * r.w;
      }
    }
    if (c.p1 >= 0) {
      const float4* t = reinterpret_cast<const float4*>(cs + c.p1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 r = t[u];
        const float a0 = x1[4 * u], b0 = x1[4 * u + 1], a1 = x1[4 * u + 2], b1 = x1[4 * u + 3];
        x1[4 * u] = a0 * r.x - b0 * r.y;
        x1[4 * u + 1] = b0 * r.x + a0 * r.y;
        x1[4 * u + 2] = a1 * r.z - b1 * r.w;
        x1[4 * u + 3] = b1 * r.z + a1 * r.w;
      }
    }
  } else if (c.p0 >= 0) {
    const float4* t = reinterpret_cast<const float4*>(cs + c.p0);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float4 r = t[u];
      const float a0 = x0[2 * u], b0 = x1[2 * u], a1 = x0[2 * u + 1], b1 = x1[2 * u + 1];
      x0[2 * u] = a0 * r.x - b0 * r.y;
      x1[2 * u] = b0 * r.x + a0 * r.y;
      x0[2 * u + 1] = a1 * r.z - b1 * r.w;
      x1[2 * u + 1] = b1 * r.z + a1 * r.w;
    }
  }
}

__device__ __forceinline__ void load_weights(const float* w, const Chunks& c, float (&w0)[8], float (&w1)[8]) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float4 a = *reinterpret_cast<const float4*>(w + c.c0 + 4 * u), b = *reinterpret_cast<const float4*>(w + c.c1 + 4 * u);
    w0[4 * u] = a.x; w0[4 * u + 1] = a.y; w0[4 * u + 2] = a.z; w0[4 * u + 3] = a.w;
    w1[4 * u] = b.x; w1[4 * u + 1] = b.y; w1[4 * u + 2] = b.z; w1[4 * u + 3] = b.w;
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

// The positions (an append's places too) and the angles of a block's tokens.
__device__ __forceinline__ void prepare_tokens(const RopeArgs& a, int64_t t0, int nt, Token* tok, float2* cs) {
  const int tid = threadIdx.x, half = a.rot >> 1;
  if (a.append) {
    for (int i = tid >> 5; i < nt; i += kWarps) {
      const Token r = locate(a, t0 + i, tid & 31);
      if ((tid & 31) == 0) tok[i] = r;
    }
  } else if (tid < nt) {
    tok[tid].pos = a.positions != nullptr ? a.positions[t0 + tid] : a.pos0 + t0 + tid;
    tok[tid].page = 0;
  }
  __syncthreads();
  for (int i = tid; i < nt * half; i += kThreads) {
    const int k = i / half, p = i - k * half;
    cs[i] = angle_of(a, tok[k].pos, p);
  }
}

template <int kLanes>
__global__ void __launch_bounds__(kThreads, kBlocks) norm_rope_kernel(const __grid_constant__ NormArgs n, int tb) {
  extern __shared__ __align__(16) float2 cs[];       // [token][pair], then weights [2][D]
  __shared__ Token tok[kMaxTok];
  constexpr int kSlots = kThreads / kLanes;
  const RopeArgs& a = n.r;
  const int tid = threadIdx.x, half = a.rot >> 1;
  float* weights = reinterpret_cast<float*>(cs + ((tb * half + 1) & ~1));
  const int slot = tid / kLanes, j = tid % kLanes;
  const bool mine = 16 * j < a.D;
  const Chunks c = chunks_of(a, j);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tb;
  const int nt = static_cast<int>(a.T - t0 < tb ? a.T - t0 : tb);
  const int H = a.Hq + a.Hk + (a.append ? a.Hk : 0), total = nt * H;

  int k = 0, h = slot;             // this lane's token and head
  while (h >= H) {
    h -= H;
    ++k;
  }
  uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
  if (slot < total && mine) {
    const uint16_t* p = source(a, t0 + k, h);
    v0 = *reinterpret_cast<const uint4*>(p + c.c0);
    v1 = *reinterpret_cast<const uint4*>(p + c.c1);
  }
  for (int i = tid; i < 2 * a.D; i += kThreads) weights[i] = weight_of(n, i >= a.D, i >= a.D ? i - a.D : i);
  prepare_tokens(a, t0, nt, tok, cs);
  __syncthreads();

  const float inv_d = 1.0f / static_cast<float>(a.D);
#pragma unroll 1
  for (int i = slot; i - slot < total; i += kSlots) {
    const uint4 x0v = v0, x1v = v1;
    const int kk = k, hh = h;
    h += kSlots;
    while (h >= H) {
      h -= H;
      ++k;
    }
    if (i + kSlots < total && mine) {
      const uint16_t* p = source(a, t0 + k, h);
      v0 = *reinterpret_cast<const uint4*>(p + c.c0);
      v1 = *reinterpret_cast<const uint4*>(p + c.c1);
    }
    float x0[8], x1[8];
    unpack8(x0v, x0);
    unpack8(x1v, x1);
    float ss = 0.0f, st = 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      ss = fmaf(x0[u], x0[u], ss);
      st = fmaf(x1[u], x1[u], st);
    }
    const float r = rsqrtf(fmaf(lane_sum<kLanes>(ss + st), inv_d, n.eps));
    if (i >= total || !mine) continue;
    const int64_t page = tok[kk].page;
    if (page < 0) continue;
    uint16_t* out = target(a, t0 + kk, hh, page);
    if (hh >= a.Hq + a.Hk) {         // a value: as it is
      *reinterpret_cast<uint4*>(out + c.c0) = x0v;
      *reinterpret_cast<uint4*>(out + c.c1) = x1v;
      continue;
    }
    float w0[8], w1[8];
    load_weights(weights + (hh < a.Hq ? 0 : a.D), c, w0, w1);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      x0[u] *= r * w0[u];
      x1[u] *= r * w1[u];
    }
    turn(c, a.interleaved, cs + kk * half, x0, x1);
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
  prepare_tokens(a, t, 1, tok, cs);
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
    const float r = rsqrtf(lane_sum<32>(ss) / static_cast<float>(a.D) + n.eps);
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
__global__ void __launch_bounds__(kThreads, kBwdBlocks) norm_rope_bwd_kernel(const __grid_constant__ NormArgs n, int tb) {
  extern __shared__ __align__(16) float2 cs[];       // [token][pair], weights [2][D], sums [warps][D]
  __shared__ Token tok[kMaxTok];
  constexpr int kSlots = kThreads / kLanes;
  const RopeArgs& a = n.r;
  const int tid = threadIdx.x, half = a.rot >> 1, lane = tid & 31, warp = tid >> 5;
  float* weights = reinterpret_cast<float*>(cs + ((tb * half + 1) & ~1));
  float* sums = weights + 2 * a.D;
  const int slot = tid / kLanes, j = tid % kLanes;
  const bool mine = 16 * j < a.D;
  const Chunks c = chunks_of(a, j);
  for (int i = tid; i < 2 * a.D; i += kThreads) weights[i] = weight_of(n, i >= a.D, i >= a.D ? i - a.D : i);
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);

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
    float acc0[8], acc1[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) acc0[u] = acc1[u] = 0.0f;
#pragma unroll 1
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * tb; t0 < a.T; t0 += static_cast<int64_t>(gridDim.x) * tb) {
      const int nt = static_cast<int>(a.T - t0 < tb ? a.T - t0 : tb);
      const int total = nt * H;
      int k = 0, h = slot;
      while (h >= H) {
        h -= H;
        ++k;
      }
      uint4 g0v = none, g1v = none, x0v = none, x1v = none;
      if (slot < total && mine) {
        const uint16_t* p = dy + (t0 + k) * dys + h * a.D;
        g0v = *reinterpret_cast<const uint4*>(p + c.c0);
        g1v = *reinterpret_cast<const uint4*>(p + c.c1);
        p = x + (t0 + k) * xs + h * a.D;
        x0v = *reinterpret_cast<const uint4*>(p + c.c0);
        x1v = *reinterpret_cast<const uint4*>(p + c.c1);
      }
      __syncthreads();             // the last tokens' angles are no longer read
      prepare_tokens(a, t0, nt, tok, cs);
      __syncthreads();
#pragma unroll 1
      for (int i = slot; i - slot < total; i += kSlots) {
        float g0[8], g1[8], x0[8], x1[8];
        unpack8(g0v, g0);
        unpack8(g1v, g1);
        unpack8(x0v, x0);
        unpack8(x1v, x1);
        const int kk = k, hh = h;
        h += kSlots;
        while (h >= H) {
          h -= H;
          ++k;
        }
        if (i + kSlots < total && mine) {
          const uint16_t* p = dy + (t0 + k) * dys + h * a.D;
          g0v = *reinterpret_cast<const uint4*>(p + c.c0);
          g1v = *reinterpret_cast<const uint4*>(p + c.c1);
          p = x + (t0 + k) * xs + h * a.D;
          x0v = *reinterpret_cast<const uint4*>(p + c.c0);
          x1v = *reinterpret_cast<const uint4*>(p + c.c1);
        }
        const bool valid = i < total && mine;
        if (valid) turn(c, a.interleaved, cs + kk * half, g0, g1);
        float w0[8], w1[8];
        if (mine) {
          load_weights(weights + which * a.D, c, w0, w1);
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u) w0[u] = w1[u] = 0.0f;
        }
        float ss = 0.0f, su = 0.0f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          ss = fmaf(x0[u], x0[u], ss);
          ss = fmaf(x1[u], x1[u], ss);
          su = fmaf(g0[u] * w0[u], x0[u], su);
          su = fmaf(g1[u] * w1[u], x1[u], su);
        }
        ss = lane_sum<kLanes>(ss);
        su = lane_sum<kLanes>(su);
        if (!valid) continue;
        const float r = rsqrtf(fmaf(ss, inv_d, n.eps));
        const float m = r * r * su * inv_d;
        float d0[8], d1[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          acc0[u] = fmaf(g0[u], x0[u] * r, acc0[u]);
          acc1[u] = fmaf(g1[u], x1[u] * r, acc1[u]);
          d0[u] = r * (g0[u] * w0[u] - x0[u] * m);
          d1[u] = r * (g1[u] * w1[u] - x1[u] * m);
        }
        uint16_t* out = dx + (t0 + kk) * dxs + hh * a.D;
        *reinterpret_cast<uint4*>(out + c.c0) = pack8(d0);
        *reinterpret_cast<uint4*>(out + c.c1) = pack8(d1);
      }
    }
    if (n.partial == nullptr) continue;
    // the lanes of one column: within the warp, then the warps in order
#pragma unroll
    for (int u = 0; u < 8; ++u) {
#pragma unroll
      for (int off = 16; off >= kLanes; off >>= 1) {
        acc0[u] += __shfl_xor_sync(0xffffffffu, acc0[u], off);
        acc1[u] += __shfl_xor_sync(0xffffffffu, acc1[u], off);
      }
    }
    __syncthreads();               // (the sums of the queries are read)
    if (lane < kLanes && mine) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        sums[warp * a.D + c.c0 + u] = acc0[u];
        sums[warp * a.D + c.c1 + u] = acc1[u];
      }
    }
    __syncthreads();
    for (int d = tid; d < a.D; d += kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w * a.D + d];
      n.partial[(static_cast<int64_t>(blockIdx.x) * 2 + which) * a.D + d] = s;
    }
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
      prepare_tokens(a, t, 1, tok, cs);
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
        const float r = rsqrtf(lane_sum<32>(ss) / static_cast<float>(a.D) + n.eps);
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

// The blocks' partial rows summed in order: a block 32 columns, a warp every kWarps-th row.
__global__ void __launch_bounds__(kThreads) norm_rope_sum_kernel(const float* partial, int blocks, int D, float* dwq, float* dwk) {
  __shared__ float s[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = static_cast<int>(blockIdx.x) * 32 + lane;        // of [2][D]
  pdl_wait();
  float x = 0.0f;
  const bool want = col < 2 * D && (col < D ? dwq : dwk) != nullptr;
  if (want) {
#pragma unroll 8
    for (int b = warp; b < blocks; b += kWarps) x += __ldcg(partial + static_cast<int64_t>(b) * 2 * D + col);
  }
  s[warp][lane] = x;
  __syncthreads();
  if (warp > 0 || !want) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) x += s[w][lane];
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

// Tokens of a block at a time: the least with which its lanes are busiest in the last round of heads too, while
// that leaves every SM two rounds of blocks.
int tokens_of(int64_t T, int H, int lanes) {
  const int slots = kThreads / lanes;
  int best = 1;
  double most = 0.0;
  for (int tb = 1; tb <= kMaxTok && (tb == 1 || T / tb >= 2ll * kBlocks * num_sms()); tb *= 2) {
    const double busy = static_cast<double>(tb * H) / ((tb * H + slots - 1) / slots * slots);
    if (busy > most + 0.02) {
      most = busy;
      best = tb;
    }
  }
  return best;
}

size_t angles_bytes(const RopeArgs& a, int tb) { return static_cast<size_t>((tb * (a.rot / 2) + 1) & ~1) * sizeof(float2); }

}  // namespace

cudaError_t launch_norm_rope(const NormArgs& n, cudaStream_t s) {
  const RopeArgs& a = n.r;
  const int lanes = lanes_of(n);
  if (lanes == 0) {
    norm_rope_any_kernel<<<static_cast<unsigned>(a.T), kThreads, angles_bytes(a, 1), s>>>(n);
    return cudaGetLastError();
  }
  const int tb = tokens_of(a.T, a.Hq + a.Hk + (a.append ? a.Hk : 0), lanes);
  const unsigned grid = static_cast<unsigned>((a.T + tb - 1) / tb);
  const size_t smem = angles_bytes(a, tb) + 2 * static_cast<size_t>(a.D) * sizeof(float);
  switch (lanes) {
    case 1: norm_rope_kernel<1><<<grid, kThreads, smem, s>>>(n, tb); break;
    case 2: norm_rope_kernel<2><<<grid, kThreads, smem, s>>>(n, tb); break;
    case 4: norm_rope_kernel<4><<<grid, kThreads, smem, s>>>(n, tb); break;
    case 8: norm_rope_kernel<8><<<grid, kThreads, smem, s>>>(n, tb); break;
    default: norm_rope_kernel<16><<<grid, kThreads, smem, s>>>(n, tb); break;
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
    norm_rope_bwd_any_kernel<<<grid, kThreads, angles_bytes(a, 1), s>>>(n);
  } else {
    const int tb = 1;
    const size_t smem = angles_bytes(a, tb) + (2 + kWarps) * static_cast<size_t>(a.D) * sizeof(float);
    switch (lanes) {
      case 1: norm_rope_bwd_kernel<1><<<grid, kThreads, smem, s>>>(n, tb); break;
      case 2: norm_rope_bwd_kernel<2><<<grid, kThreads, smem, s>>>(n, tb); break;
      case 4: norm_rope_bwd_kernel<4><<<grid, kThreads, smem, s>>>(n, tb); break;
      case 8: norm_rope_bwd_kernel<8><<<grid, kThreads, smem, s>>>(n, tb); break;
      default: norm_rope_bwd_kernel<16><<<grid, kThreads, smem, s>>>(n, tb); break;
    }
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || n.partial == nullptr) return e;
  return launch_after(norm_rope_sum_kernel, dim3(static_cast<unsigned>((2 * a.D + 31) / 32)), kThreads, 0, s,
                      static_cast<const float*>(n.partial), static_cast<int>(grid), a.D, dwq, dwk);
}

}  // namespace ls
