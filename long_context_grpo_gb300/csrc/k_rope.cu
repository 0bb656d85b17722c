// Rotary positions of queries and keys (forward and gradient), and the append of new keys and
// values to a paged cache with the rotation on the way.
//
//   (x, y) -> f (x cos a - y sin a, y cos a + x sin a),   a = position * inv_freq[i]
//
// Angles: position * (inv_freq / 2 pi mod 1) as one 64-bit integer product modulo 2^64 is the
// exact fraction of a turn (the host rounds each fraction to 2^-64, so position 2^31 is off by
// 2^-33 turns); its top 32 bits give the angle in half turns for sincospi in fp32.  No fp64 and no
// range reduction on the device.  A block computes the cosines and sines of its tokens once, in
// shared memory, and every head of the token uses them.
//
// Bound by HBM: 2 bytes read and 2 written a value.  Vector path: 16-byte accesses, eight
// pairs of the half layout (or four interleaved ones) an item.  Element path for rows that are
// not 16-byte aligned or rot_dim not a multiple of 16 (8 interleaved).
#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"

namespace ls {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;      // tokens of a block

__device__ __forceinline__ float bf(uint32_t w, int hi) {
  return __uint_as_float(hi ? (w & 0xFFFF0000u) : (w << 16));
}
__device__ __forceinline__ uint16_t to_bf16(float x) {
  return static_cast<uint16_t>(pack_bf16x2(x, 0.0f) & 0xFFFFu);
}

struct Token {
  int64_t pos;
  int64_t page;     // element offset of the token's slot in the pages; -1: left out
};

// Position and page slot of packed row t of an append, found by the calling warp.
__device__ __forceinline__ Token locate(const RopeArgs& a, int64_t t, int lane) {
  Token r;
  r.pos = 0;
  r.page = -1;
  // the entry of row t: the number of entries that end at or before it
  int b = 0;
  for (int i = lane; i < a.S; i += 32) b += (a.cu[i + 1] <= t) ? 1 : 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) b += __shfl_xor_sync(0xffffffffu, b, off);
  if (b >= a.S || t < a.cu[b]) return r;
  const int row = a.rows != nullptr ? a.rows[b] : b;
  if (row < 0 || row >= a.c.num_rows) {
    if (lane == 0) set_device_status(a.status, DEV_BAD_INDEX);
    return r;
  }
  const int64_t len = a.c.len[row];
  r.pos = len - (a.cu[b + 1] - t);
  if (r.pos < 0) return r;
  const int64_t j = r.pos >> a.c.ps_log2;
  const int page = j < a.c.width ? a.c.table[static_cast<int64_t>(row) * a.c.width + j] : -1;
  if (page < 0 || page >= a.c.num_pages) {
    if (lane == 0) set_device_status(a.status, DEV_BAD_INDEX);
    return r;
  }
  const int64_t slot = r.pos & ((1 << a.c.ps_log2) - 1);
  r.page = page * a.c.page_stride + slot * a.c.tok_stride;
  return r;
}

// Where head h of block token i lives: source, destination and whether they are the same.
struct Place {
  const uint16_t* src;
  uint16_t* dst;
};
__device__ __forceinline__ Place place_of(const RopeArgs& a, int64_t t, int h, int64_t page) {
  Place p;
  if (h < a.Hq) {
    p.src = a.q + t * a.qs + h * a.D;
    p.dst = a.qo + t * a.qos + h * a.D;
  } else if (h < a.Hq + a.Hk) {
    const int hk = h - a.Hq;
    p.src = a.k + t * a.ks + hk * a.D;
    p.dst = a.append ? a.c.k + page + hk * a.c.head_stride : a.ko + t * a.kos + hk * a.D;
  } else {
    const int hk = h - a.Hq - a.Hk;
    p.src = a.v + t * a.vs + hk * a.D;
    p.dst = a.c.v + page + hk * a.c.head_stride;
  }
  return p;
}

template <bool kVec>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, int tb) {
  __shared__ float2 cs[kMaxTok][kMaxRot];
  __shared__ Token tok[kMaxTok];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = a.rot >> 1;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tb;
  const int nt = static_cast<int>(a.T - t0 < tb ? a.T - t0 : tb);

  if (a.append) {
    for (int i = warp; i < nt; i += kThreads / 32) {
      const Token r = locate(a, t0 + i, lane);
      if (lane == 0) tok[i] = r;
    }
  } else if (tid < nt) {
    tok[tid].pos = a.positions != nullptr ? a.positions[t0 + tid] : a.pos0 + t0 + tid;
    tok[tid].page = 0;
  }
  __syncthreads();
  for (int i = tid; i < nt * half; i += kThreads) {
    const int k = i / half, p = i - k * half;
    const uint64_t turn = static_cast<uint64_t>(tok[k].pos) * a.turns[p];
    // fraction of a turn in [-1/2, 1/2) -> half turns
    const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;
    float s, c;
    sincospif(x, &s, &c);
    cs[k][p] = make_float2(c * a.factor, (a.inverse ? -s : s) * a.factor);
  }
  __syncthreads();

  const int H = a.Hq + a.Hk + (a.append ? a.Hk : 0);
  const int Hr = a.rot > 0 ? a.Hq + a.Hk : 0;       // heads that are rotated
  if constexpr (kVec) {
    const int n8 = a.D / 8;
    const int nr = a.interleaved ? a.rot / 8 : a.rot / 16;
    const int per = Hr * (nr + (a.D - a.rot) / 8) + (H - Hr) * n8;
    for (int i = tid; i < nt * per; i += kThreads) {
      const int k = i / per;
      int j = i - k * per;
      const int64_t page = tok[k].page;
      if (page < 0) continue;
      const int rot_items = Hr * nr;
      if (j < rot_items) {
        const int h = j / nr, c = j - h * nr;
        const Place p = place_of(a, t0 + k, h, page);
        if (a.interleaved) {
          const uint4 v = *reinterpret_cast<const uint4*>(p.src + 8 * c);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 t = cs[k][4 * c + u];
            const float x = bf(w[u], 0), y = bf(w[u], 1);
            o[u] = pack_bf16x2(x * t.x - y * t.y, y * t.x + x * t.y);
          }
          *reinterpret_cast<uint4*>(p.dst + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          const uint4 vx = *reinterpret_cast<const uint4*>(p.src + 8 * c);
          const uint4 vy = *reinterpret_cast<const uint4*>(p.src + half + 8 * c);
          const uint32_t wx[4] = {vx.x, vx.y, vx.z, vx.w}, wy[4] = {vy.x, vy.y, vy.z, vy.w};
          uint32_t ox[4], oy[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 t0v = cs[k][8 * c + 2 * u], t1v = cs[k][8 * c + 2 * u + 1];
            const float x0 = bf(wx[u], 0), x1 = bf(wx[u], 1), y0 = bf(wy[u], 0), y1 = bf(wy[u], 1);
            ox[u] = pack_bf16x2(x0 * t0v.x - y0 * t0v.y, x1 * t1v.x - y1 * t1v.y);
            oy[u] = pack_bf16x2(y0 * t0v.x + x0 * t0v.y, y1 * t1v.x + x1 * t1v.y);
          }
          *reinterpret_cast<uint4*>(p.dst + 8 * c) = make_uint4(ox[0], ox[1], ox[2], ox[3]);
          *reinterpret_cast<uint4*>(p.dst + half + 8 * c) = make_uint4(oy[0], oy[1], oy[2], oy[3]);
        }
        continue;
      }
      j -= rot_items;
      // values behind the rotated part, then the heads that are only copied
      const int np = (a.D - a.rot) / 8;
      int h, c;
      if (j < Hr * np) {
        h = j / np;
        c = a.rot / 8 + (j - h * np);
      } else {
        j -= Hr * np;
        h = Hr + j / n8;
        c = j - (h - Hr) * n8;
      }
      const Place p = place_of(a, t0 + k, h, page);
      if (p.src != p.dst)
        *reinterpret_cast<uint4*>(p.dst + 8 * c) = *reinterpret_cast<const uint4*>(p.src + 8 * c);
    }
  } else {
    // element path: pair items, then single values
    const int per = Hr * (a.D - half) + (H - Hr) * a.D;
    for (int i = tid; i < nt * per; i += kThreads) {
      const int k = i / per;
      int j = i - k * per;
      const int64_t page = tok[k].page;
      if (page < 0) continue;
      if (j < Hr * half) {
        const int h = j / half, c = j - h * half;
        const Place p = place_of(a, t0 + k, h, page);
        const int ix = a.interleaved ? 2 * c : c, iy = a.interleaved ? 2 * c + 1 : c + half;
        const float2 t = cs[k][c];
        const float x = bf(p.src[ix], 0), y = bf(p.src[iy], 0);
        p.dst[ix] = to_bf16(x * t.x - y * t.y);
        p.dst[iy] = to_bf16(y * t.x + x * t.y);
        continue;
      }
      j -= Hr * half;
      const int np = a.D - a.rot;
      int h, c;
      if (j < Hr * np) {
        h = j / np;
        c = a.rot + (j - h * np);
      } else {
        j -= Hr * np;
        h = Hr + j / a.D;
        c = j - (h - Hr) * a.D;
      }
      const Place p = place_of(a, t0 + k, h, page);
      if (p.src != p.dst) p.dst[c] = p.src[c];
    }
  }
}

bool vec_ok(const void* p, int64_t stride) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0;
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  bool vec = a.D % 8 == 0 && (a.interleaved ? a.rot % 8 == 0 : a.rot % 16 == 0);
  if (a.Hq > 0) vec = vec && vec_ok(a.q, a.qs) && vec_ok(a.qo, a.qos);
  if (a.Hk > 0) vec = vec && vec_ok(a.k, a.ks);
  if (a.append)
    vec = vec && vec_ok(a.v, a.vs);   // pages are 16-byte aligned
  else if (a.Hk > 0)
    vec = vec && vec_ok(a.ko, a.kos);
  // a few tokens a block once there are enough of them to fill the GPU
  int tb = static_cast<int>(a.T / (static_cast<int64_t>(num_sms()) * 8));
  tb = tb < 1 ? 1 : (tb > kMaxTok ? kMaxTok : tb);
  const unsigned grid = static_cast<unsigned>((a.T + tb - 1) / tb);
  if (vec)
    rope_kernel<true><<<grid, kThreads, 0, s>>>(a, tb);
  else
    rope_kernel<false><<<grid, kThreads, 0, s>>>(a, tb);
  return cudaGetLastError();
}

}  // namespace ls
