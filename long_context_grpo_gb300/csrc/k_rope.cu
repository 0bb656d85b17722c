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
// Bound by HBM: 2 bytes read and 2 written a value (14,000 tokens appended: 89 us, 6.3 TB/s; 3,001
// tokens of 48 heads turned: 22.5 us if they are not in L2, 17 if they are, in two and a half waves
// of blocks).  Vector path: 16-byte accesses; a thread
// keeps its place in the head and walks the heads of the block's tokens (two or four accesses in
// flight a thread, with fewer blocks an SM, measured slower: 98 us and more against 92).
// Element path for rows that are not 16-byte aligned or rot_dim not a multiple of 16 (8
// interleaved).
#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"

namespace ls {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 2;      // tokens of a block at most
constexpr int kBlocks = 8;      // blocks of an SM

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
  // the entry of row t: the number of entries that end at or before it (lower half); and the
  // number of offsets that fall or leave 0 .. T (upper half), with which the count means nothing
  int b = 0;
  for (int i = lane; i < a.S; i += 32) {
    const int start = a.cu[i], end = a.cu[i + 1];
    b += end <= t ? 1 : 0;
    if (end < start || end > a.T || start < 0) b += 1 << 16;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) b += __shfl_xor_sync(0xffffffffu, b, off);
  if (b >= 1 << 16) {
    if (lane == 0) set_device_status(a.status, DEV_BAD_INDEX);
    return r;
  }
  if (b >= a.S || t < a.cu[b]) return r;
  const int row = a.rows != nullptr ? a.rows[b] : b;
  if (row < 0 || row >= a.c.num_rows) {
    if (lane == 0) set_device_status(a.status, DEV_BAD_INDEX);
    return r;
  }
  const int64_t len = a.c.len[row];
  if (len < 0 || len > (static_cast<int64_t>(a.c.width) << a.c.ps_log2)) {
    if (lane == 0) set_device_status(a.status, DEV_BAD_INDEX);
    return r;
  }
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
template <bool kAppend>
__device__ __forceinline__ Place place_of(const RopeArgs& a, int64_t t, int h, int64_t page) {
  Place p;
  if (h < a.Hq) {
    p.src = a.q + t * a.qs + h * a.D;
    p.dst = a.qo + t * a.qos + h * a.D;
  } else if (!kAppend || h < a.Hq + a.Hk) {
    const int hk = h - a.Hq;
    p.src = a.k + t * a.ks + hk * a.D;
    p.dst = kAppend && a.append ? a.c.k + page + hk * a.c.head_stride : a.ko + t * a.kos + hk * a.D;
  } else {
    const int hk = h - a.Hq - a.Hk;
    p.src = a.v + t * a.vs + hk * a.D;
    p.dst = a.c.v + page + hk * a.c.head_stride;
  }
  return p;
}

// Walks the (token, head) pairs of a block, `step` heads at a time: no divisions in the loop.
struct Walk {
  int tok, head;
  __device__ __forceinline__ void next(int step, int H) {
    head += step;
    while (head >= H) {
      head -= H;
      ++tok;
    }
  }
};

// What a thread reads of one (token, head): a 16-byte chunk and, with kPair, its partner.
struct Chunk {
  uint4 x, y;
};
template <bool kPair>
__device__ __forceinline__ void load_chunk(Chunk* v, const uint16_t* src, int partner) {
  v->x = *reinterpret_cast<const uint4*>(src);
  if constexpr (kPair) v->y = *reinterpret_cast<const uint4*>(src + partner);
}

// One 16-byte chunk (kPair: chunk c of the first half with its partner in the second) of the heads
// that this thread walks.  kTurn: rotated by the chunk's angles; else copied.  kLoaded: v is the
// first of them, loaded by first_chunk before the angles were there.
template <bool kPair>
__device__ __forceinline__ void first_chunk(Chunk* v, const RopeArgs& a, int64_t t0, int nt, int h_first, int h_count,
                                            int c, int partner, int first) {
  Walk w = {0, first};
  w.next(0, h_count);
  if (w.tok < nt) load_chunk<kPair>(v, place_of<false>(a, t0 + w.tok, h_first + w.head, 0).src + c, partner);
}
template <bool kTurn, bool kPair, bool kLoaded>
__device__ __forceinline__ void chunks(Chunk ahead, const RopeArgs& a, const Token* tok, const float2* cs, int64_t t0, int nt,
                                       int h_first, int h_count, int c, int partner, int first, int step) {
  const int half = a.rot >> 1;
  bool loaded = kLoaded;
  Walk w = {0, first};
  for (w.next(0, h_count); w.tok < nt; w.next(step, h_count)) {
    const bool have = loaded;
    loaded = false;
    const int64_t page = kLoaded ? 0 : tok[w.tok].page;     // (an append's; it loads nothing ahead)
    if (page < 0) continue;
    const Place p = place_of<!kLoaded>(a, t0 + w.tok, h_first + w.head, page);
    if (!kTurn && p.src == p.dst) continue;
    if (!have) load_chunk<kPair>(&ahead, p.src + c, partner);
    const Chunk& v = ahead;
    const uint4 x = v.x;
    if constexpr (!kTurn) {
      *reinterpret_cast<uint4*>(p.dst + c) = x;
    } else if constexpr (kPair) {
      const uint4 y = v.y;
      const float4* t = reinterpret_cast<const float4*>(cs + w.tok * half + c);
      const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
      uint32_t ox[4], oy[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4 r = t[u];        // cos, sin of two pairs
        const float x0 = bf(wx[u], 0), x1 = bf(wx[u], 1), y0 = bf(wy[u], 0), y1 = bf(wy[u], 1);
        ox[u] = pack_bf16x2(x0 * r.x - y0 * r.y, x1 * r.z - y1 * r.w);
        oy[u] = pack_bf16x2(y0 * r.x + x0 * r.y, y1 * r.z + x1 * r.w);
      }
      *reinterpret_cast<uint4*>(p.dst + c) = make_uint4(ox[0], ox[1], ox[2], ox[3]);
      *reinterpret_cast<uint4*>(p.dst + c + partner) = make_uint4(oy[0], oy[1], oy[2], oy[3]);
    } else {
      const float4* t = reinterpret_cast<const float4*>(cs + w.tok * half + (c >> 1));
      const uint32_t wx[4] = {x.x, x.y, x.z, x.w};
      uint32_t o[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 r = t[u];
        const float x0 = bf(wx[2 * u], 0), y0 = bf(wx[2 * u], 1), x1 = bf(wx[2 * u + 1], 0), y1 = bf(wx[2 * u + 1], 1);
        o[2 * u] = pack_bf16x2(x0 * r.x - y0 * r.y, y0 * r.x + x0 * r.y);
        o[2 * u + 1] = pack_bf16x2(x1 * r.z - y1 * r.w, y1 * r.z + x1 * r.w);
      }
      *reinterpret_cast<uint4*>(p.dst + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <bool kVec, bool kAhead>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_kernel(const __grid_constant__ RopeArgs a, int tb) {
  extern __shared__ __align__(16) float2 cs[];      // [token][pair]: cosine, sine
  __shared__ Token tok[kMaxTok];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = a.rot >> 1;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tb;
  const int nt = static_cast<int>(a.T - t0 < tb ? a.T - t0 : tb);

  // A thread keeps its chunk of a head and walks the heads: rotated chunks (pairs of them in
  // the half layout) and the copied rest of the rotated heads, then the heads that are copied.
  // With kAhead the first chunk is on its way while the angles are computed (3,001 tokens that
  // are not in L2: 22.5 us, without 24.6; an append reads the page table first and gains nothing:
  // 92 us, without 91).
  Chunk v = {};
  if constexpr (kAhead) {
    const int nr = a.interleaved ? a.rot / 8 : a.rot / 16;
    const int per = nr + (a.D - a.rot) / 8;
    const int groups = kThreads / per, first = tid / per, j = tid - first * per;
    const int Hr = a.Hq + a.Hk;
    if (first < groups) {
      if (j >= nr)
        first_chunk<false>(&v, a, t0, nt, 0, Hr, a.rot + 8 * (j - nr), 0, first);
      else if (a.interleaved)
        first_chunk<false>(&v, a, t0, nt, 0, Hr, 8 * j, 0, first);
      else
        first_chunk<true>(&v, a, t0, nt, 0, Hr, 8 * j, half, first);
    }
  }

  if (!kAhead && a.append) {              // (an append loads nothing ahead)
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
    cs[i] = make_float2(c * a.factor, (a.inverse ? -s : s) * a.factor);
  }
  __syncthreads();

  const int H = a.Hq + a.Hk + (!kAhead && a.append ? a.Hk : 0);
  const int Hr = kAhead || a.rot > 0 ? a.Hq + a.Hk : 0;       // heads that are rotated
  if constexpr (kVec) {
    const int nr = a.interleaved ? a.rot / 8 : a.rot / 16;
    const int per = nr + (a.D - a.rot) / 8;
    if (Hr > 0) {
      const int groups = kThreads / per, first = tid / per, j = tid - first * per;
      if (first < groups) {
        if (j >= nr)
          chunks<false, false, kAhead>(v, a, tok, cs, t0, nt, 0, Hr, a.rot + 8 * (j - nr), 0, first, groups);
        else if (a.interleaved)
          chunks<true, false, kAhead>(v, a, tok, cs, t0, nt, 0, Hr, 8 * j, 0, first, groups);
        else
          chunks<true, true, kAhead>(v, a, tok, cs, t0, nt, 0, Hr, 8 * j, half, first, groups);
      }
    }
    if (!kAhead && H > Hr) {
      const int n8 = a.D / 8;
      const int groups = kThreads / n8, first = tid / n8, j = tid - first * n8;
      if (first < groups) chunks<false, false, false>(v, a, tok, cs, t0, nt, Hr, H - Hr, 8 * j, 0, first, groups);
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
        const Place p = place_of<true>(a, t0 + k, h, page);
        const int ix = a.interleaved ? 2 * c : c, iy = a.interleaved ? 2 * c + 1 : c + half;
        const float2 t = cs[k * half + c];
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
      const Place p = place_of<true>(a, t0 + k, h, page);
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
  // two tokens share a block's prologue once that leaves four waves of blocks (14,000 tokens
  // appended: 92 us, with one 103; 3,000 rotated: 19 us either way)
  const int64_t tb = a.T >= static_cast<int64_t>(num_sms()) * kBlocks * 4 * kMaxTok ? kMaxTok : 1;
  const unsigned grid = static_cast<unsigned>((a.T + tb - 1) / tb);
  const size_t smem = static_cast<size_t>(tb) * (a.rot / 2) * sizeof(float2);
  if (vec && !a.append)
    rope_kernel<true, true><<<grid, kThreads, smem, s>>>(a, static_cast<int>(tb));
  else if (vec)
    rope_kernel<true, false><<<grid, kThreads, smem, s>>>(a, static_cast<int>(tb));
  else
    rope_kernel<false, false><<<grid, kThreads, smem, s>>>(a, static_cast<int>(tb));
  return cudaGetLastError();
}

}  // namespace ls
