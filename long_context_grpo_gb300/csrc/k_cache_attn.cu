// Attention of packed new tokens over the cache's pages.
//
//   o = softmax(s q K^T) V over the keys 0 .. position of the token's own sequence,
//   lse = log sum exp(s q k)
//
// One warp per (new token, query head): a pass over the keys with the running maximum and sum in
// fp32, a key's dot product summed over the warp.
#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"

namespace ls {
namespace {

constexpr int kThreads = 256;

template <int D>
__global__ void __launch_bounds__(kThreads) cache_attn_warp(const __grid_constant__ CacheAttnArgs a) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5);
  if (item >= a.T * a.c.Hq) return;
  const int64_t t = item / a.c.Hq;
  const int h = static_cast<int>(item - t * a.c.Hq);
  int b = 0;
  for (int i = lane; i < a.S; i += 32) b += (a.cu[i + 1] <= t) ? 1 : 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) b += __shfl_xor_sync(0xffffffffu, b, off);
  if (b >= a.S || t < a.cu[b]) return;
  const int row = a.rows != nullptr ? a.rows[b] : b;
  const int n = a.cu[b + 1] - a.cu[b];
  int64_t len = 0;
  bool bad = row < 0 || row >= a.c.num_rows || n > a.max_new;
  if (!bad) {
    len = a.c.len[row];
    bad = len < 0 || len > a.max_len || len > (static_cast<int64_t>(a.c.width) << a.c.ps_log2);
  }
  if (bad && lane == 0) set_device_status(a.status, DEV_BAD_INDEX);
  const int64_t keys = bad ? 0 : len - (a.cu[b + 1] - t) + 1;
  const int kv = h / (a.c.Hq / a.c.Hkv);
  const int ps = 1 << a.c.ps_log2;
  float q[kPer], acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = __uint_as_float(static_cast<uint32_t>(a.q[t * a.qs + h * D + lane + 32 * i]) << 16);
    acc[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t k0 = 0; k0 < keys; k0 += ps) {
    const int page = a.c.table[static_cast<int64_t>(row) * a.c.width + (k0 >> a.c.ps_log2)];
    const bool in = page >= 0 && page < a.c.num_pages;
    if (!in && lane == 0) set_device_status(a.status, DEV_BAD_INDEX);
    const int64_t base = (in ? page : 0) * a.c.page_stride + kv * a.c.head_stride;
    const int cnt = keys - k0 < ps ? static_cast<int>(keys - k0) : ps;
    for (int j = 0; j < cnt; ++j) {
      const int64_t at = base + j * a.c.tok_stride + lane;
      float d = 0.0f, v[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        v[i] = 0.0f;
        if (in) {
          d = fmaf(q[i], __uint_as_float(static_cast<uint32_t>(a.c.k[at + 32 * i]) << 16), d);
          v[i] = __uint_as_float(static_cast<uint32_t>(a.c.v[at + 32 * i]) << 16);
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
      d *= a.scale;
      const float mn = fmaxf(m, d);
      const float f = mn == -INFINITY ? 1.0f : expf(m - mn), p = mn == -INFINITY ? 0.0f : expf(d - mn);
      m = mn;
      l = l * f + p;
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] = fmaf(acc[i], f, p * v[i]);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    a.o[(t * a.c.Hq + h) * D + lane + 32 * i] =
        static_cast<uint16_t>(pack_bf16x2(acc[i] * inv, 0.0f) & 0xFFFFu);
  if (lane == 0) a.lse[t * a.c.Hq + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t cache_attn_ws_bytes(const CacheView&, int, int64_t, int, int64_t) { return 256; }

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.T * a.c.Hq + kThreads / 32 - 1) / (kThreads / 32));
  if (a.c.D == 128)
    cache_attn_warp<128><<<grid, kThreads, 0, s>>>(a);
  else
    cache_attn_warp<64><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ls
