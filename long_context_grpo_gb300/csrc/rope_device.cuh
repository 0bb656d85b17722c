// Device pieces shared by the rotary kernels: bf16 values, the place of an appended token, the angles.
#pragma once

#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"

namespace ls {

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

// Cosine and sine of pair p at a position, with the factor (and the sign of the inverse).
__device__ __forceinline__ float2 angle_of(const RopeArgs& a, int64_t pos, int p) {
  const uint64_t turn = static_cast<uint64_t>(pos) * a.turns[p];
  // fraction of a turn in [-1/2, 1/2) -> half turns
  const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c * a.factor, (a.inverse ? -s : s) * a.factor);
}

}  // namespace ls
