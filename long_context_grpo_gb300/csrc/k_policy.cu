// Clipped policy loss with a KL term over packed tokens, forward and backward.
//
// policy_rows: one CTA per token row at a time: maximum, sum of exponentials, the token's
//   scalar chain in fp64 by one thread, then dlogits = g (onehot - softmax).
// policy_reduce: the fp64 sum of the tokens' terms in a fixed order, rounded once.
#include "ls_internal.h"
#include "ls_ops.h"
#include "ptx.cuh"

namespace ls {
namespace {

constexpr int kThreads = 512;

__device__ __forceinline__ float bf16_at(const uint16_t* x, int64_t i) {
  return __uint_as_float(static_cast<uint32_t>(x[i]) << 16);
}

// What the softmax pass of a row needs, and the token's loss term.
struct TokenGrad {
  float g;          // d loss / d logp
  double term;
};

// The token's scalar chain in fp64, its outputs written (all but the gradient row).
__device__ __forceinline__ TokenGrad policy_token(const PolicyArgs& a, int64_t row, double logp) {
  const double A = a.adv[row], w = a.weight[row];
  const double d = logp - static_cast<double>(a.old[row]);
  const bool clipped = (A > 0.0 && d > a.log_hi) || (A < 0.0 && d < a.log_lo);
  const double rho_a = exp(d) * A;
  const double surr = clipped ? (A > 0.0 ? a.clip_hi : a.clip_lo) * A : rho_a;
  double kl = 0.0, slope = 0.0;
  if (a.ref != nullptr) {
    const double r = logp - static_cast<double>(a.ref[row]);
    if (a.kl == 1) {
      kl = r;
      slope = 1.0;
    } else if (a.kl == 2) {
      kl = 0.5 * r * r;
      slope = r;
    } else {
      const double em = expm1(-r);
      kl = em + r;
      slope = -em;
    }
  }
  TokenGrad t;
  t.term = w * (a.beta * kl - surr);
  t.g = static_cast<float>(w * (a.beta * slope - (clipped ? 0.0 : rho_a)));
  a.clip_mask[row] = clipped ? 1 : 0;
  if (a.logp_out != nullptr) a.logp_out[row] = static_cast<float>(logp);
  if (a.kl_out != nullptr) a.kl_out[row] = static_cast<float>(kl);
  return t;
}

// A token that is left out (weight 0, or an id outside the vocabulary): zeros.
__device__ __forceinline__ void policy_no_token(const PolicyArgs& a, int64_t row) {
  a.clip_mask[row] = 0;
  if (a.logp_out != nullptr) a.logp_out[row] = 0.0f;
  if (a.kl_out != nullptr) a.kl_out[row] = 0.0f;
  a.terms[row] = 0.0;
}

__global__ void __launch_bounds__(kThreads) policy_rows(const __grid_constant__ PolicyArgs a) {
  __shared__ float sh_m[kThreads / 32];
  __shared__ double sh_s[kThreads / 32];
  __shared__ float sh_g, sh_lse;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const uint16_t* x = a.logits + row * a.ldx;
    uint16_t* d = a.dlogits + row * a.ldd;
    const int y = a.ids[row];
    const bool used = a.weight[row] != 0.0f;
    if (!used || y < 0 || y >= a.V) {
      for (int64_t i = tid; i < a.V; i += kThreads) d[i] = 0;
      if (tid == 0) {
        if (used) set_device_status(a.status, DEV_BAD_INDEX);
        policy_no_token(a, row);
      }
      continue;
    }
    float m = -INFINITY;
    for (int64_t i = tid; i < a.V; i += kThreads) m = fmaxf(m, bf16_at(x, i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) sh_m[warp] = m;
    __syncthreads();
    m = sh_m[0];
    for (int w = 1; w < kThreads / 32; ++w) m = fmaxf(m, sh_m[w]);
    double s = 0.0;
    for (int64_t i = tid; i < a.V; i += kThreads) s += static_cast<double>(expf(bf16_at(x, i) - m));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) sh_s[warp] = s;
    __syncthreads();
    if (tid == 0) {
      s = 0.0;
      for (int w = 0; w < kThreads / 32; ++w) s += sh_s[w];
      const double lse = static_cast<double>(m) + log(s);
      const TokenGrad t = policy_token(a, row, static_cast<double>(bf16_at(x, y)) - lse);
      a.terms[row] = t.term;
      sh_g = t.g;
      sh_lse = static_cast<float>(log(s));
    }
    __syncthreads();
    const float g = sh_g, ls = sh_lse;
    for (int64_t i = tid; i < a.V; i += kThreads) {
      const float p = expf(bf16_at(x, i) - m - ls);
      d[i] = static_cast<uint16_t>(pack_bf16x2(g * ((i == y ? 1.0f : 0.0f) - p), 0.0f));
    }
    __syncthreads();
  }
}

constexpr int kReduceThreads = 1024;

__global__ void __launch_bounds__(kReduceThreads) policy_reduce(const double* terms, int64_t n,
                                                               float* loss) {
  __shared__ double sh[kReduceThreads];
  const int tid = threadIdx.x;
  double acc = 0.0;
  for (int64_t i = tid; i < n; i += kReduceThreads) acc += terms[i];
  sh[tid] = acc;
  __syncthreads();
  for (int w = kReduceThreads / 2; w > 0; w >>= 1) {
    if (tid < w) sh[tid] += sh[tid + w];
    __syncthreads();
  }
  if (tid == 0) *loss = static_cast<float>(sh[0]);
}

}  // namespace

cudaError_t launch_policy_loss(const PolicyArgs& a, cudaStream_t s) {
  int64_t grid = static_cast<int64_t>(num_sms()) * 4;
  if (grid > a.T) grid = a.T;
  policy_rows<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  policy_reduce<<<1, kReduceThreads, 0, s>>>(a.terms, a.T, a.loss);
  return cudaGetLastError();
}

}  // namespace ls
