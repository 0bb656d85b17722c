// Host side of ls_policy_loss and ls_rope: argument checks and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/longstraw.h"
#include "ls_host.h"
#include "ls_internal.h"
#include "ls_ops.h"
#include "ls_rope_host.h"

using namespace ls;

namespace ls {

// Checks of the norm's part, and its arguments.
int head_norm_args(const ls_head_norm* n, NormArgs* a) {
  if (n == nullptr || !(n->eps > 0.0) || !std::isfinite(n->eps) || !std::isfinite(n->weight_offset) ||
      !(static_cast<float>(n->eps) > 0.0f) || !std::isfinite(static_cast<float>(n->weight_offset)))
    return LS_ERR_INVALID_ARGUMENT;
  if (!aligned_n(n->q_weight, n->weight_fp32 ? 4 : 2) || !aligned_n(n->k_weight, n->weight_fp32 ? 4 : 2))
    return LS_ERR_MISALIGNED;
  a->wq = n->q_weight;
  a->wk = n->k_weight;
  a->w_fp32 = n->weight_fp32 != 0;
  a->offset = static_cast<float>(n->weight_offset);
  a->eps = static_cast<float>(n->eps);
  return LS_OK;
}

}  // namespace ls

extern "C" {

size_t ls_policy_loss_workspace_bytes(int64_t T) {
  if (T < 1) return 0;
  return align_up(static_cast<size_t>(T) * sizeof(float2), 256) + kMaxPartials * sizeof(double) + 256;
}

ls_status ls_policy_loss(const ls_policy_loss_desc* d, void* workspace, size_t workspace_bytes,
                         void* stream) {
  NvtxRange nvtx_range("ls_policy_loss");
  if (d == nullptr || d->logits == nullptr || d->ids == nullptr || d->logp_old == nullptr ||
      d->advantages == nullptr || d->weights == nullptr || d->loss == nullptr ||
      d->dlogits == nullptr || d->clip_mask == nullptr)
    return LS_ERR_INVALID_ARGUMENT;
  if (d->T < 1 || d->V < 1 || d->logits_stride < d->V || d->dlogits_stride < d->V)
    return LS_ERR_INVALID_ARGUMENT;
  if (!(d->eps_low >= 0.0 && d->eps_low < 1.0) || !(d->eps_high >= 0.0) ||
      !std::isfinite(d->eps_high) || !std::isfinite(d->beta))
    return LS_ERR_INVALID_ARGUMENT;
  if (d->kl < LS_KL_NONE || d->kl > LS_KL_K3) return LS_ERR_INVALID_ARGUMENT;
  if (d->kl != LS_KL_NONE && d->logp_ref == nullptr) return LS_ERR_INVALID_ARGUMENT;
  if (d->logits == d->dlogits && d->logits_stride != d->dlogits_stride)
    return LS_ERR_INVALID_ARGUMENT;
  if (d->T >= (int64_t(1) << 31) || d->V >= (int64_t(1) << 31) ||
      d->logits_stride >= (int64_t(1) << 31) || d->dlogits_stride >= (int64_t(1) << 31))
    return LS_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < ls_policy_loss_workspace_bytes(d->T))
    return LS_ERR_WORKSPACE;
  if (!aligned_n(d->logits, 2) || !aligned_n(d->dlogits, 2) || !aligned_n(d->ids, 4) ||
      !aligned_n(d->logp_old, 4) || !aligned_n(d->logp_ref, 4) || !aligned_n(d->advantages, 4) ||
      !aligned_n(d->weights, 4) || !aligned_n(d->loss, 4) || !aligned_n(d->logp_out, 4) ||
      !aligned_n(d->kl_out, 4) || !aligned16(workspace))
    return LS_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  ls_status st = static_cast<ls_status>(enter_call(stream, &status));
  if (st != LS_OK) return st;
  PolicyArgs a{};
  a.T = d->T;
  a.V = d->V;
  a.ldx = d->logits_stride;
  a.ldd = d->dlogits_stride;
  a.logits = static_cast<const uint16_t*>(d->logits);
  a.ids = d->ids;
  a.old = d->logp_old;
  a.ref = d->kl == LS_KL_NONE ? nullptr : d->logp_ref;
  a.adv = d->advantages;
  a.weight = d->weights;
  a.clip_lo = 1.0 - d->eps_low;
  a.clip_hi = 1.0 + d->eps_high;
  const double lo = std::log(a.clip_lo), hi = std::log(a.clip_hi);
  a.log_lo[0] = static_cast<float>(lo);
  a.log_lo[1] = static_cast<float>(lo - a.log_lo[0]);
  a.log_hi[0] = static_cast<float>(hi);
  a.log_hi[1] = static_cast<float>(hi - a.log_hi[0]);
  a.beta = d->beta;
  a.kl = d->kl;
  a.loss = d->loss;
  a.dlogits = static_cast<uint16_t*>(d->dlogits);
  a.clip_mask = d->clip_mask;
  a.logp_out = d->logp_out;
  a.kl_out = d->kl_out;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.logp_pair = reinterpret_cast<float2*>(ws);
  ws += align_up(static_cast<size_t>(d->T) * sizeof(float2), 256);
  a.partial = reinterpret_cast<double*>(ws);
  a.counter = reinterpret_cast<unsigned*>(ws + kMaxPartials * sizeof(double));
  a.status = status;
  a.wait_ns = wait_limit_ns();
  cudaError_t e;
  {
    LaunchTimer t(LS_KERNEL_POLICY_LOSS, static_cast<cudaStream_t>(stream));
    e = injected_failure() ? cudaErrorLaunchFailure
                           : launch_policy_loss(a, static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? LS_OK : static_cast<ls_status>(launch_failed(e, "policy loss launch"));
}

// 1 / temperature and log2 e / temperature are fp32 factors: neither may pass its range, 0 x -inf would be NaN.
static bool temperature_ok(double t) { return t >= 0x1p-120 && t <= 0x1p120; }

ls_status ls_token_scores(const ls_token_scores_desc* d, void* stream) {
  NvtxRange nvtx_range("ls_token_scores");
  if (d == nullptr || d->logits == nullptr || d->ids == nullptr || d->logp == nullptr) return LS_ERR_INVALID_ARGUMENT;
  if (d->T < 1 || d->V < 1 || d->logits_stride < d->V || d->top < 0 || d->top > d->V) return LS_ERR_INVALID_ARGUMENT;
  if (!temperature_ok(d->temperature)) return LS_ERR_INVALID_ARGUMENT;
  if (d->top > 0 && (d->top_ids == nullptr || d->top_logp == nullptr)) return LS_ERR_INVALID_ARGUMENT;
  if (d->top > kMaxTop || (d->top > 0 && d->V > kMaxScoresVocab) || d->T >= (int64_t(1) << 28) ||
      d->V >= (int64_t(1) << 31) || d->logits_stride >= (int64_t(1) << 31))
    return LS_ERR_UNSUPPORTED;
  if (!aligned_n(d->logits, 2) || !aligned_n(d->ids, 4) || !aligned_n(d->logp, 4) || !aligned_n(d->lse, 4) ||
      !aligned_n(d->entropy, 4) || !aligned_n(d->top_ids, 4) || !aligned_n(d->top_logp, 4))
    return LS_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  ls_status st = static_cast<ls_status>(enter_call(stream, &status));
  if (st != LS_OK) return st;
  ScoresArgs a{};
  a.T = d->T;
  a.V = d->V;
  a.ldx = d->logits_stride;
  a.logits = static_cast<const uint16_t*>(d->logits);
  a.ids = d->ids;
  a.scale = 1.0 / d->temperature;
  a.scale2 = static_cast<float>(1.4426950408889634074 / d->temperature);
  a.top = d->top;
  a.logp = d->logp;
  a.lse = d->lse;
  a.entropy = d->entropy;
  a.top_ids = d->top_ids;
  a.top_logp = d->top_logp;
  a.status = status;
  cudaError_t e;
  {
    LaunchTimer t(LS_KERNEL_TOKEN_LOGP, static_cast<cudaStream_t>(stream));
    e = injected_failure() ? cudaErrorLaunchFailure : launch_scores(a, static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? LS_OK : static_cast<ls_status>(launch_failed(e, "token scores launch"));
}

ls_status ls_token_scores_bwd(const ls_token_scores_bwd_desc* d, void* stream) {
  NvtxRange nvtx_range("ls_token_scores_bwd");
  if (d == nullptr || d->logits == nullptr || d->ids == nullptr || d->logp == nullptr || d->lse == nullptr ||
      d->dlogits == nullptr)
    return LS_ERR_INVALID_ARGUMENT;
  if (d->d_logp == nullptr && d->d_entropy == nullptr) return LS_ERR_INVALID_ARGUMENT;
  if (d->d_entropy != nullptr && d->entropy == nullptr) return LS_ERR_INVALID_ARGUMENT;
  if (d->T < 1 || d->V < 1 || d->logits_stride < d->V || d->dlogits_stride < d->V) return LS_ERR_INVALID_ARGUMENT;
  if (!temperature_ok(d->temperature)) return LS_ERR_INVALID_ARGUMENT;
  if (d->logits == d->dlogits && d->logits_stride != d->dlogits_stride) return LS_ERR_INVALID_ARGUMENT;
  if (d->T >= (int64_t(1) << 28) || d->V >= (int64_t(1) << 31) || d->logits_stride >= (int64_t(1) << 31) ||
      d->dlogits_stride >= (int64_t(1) << 31))
    return LS_ERR_UNSUPPORTED;
  if (!aligned_n(d->logits, 2) || !aligned_n(d->dlogits, 2) || !aligned_n(d->ids, 4) || !aligned_n(d->logp, 4) ||
      !aligned_n(d->lse, 4) || !aligned_n(d->entropy, 4) || !aligned_n(d->d_logp, 4) || !aligned_n(d->d_entropy, 4))
    return LS_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  ls_status st = static_cast<ls_status>(enter_call(stream, &status));
  if (st != LS_OK) return st;
  ScoresBwdArgs a{};
  a.T = d->T;
  a.V = d->V;
  a.ldx = d->logits_stride;
  a.ldd = d->dlogits_stride;
  a.logits = static_cast<const uint16_t*>(d->logits);
  a.ids = d->ids;
  a.logp = d->logp;
  a.lse = d->lse;
  a.entropy = d->entropy;
  a.d_logp = d->d_logp;
  a.d_entropy = d->d_entropy;
  const int lift = std::max(std::ilogb(1.0 / d->temperature), 0);
  a.scale = static_cast<float>(std::ldexp(1.0 / d->temperature, -lift));
  a.lift = static_cast<float>(lift);
  a.lifted = std::ldexp(1.0f, lift);
  a.scale2 = static_cast<float>(1.4426950408889634074 / d->temperature);
  a.dlogits = static_cast<uint16_t*>(d->dlogits);
  a.status = status;
  cudaError_t e;
  {
    LaunchTimer t(LS_KERNEL_TOKEN_LOGP, static_cast<cudaStream_t>(stream));
    e = injected_failure() ? cudaErrorLaunchFailure : launch_scores_bwd(a, static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? LS_OK : static_cast<ls_status>(launch_failed(e, "token scores gradient launch"));
}

}  // extern "C"

namespace {

// The checks of a rotation, and its arguments but the status word; alone: without a rotation (rot_dim 0 and no
// frequencies) there is something left to do.
ls_status rope_args(const ls_rope_desc* d, bool alone, RopeArgs* out) {
  if (d == nullptr) return LS_ERR_INVALID_ARGUMENT;
  const bool turns = !alone || d->inv_freq != nullptr;
  if (turns && d->inv_freq == nullptr) return LS_ERR_INVALID_ARGUMENT;
  if (d->T < 1 || d->Hq < 0 || d->Hk < 0 || d->Hq + d->Hk < 1) return LS_ERR_INVALID_ARGUMENT;
  if (d->Hq > 65536 || d->Hk > 65536 || d->T >= (int64_t(1) << 31)) return LS_ERR_UNSUPPORTED;
  if (d->D < 2 || d->D > 2 * kMaxRot || d->D % 2 != 0) return LS_ERR_UNSUPPORTED;
  if (turns ? (d->rot_dim < 2 || d->rot_dim > d->D || d->rot_dim % 2 != 0) : d->rot_dim != 0) return LS_ERR_INVALID_ARGUMENT;
  if ((d->Hq > 0 && (d->q == nullptr || d->q_out == nullptr)) ||
      (d->Hk > 0 && (d->k == nullptr || d->k_out == nullptr)))
    return LS_ERR_INVALID_ARGUMENT;
  const int64_t nq = static_cast<int64_t>(d->Hq) * d->D, nk = static_cast<int64_t>(d->Hk) * d->D;
  if ((d->Hq > 0 && (d->q_stride < nq || d->q_out_stride < nq)) ||
      (d->Hk > 0 && (d->k_stride < nk || d->k_out_stride < nk)))
    return LS_ERR_INVALID_ARGUMENT;
  if ((d->Hq > 0 && d->q == d->q_out && d->q_stride != d->q_out_stride) ||
      (d->Hk > 0 && d->k == d->k_out && d->k_stride != d->k_out_stride))
    return LS_ERR_INVALID_ARGUMENT;
  if (!aligned_n(d->q, 2) || !aligned_n(d->q_out, 2) || !aligned_n(d->k, 2) ||
      !aligned_n(d->k_out, 2) || !aligned_n(d->positions, 8))
    return LS_ERR_MISALIGNED;
  RopeArgs& a = *out;
  if (turns && !rope_turns(d->inv_freq, d->rot_dim, d->attn_factor, &a)) return LS_ERR_INVALID_ARGUMENT;
  a.T = d->T;
  a.Hq = d->Hq;
  a.Hk = d->Hk;
  a.D = d->D;
  a.interleaved = d->interleaved != 0;
  a.inverse = d->inverse != 0;
  a.positions = d->positions;
  a.pos0 = d->pos0;
  a.q = static_cast<const uint16_t*>(d->q);
  a.qs = d->q_stride;
  a.qo = static_cast<uint16_t*>(d->q_out);
  a.qos = d->q_out_stride;
  a.k = static_cast<const uint16_t*>(d->k);
  a.ks = d->k_stride;
  a.ko = static_cast<uint16_t*>(d->k_out);
  a.kos = d->k_out_stride;
  return LS_OK;
}

}  // namespace

extern "C" {

ls_status ls_rope(const ls_rope_desc* d, void* stream) {
  NvtxRange nvtx_range("ls_rope");
  RopeArgs a{};
  ls_status st = rope_args(d, false, &a);
  if (st != LS_OK) return st;
  uint32_t* status = nullptr;
  st = static_cast<ls_status>(enter_call(stream, &status));
  if (st != LS_OK) return st;
  a.status = status;
  cudaError_t e;
  {
    LaunchTimer t(LS_KERNEL_ROPE, static_cast<cudaStream_t>(stream));
    e = injected_failure() ? cudaErrorLaunchFailure : launch_rope(a, static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? LS_OK : static_cast<ls_status>(launch_failed(e, "rotary launch"));
}

ls_status ls_norm_rope(const ls_rope_desc* d, const ls_head_norm* n, void* stream) {
  NvtxRange nvtx_range("ls_norm_rope");
  NormArgs a{};
  if (d != nullptr && d->inverse != 0) return LS_ERR_INVALID_ARGUMENT;
  ls_status st = rope_args(d, true, &a.r);
  if (st == LS_OK) st = static_cast<ls_status>(head_norm_args(n, &a));
  if (st != LS_OK) return st;
  uint32_t* status = nullptr;
  st = static_cast<ls_status>(enter_call(stream, &status));
  if (st != LS_OK) return st;
  a.r.status = status;
  cudaError_t e;
  {
    LaunchTimer t(LS_KERNEL_ROPE, static_cast<cudaStream_t>(stream));
    e = injected_failure() ? cudaErrorLaunchFailure : launch_norm_rope(a, static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? LS_OK : static_cast<ls_status>(launch_failed(e, "norm and rotary launch"));
}

size_t ls_norm_rope_bwd_workspace_bytes(int64_t T, int32_t D) {
  if (T < 1 || D < 2 || D > 2 * kMaxRot) return 0;
  return align_up(static_cast<size_t>(norm_rope_bwd_blocks(T)) * 2 * D * sizeof(float), 256);
}

ls_status ls_norm_rope_bwd(const ls_rope_desc* d, const ls_head_norm* n, const ls_head_norm_grad* g, void* workspace,
                           size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("ls_norm_rope_bwd");
  NormArgs a{};
  if (g == nullptr || (d != nullptr && d->inverse != 0)) return LS_ERR_INVALID_ARGUMENT;
  ls_status st = rope_args(d, true, &a.r);
  if (st == LS_OK) st = static_cast<ls_status>(head_norm_args(n, &a));
  if (st != LS_OK) return st;
  if ((d->Hq > 0 && (g->q_in == nullptr || g->q_in_stride < static_cast<int64_t>(d->Hq) * d->D)) ||
      (d->Hk > 0 && (g->k_in == nullptr || g->k_in_stride < static_cast<int64_t>(d->Hk) * d->D)))
    return LS_ERR_INVALID_ARGUMENT;
  // (a weight's gradient is of heads that are there)
  if ((d->Hq == 0 && g->dq_weight != nullptr) || (d->Hk == 0 && g->dk_weight != nullptr)) return LS_ERR_INVALID_ARGUMENT;
  const bool sums = g->dq_weight != nullptr || g->dk_weight != nullptr;
  if (sums && (workspace == nullptr || workspace_bytes < ls_norm_rope_bwd_workspace_bytes(d->T, d->D)))
    return LS_ERR_WORKSPACE;
  if (!aligned_n(g->q_in, 2) || !aligned_n(g->k_in, 2) || !aligned_n(g->dq_weight, 4) || !aligned_n(g->dk_weight, 4) ||
      (sums && !aligned16(workspace)))
    return LS_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  st = static_cast<ls_status>(enter_call(stream, &status));
  if (st != LS_OK) return st;
  a.r.inverse = 1;
  a.r.status = status;
  a.xq = static_cast<const uint16_t*>(g->q_in);
  a.xqs = g->q_in_stride;
  a.xk = static_cast<const uint16_t*>(g->k_in);
  a.xks = g->k_in_stride;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  cudaError_t e;
  {
    LaunchTimer t(LS_KERNEL_ROPE, static_cast<cudaStream_t>(stream));
    e = injected_failure() ? cudaErrorLaunchFailure
                           : launch_norm_rope_bwd(a, g->dq_weight, g->dk_weight, static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? LS_OK : static_cast<ls_status>(launch_failed(e, "norm and rotary gradient launch"));
}

ls_status ls_rope_freqs(int32_t rot_dim, double theta, int32_t scaling, double factor,
                        int64_t orig_len, double beta_fast, double beta_slow, double* inv_freq,
                        double* attn_factor) {
  if (inv_freq == nullptr || attn_factor == nullptr) return LS_ERR_INVALID_ARGUMENT;
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 2 * kMaxRot) return LS_ERR_INVALID_ARGUMENT;
  if (!(theta > 1.0) || !std::isfinite(theta)) return LS_ERR_INVALID_ARGUMENT;
  if (scaling < LS_ROPE_NONE || scaling > LS_ROPE_RAMP) return LS_ERR_INVALID_ARGUMENT;
  if (scaling != LS_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return LS_ERR_INVALID_ARGUMENT;
  double lo = 0.0, hi = 1.0;
  if (scaling == LS_ROPE_RAMP) {
    if (orig_len < 1 || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) || !std::isfinite(beta_fast))
      return LS_ERR_INVALID_ARGUMENT;
    // index of the pair that turns `beta` times over orig_len tokens
    const double two_pi = 6.283185307179586476925;
    const double per = rot_dim / (2.0 * std::log(theta));
    lo = std::floor(per * std::log(orig_len / (beta_fast * two_pi)));
    hi = std::ceil(per * std::log(orig_len / (beta_slow * two_pi)));
    if (lo < 0.0) lo = 0.0;
    if (hi > rot_dim - 1.0) hi = rot_dim - 1.0;
    if (hi - lo < 1e-3) hi = lo + 1e-3;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(theta, -2.0 * i / rot_dim);
    if (scaling == LS_ROPE_NONE) {
      inv_freq[i] = f;
    } else if (scaling == LS_ROPE_LINEAR) {
      inv_freq[i] = f / factor;
    } else {
      double r = (i - lo) / (hi - lo);
      r = r < 0.0 ? 0.0 : (r > 1.0 ? 1.0 : r);
      inv_freq[i] = f * (1.0 - r) + f / factor * r;
    }
  }
  *attn_factor = scaling == LS_ROPE_RAMP ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return LS_OK;
}

}  // extern "C"
