// Host entry points of the post-training operators declared in
// include/flce.h: argument checks, workspace layout and launch sequence.
#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <cmath>

#include "flce.h"
#include "post_training.h"

using namespace flce;

namespace {

constexpr size_t kHeader = 256;   // status word at 0, finished-block counter at 8

size_t elem_bytes(int dtype) { return dtype == FLCE_F32 ? 4 : 2; }

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int refuse(int code, const char* msg) {
  set_error_detail(msg);
  return code;
}

int check_tokens(const flce_tokens& t) {
  const int64_t lim = int64_t(1) << 30;
  if (t.sequences < 0 || t.sequences > lim) return refuse(FLCE_ERR_INVALID_ARG, "sequences");
  if (t.packed != 0 && t.packed != 1) return refuse(FLCE_ERR_INVALID_ARG, "packed");
  if (t.packed) {
    if (t.tokens < 0 || t.tokens > 2147483647ll - 1024) return refuse(FLCE_ERR_INVALID_ARG, "tokens");
    if (t.cu_seqlens == nullptr) return refuse(FLCE_ERR_INVALID_ARG, "cu_seqlens is NULL");
    if (!aligned(t.cu_seqlens, 4)) return refuse(FLCE_ERR_ALIGNMENT, "cu_seqlens");
  } else {
    if (t.cols < 0 || (t.sequences > 0 && t.cols > (int64_t(1) << 40) / t.sequences))
      return refuse(FLCE_ERR_INVALID_ARG, "cols");
    if (t.cu_seqlens != nullptr) return refuse(FLCE_ERR_INVALID_ARG, "cu_seqlens without packed");
  }
  if (t.mask_kind < FLCE_MASK_NONE || t.mask_kind > FLCE_MASK_LABELS)
    return refuse(FLCE_ERR_INVALID_ARG, "mask_kind");
  return FLCE_OK;
}

int64_t token_total(const flce_tokens& t) { return t.packed ? t.tokens : t.sequences * t.cols; }

// A tensor laid out as the tokens.
int check_tensor(const flce_tokens& t, const void* p, int64_t ld, size_t elem, bool optional,
                 const char* name) {
  if (p == nullptr) {
    if (optional || token_total(t) == 0) return FLCE_OK;
    return refuse(FLCE_ERR_INVALID_ARG, name);
  }
  if (!aligned(p, elem)) return refuse(FLCE_ERR_ALIGNMENT, name);
  if (!t.packed && t.sequences > 1 && (ld < t.cols || ld > (int64_t(1) << 40)))
    return refuse(FLCE_ERR_INVALID_ARG, name);
  return FLCE_OK;
}

int check_mask(const flce_tokens& t) {
  if (t.mask_kind == FLCE_MASK_NONE)
    return t.mask == nullptr ? FLCE_OK : refuse(FLCE_ERR_INVALID_ARG, "mask without mask_kind");
  return check_tensor(t, t.mask, t.ld_mask, t.mask_kind == FLCE_MASK_LABELS ? 8 : 1, false, "mask");
}

TokenView view_of(const flce_tokens& t) {
  TokenView v{};
  v.S = t.sequences;
  v.cols = t.packed ? 0 : t.cols;
  v.N = token_total(t);
  v.cu = t.packed ? t.cu_seqlens : nullptr;
  v.mask = t.mask;
  v.ld_mask = t.ld_mask;
  v.ignore_index = t.ignore_index;
  v.mask_kind = t.mask_kind;
  return v;
}

// The elements that a strided token tensor spans.
size_t span(const flce_tokens& t, int64_t ld) {
  if (t.packed) return static_cast<size_t>(t.tokens);
  return t.sequences == 0 ? 0 : static_cast<size_t>((t.sequences - 1) * ld + t.cols);
}

int check_policy(const flce_policy_args* a) {
  if (a == nullptr) return refuse(FLCE_ERR_INVALID_ARG, "arguments are NULL");
  int v = check_tokens(a->tokens);
  if (v != FLCE_OK) return v;
  if (a->dtype < FLCE_F32 || a->dtype > FLCE_F16) return refuse(FLCE_ERR_INVALID_ARG, "dtype");
  if (a->reduction != FLCE_TOKEN_SUM && a->reduction != FLCE_TOKEN_MEAN &&
      a->reduction != FLCE_SEQUENCE_MEAN)
    return refuse(FLCE_ERR_INVALID_ARG, "reduction");
  if (a->kl_estimator < FLCE_KL_K1 || a->kl_estimator > FLCE_KL_K3)
    return refuse(FLCE_ERR_INVALID_ARG, "kl_estimator");
  if (!(a->clip_low >= 0.0 && a->clip_low < 1.0) || !(a->clip_high >= 0.0) ||
      !std::isfinite(a->clip_high))
    return refuse(FLCE_ERR_INVALID_ARG, "clip_low or clip_high");
  if (!(a->dual_clip == 0.0 || (a->dual_clip > 1.0 && std::isfinite(a->dual_clip))))
    return refuse(FLCE_ERR_INVALID_ARG, "dual_clip");
  if (!std::isfinite(a->kl_coef)) return refuse(FLCE_ERR_INVALID_ARG, "kl_coef");
  if ((a->advantage_per_token & ~1) != 0 || (a->negated & ~1) != 0 || a->reserved != 0)
    return refuse(FLCE_ERR_INVALID_ARG, "advantage_per_token, negated or reserved");
  return FLCE_OK;
}

struct PolicyLayout {
  size_t counts, loss, kl, clipped, total;
};

PolicyLayout policy_layout(const flce_policy_args* a) {
  PolicyLayout L{};
  const size_t S = static_cast<size_t>(a->tokens.sequences > 0 ? a->tokens.sequences : 2);
  L.counts = kHeader;
  L.loss = L.counts + S * 8;
  L.kl = L.loss + S * 8;
  L.clipped = L.kl + S * 8;
  L.total = L.clipped + S * 8;
  return L;
}

int check_preference(const flce_preference_args* a) {
  if (a == nullptr) return refuse(FLCE_ERR_INVALID_ARG, "arguments are NULL");
  int v = check_tokens(a->tokens);
  if (v != FLCE_OK) return v;
  if (a->tokens.sequences % 2 != 0)
    return refuse(FLCE_ERR_INVALID_ARG, "an odd number of sequences");
  if (a->dtype < FLCE_F32 || a->dtype > FLCE_F16) return refuse(FLCE_ERR_INVALID_ARG, "dtype");
  if (a->loss_type < FLCE_PREF_SIGMOID || a->loss_type > FLCE_PREF_IPO)
    return refuse(FLCE_ERR_INVALID_ARG, "loss_type");
  if (!std::isfinite(a->beta) || a->beta <= 0.0) return refuse(FLCE_ERR_INVALID_ARG, "beta");
  if (!std::isfinite(a->margin)) return refuse(FLCE_ERR_INVALID_ARG, "margin");
  if (!(a->label_smoothing >= 0.0 && a->label_smoothing <= 0.5))
    return refuse(FLCE_ERR_INVALID_ARG, "label_smoothing");
  if ((a->average & ~1) != 0 || (a->negated & ~1) != 0)
    return refuse(FLCE_ERR_INVALID_ARG, "average or negated");
  return FLCE_OK;
}

struct PreferenceLayout {
  size_t sums, counts, loss, total;
};

PreferenceLayout preference_layout(const flce_preference_args* a) {
  PreferenceLayout L{};
  const size_t S = static_cast<size_t>(a->tokens.sequences > 0 ? a->tokens.sequences : 2);
  L.sums = kHeader;
  L.counts = L.sums + S * 8;
  L.loss = L.counts + S * 8;
  L.total = L.loss + S / 2 * 8;
  return L;
}

int check_workspace(const void* ws, uint64_t have, size_t need) {
  if (ws == nullptr || have < need) return refuse(FLCE_ERR_WORKSPACE, "workspace");
  return aligned(ws, 16) ? FLCE_OK : refuse(FLCE_ERR_ALIGNMENT, "workspace");
}

int cuda_error(cudaError_t e, const char* what) {
  char msg[200];
  snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return refuse(FLCE_ERR_CUDA, msg);
}

}  // namespace

extern "C" {

int flce_policy_workspace_bytes(const flce_policy_args* a, size_t* bytes) {
  const int v = check_policy(a);
  if (v != FLCE_OK) return v;
  if (bytes == nullptr) return refuse(FLCE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = policy_layout(a).total;
  return FLCE_OK;
}

int flce_policy_loss(const flce_policy_args* a, flce_stream_t stream) {
  int v = check_policy(a);
  if (v != FLCE_OK) return v;
  const flce_tokens& t = a->tokens;
  const size_t elem = elem_bytes(a->dtype);
  if ((v = check_mask(t)) != FLCE_OK ||
      (v = check_tensor(t, a->log_probs, a->ld_log_probs, elem, false, "log_probs")) != FLCE_OK ||
      (v = check_tensor(t, a->old_log_probs, a->ld_old, elem, true, "old_log_probs")) != FLCE_OK ||
      (v = check_tensor(t, a->ref_log_probs, a->ld_ref, elem, a->kl_coef == 0.0,
                        "ref_log_probs")) != FLCE_OK ||
      (v = check_tensor(t, a->grad, a->ld_grad, 4, true, "grad")) != FLCE_OK)
    return v;
  if (a->advantage_per_token) {
    if ((v = check_tensor(t, a->advantages, a->ld_advantages, 4, false, "advantages")) != FLCE_OK)
      return v;
  } else if (a->advantages == nullptr && token_total(t) > 0) {
    return refuse(FLCE_ERR_INVALID_ARG, "advantages");
  } else if (!aligned(a->advantages, 4)) {
    return refuse(FLCE_ERR_ALIGNMENT, "advantages");
  }
  if (a->loss == nullptr) return refuse(FLCE_ERR_INVALID_ARG, "loss is NULL");
  if (!aligned(a->loss, 4) || !aligned(a->kl_sum, 4) || !aligned(a->num_tokens, 8) ||
      !aligned(a->num_clipped, 8))
    return refuse(FLCE_ERR_ALIGNMENT, "loss, kl_sum, num_tokens or num_clipped");
  const PolicyLayout L = policy_layout(a);
  if ((v = check_workspace(a->workspace, a->ws_bytes, L.total)) != FLCE_OK) return v;
  int sms = 0;
  if ((v = require_device(&sms)) != FLCE_OK) return v;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(a->workspace);

  PolicyArgs k{};
  k.t = view_of(t);
  k.lp = a->log_probs;
  k.old = a->old_log_probs;
  k.ref = a->ref_log_probs;
  k.adv = a->advantages;
  k.grad = a->grad;
  k.ld_lp = a->ld_log_probs;
  k.ld_old = a->ld_old;
  k.ld_ref = a->ld_ref;
  k.ld_adv = a->ld_advantages;
  k.ld_grad = a->ld_grad;
  k.sign = a->negated ? -1.f : 1.f;
  k.lo = static_cast<float>(log(1.0 - a->clip_low));
  k.hi = static_cast<float>(log(1.0 + a->clip_high));
  k.dual = static_cast<float>(a->dual_clip);
  k.log_dual = a->dual_clip > 0.0 ? static_cast<float>(log(a->dual_clip)) : 0.f;
  k.kl_coef = static_cast<float>(a->kl_coef);
  k.adv_per_token = a->advantage_per_token;
  k.kl = a->kl_estimator;
  k.reduction = a->reduction;
  k.loss = a->loss;
  k.num_tokens = a->num_tokens;
  k.num_clipped = a->num_clipped;
  k.kl_sum = a->kl_sum;
  k.status = reinterpret_cast<int*>(ws);
  k.done = reinterpret_cast<int*>(ws + 8);
  k.counts = reinterpret_cast<long long*>(ws + L.counts);
  k.part_loss = reinterpret_cast<double*>(ws + L.loss);
  k.part_kl = reinterpret_cast<double*>(ws + L.kl);
  k.part_clipped = reinterpret_cast<long long*>(ws + L.clipped);
  k.r_grad = DevRegion{a->grad, span(t, a->ld_grad) * 4};
  k.r_ws = DevRegion{ws, L.total};

  cudaError_t e = cudaMemsetAsync(ws, 0, kHeader, st);
  if (e != cudaSuccess) return cuda_error(e, "cudaMemsetAsync");
  if ((v = run_kernel("flce_token_count", st, [&] { return launch_token_count(k, st); })) != FLCE_OK)
    return v;
  if ((v = run_kernel("flce_policy", st, [&] { return launch_policy(k, a->dtype, st); })) != FLCE_OK)
    return v;
  return finish_call(ws, st);
}

int flce_preference_workspace_bytes(const flce_preference_args* a, size_t* bytes) {
  const int v = check_preference(a);
  if (v != FLCE_OK) return v;
  if (bytes == nullptr) return refuse(FLCE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = preference_layout(a).total;
  return FLCE_OK;
}

int flce_preference_loss(const flce_preference_args* a, flce_stream_t stream) {
  int v = check_preference(a);
  if (v != FLCE_OK) return v;
  const flce_tokens& t = a->tokens;
  const size_t elem = elem_bytes(a->dtype);
  if ((v = check_mask(t)) != FLCE_OK ||
      (v = check_tensor(t, a->log_probs, a->ld_log_probs, elem, false, "log_probs")) != FLCE_OK ||
      (v = check_tensor(t, a->ref_log_probs, a->ld_ref, elem, true, "ref_log_probs")) != FLCE_OK ||
      (v = check_tensor(t, a->grad, a->ld_grad, 4, true, "grad")) != FLCE_OK)
    return v;
  if (a->loss == nullptr) return refuse(FLCE_ERR_INVALID_ARG, "loss is NULL");
  if (!aligned(a->loss, 4) || !aligned(a->chosen_rewards, 4) || !aligned(a->rejected_rewards, 4))
    return refuse(FLCE_ERR_ALIGNMENT, "loss, chosen_rewards or rejected_rewards");
  const PreferenceLayout L = preference_layout(a);
  if ((v = check_workspace(a->workspace, a->ws_bytes, L.total)) != FLCE_OK) return v;
  int sms = 0;
  if ((v = require_device(&sms)) != FLCE_OK) return v;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(a->workspace);

  PreferenceArgs k{};
  k.t = view_of(t);
  k.lp = a->log_probs;
  k.ref = a->ref_log_probs;
  k.grad = a->grad;
  k.ld_lp = a->ld_log_probs;
  k.ld_ref = a->ld_ref;
  k.ld_grad = a->ld_grad;
  k.sign = a->negated ? -1.f : 1.f;
  k.beta = a->beta;
  k.smoothing = a->label_smoothing;
  k.margin = a->margin;
  k.type = a->loss_type;
  k.average = a->average;
  k.loss = a->loss;
  k.chosen = a->chosen_rewards;
  k.rejected = a->rejected_rewards;
  k.status = reinterpret_cast<int*>(ws);
  k.done = reinterpret_cast<int*>(ws + 8);
  k.sums = reinterpret_cast<double*>(ws + L.sums);
  k.counts = reinterpret_cast<long long*>(ws + L.counts);
  k.pair_loss = reinterpret_cast<double*>(ws + L.loss);
  k.r_grad = DevRegion{a->grad, span(t, a->ld_grad) * 4};
  k.r_ws = DevRegion{ws, L.total};

  cudaError_t e = cudaMemsetAsync(ws, 0, kHeader, st);
  if (e != cudaSuccess) return cuda_error(e, "cudaMemsetAsync");
  if ((v = run_kernel("flce_sequence_sum", st,
                      [&] { return launch_sequence_sum(k, a->dtype, st); })) != FLCE_OK)
    return v;
  if ((v = run_kernel("flce_preference", st,
                      [&] { return launch_preference(k, a->dtype, st); })) != FLCE_OK)
    return v;
  return finish_call(ws, st);
}

int flce_adamw(const flce_adamw_args* a, flce_stream_t stream) {
  if (a == nullptr) return refuse(FLCE_ERR_INVALID_ARG, "arguments are NULL");
  if (a->count < 0 || a->count > (int64_t(1) << 30) || (a->count > 0 && a->tensors == nullptr))
    return refuse(FLCE_ERR_INVALID_ARG, "tensors or count");
  if (a->step < 1) return refuse(FLCE_ERR_INVALID_ARG, "step");
  const double scalars[] = {a->lr, a->eps, a->weight_decay};
  for (double x : scalars)
    if (!std::isfinite(x) || x < 0.0) return refuse(FLCE_ERR_INVALID_ARG, "lr, eps or weight_decay");
  if (!(a->beta1 >= 0.0 && a->beta1 < 1.0) || !(a->beta2 >= 0.0 && a->beta2 < 1.0))
    return refuse(FLCE_ERR_INVALID_ARG, "beta1 or beta2");
  if (a->dtype < FLCE_F32 || a->dtype > FLCE_F16) return refuse(FLCE_ERR_INVALID_ARG, "dtype");
  if (a->grad_dtype != a->dtype && a->grad_dtype != FLCE_F32)
    return refuse(FLCE_ERR_INVALID_ARG, "grad_dtype");
  if (a->state_bits != 8 && a->state_bits != 32) return refuse(FLCE_ERR_INVALID_ARG, "state_bits");
  if (!aligned(a->grad_scale, 4)) return refuse(FLCE_ERR_ALIGNMENT, "grad_scale");
  const size_t pe = elem_bytes(a->dtype), ge = elem_bytes(a->grad_dtype);
  const size_t se = a->state_bits == 8 ? 1 : 4;
  const flce_adamw_tensor* first = nullptr;
  for (int64_t i = 0; i < a->count; ++i) {
    const flce_adamw_tensor& t = a->tensors[i];
    if (t.numel < 0 || t.numel > (int64_t(1) << 38)) return refuse(FLCE_ERR_INVALID_ARG, "numel");
    if (t.numel > 0 &&
        (t.param == nullptr || t.grad == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr))
      return refuse(FLCE_ERR_INVALID_ARG, "param, grad, exp_avg or exp_avg_sq is NULL");
    if (t.numel > 0 && a->state_bits == 8 &&
        (t.exp_avg_scale == nullptr || t.exp_avg_sq_scale == nullptr))
      return refuse(FLCE_ERR_INVALID_ARG, "exp_avg_scale or exp_avg_sq_scale is NULL");
    if (a->state_bits == 32 && (t.exp_avg_scale != nullptr || t.exp_avg_sq_scale != nullptr))
      return refuse(FLCE_ERR_INVALID_ARG, "scales with 32-bit states");
    if (t.master != nullptr && a->dtype == FLCE_F32)
      return refuse(FLCE_ERR_INVALID_ARG, "a master copy of fp32 parameters");
    if (t.numel > 0) {   // an empty tensor may have any pointers
      if (first == nullptr) first = &t;
      if ((t.master != nullptr) != (first->master != nullptr))
        return refuse(FLCE_ERR_INVALID_ARG, "master copies of some tensors only");
    }
    if (!aligned(t.param, pe) || !aligned(t.grad, ge) || !aligned(t.exp_avg, se) ||
        !aligned(t.exp_avg_sq, se) || !aligned(t.exp_avg_scale, 4) ||
        !aligned(t.exp_avg_sq_scale, 4) || !aligned(t.master, 4))
      return refuse(FLCE_ERR_ALIGNMENT, "a tensor of the table");
  }
  if (a->count == 0) return FLCE_OK;
  int sms = 0, v;
  if ((v = require_device(&sms)) != FLCE_OK) return v;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);

  AdamWArgs k;
  cudaError_t e = adamw_status(&k.status);
  if (e != cudaSuccess) return cuda_error(e, "cudaGetSymbolAddress");
  if (k.status != nullptr && (e = cudaMemsetAsync(k.status, 0, sizeof(int), st)) != cudaSuccess)
    return cuda_error(e, "cudaMemsetAsync");
  k.grad_scale = a->grad_scale;
  k.decay = static_cast<float>(1.0 - a->lr * a->weight_decay);
  k.step_size = static_cast<float>(a->lr / (1.0 - pow(a->beta1, static_cast<double>(a->step))));
  k.inv_root_bc2 = static_cast<float>(1.0 / sqrt(1.0 - pow(a->beta2, static_cast<double>(a->step))));
  k.beta1 = static_cast<float>(a->beta1);
  k.beta2 = static_cast<float>(a->beta2);
  k.one_beta1 = static_cast<float>(1.0 - a->beta1);
  k.one_beta2 = static_cast<float>(1.0 - a->beta2);
  k.eps = static_cast<float>(a->eps);
  unsigned key = a->seed * 0x9E3779B1u + static_cast<unsigned>(a->step) * 0x85A308D3u;
  key ^= key >> 16;
  k.key = key * 0x9E3779B1u;

  // Tables of at most FLCE_ADAMW_TABLE tensors and 2^31 blocks: one launch each.
  unsigned first_block = 0;
  int64_t i = 0;
  while (i < a->count) {
    k.count = 0;
    k.first_block = first_block;
    uint64_t blocks = 0;
    for (; i < a->count && k.count < FLCE_ADAMW_TABLE; ++i) {
      const uint64_t n = static_cast<uint64_t>(a->tensors[i].numel + 255) / 256;
      if (n == 0) continue;
      if (blocks + n > (uint64_t(1) << 31)) break;
      k.t[k.count] = a->tensors[i];
      k.block0[k.count++] = static_cast<unsigned>(blocks);
      blocks += n;
    }
    k.block0[k.count] = static_cast<unsigned>(blocks);
    if (k.count == 0) break;
    first_block += static_cast<unsigned>(blocks);
    v = run_kernel("flce_adamw", st,
                   [&] { return launch_adamw(k, a->dtype, a->grad_dtype, a->state_bits, sms, st); });
    if (v != FLCE_OK) return v;
  }
  return finish_call(k.status, st);
}

}  // extern "C"
