// Host entry points of the post-training operators declared in
// include/flce.h: argument checks, workspace layout and launch sequence.
#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <cmath>

#include "flce.h"
#include "nvtx_range.h"
#include "post_training.h"

using namespace flce;

namespace {

constexpr size_t kHeader = 256;          // of a workspace: the finished-block counter
constexpr int kMaxBlocks = 1024;        // of the streaming and counting kernels

#ifdef FLCE_DEBUG
__device__ int g_debug_status;   // the bounds check's word: these entry points have no other errors
#endif

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
    if (t.cols < 0 || t.cols > 2147483647ll - 1024 ||
        (t.sequences > 0 && t.cols > (int64_t(1) << 39) / t.sequences))
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

// A tensor of row stride ld whose offset of a token is its flat index.
bool contiguous(const flce_tokens& t, const void* p, int64_t ld) {
  return p == nullptr || t.packed || t.sequences <= 1 || ld == t.cols;
}

// n neighbouring tokens, from a multiple of n on, are aligned to n elements.
bool groups_aligned(const flce_tokens& t, bool flat, const void* p, int64_t ld, size_t elem, int n) {
  return p == nullptr || (aligned(p, n * elem) && (flat || t.sequences <= 1 || ld % n == 0));
}

struct PolicyLayout {
  bool flat, small;
  int64_t groups, row_groups, counts;   // counts: numbers in the count region
  size_t counts_at, partials_at, total;
};

PolicyLayout policy_layout(const flce_policy_args* a) {
  const flce_tokens& t = a->tokens;
  PolicyLayout L{};
  L.flat = contiguous(t, a->log_probs, a->ld_log_probs) && contiguous(t, a->old_log_probs, a->ld_old) &&
           (a->kl_coef == 0.0 || contiguous(t, a->ref_log_probs, a->ld_ref)) &&
           (!a->advantage_per_token || contiguous(t, a->advantages, a->ld_advantages)) &&
           contiguous(t, a->grad, a->ld_grad) && contiguous(t, t.mask, t.ld_mask);
  L.row_groups = t.packed ? 0 : (t.cols + 3) / 4;
  L.groups = L.flat ? (token_total(t) + 3) / 4 : t.sequences * L.row_groups;
  const bool masked = t.mask_kind != FLCE_MASK_NONE;
  const bool by_sequence = a->reduction == FLCE_SEQUENCE_MEAN;
  L.small = L.groups <= kPolicySmallGroups &&
            !(masked && by_sequence && t.sequences > kPolicySmallSequences);
  if (L.small) return L;
  L.counts = !masked || a->reduction == FLCE_TOKEN_SUM ? 0 : by_sequence ? t.sequences : kMaxBlocks;
  L.counts_at = kHeader;
  L.partials_at = L.counts_at + (static_cast<size_t>(L.counts) * 8 + 15) / 16 * 16;
  L.total = L.partials_at + kMaxBlocks * sizeof(PolicyPartial);
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
  bool small;
  size_t loss_at, total;
};

PreferenceLayout preference_layout(const flce_preference_args* a) {
  PreferenceLayout L{};
  const int64_t pairs = a->tokens.sequences / 2;
  L.small = pairs <= kPreferenceSmallPairs && token_total(a->tokens) <= kPreferenceSmallTokens;
  if (L.small) return L;
  L.loss_at = kHeader;
  L.total = L.loss_at + static_cast<size_t>(pairs) * 4;
  return L;
}

int check_workspace(const void* ws, uint64_t have, size_t need) {
  if (need == 0) return FLCE_OK;
  if (ws == nullptr || have < need) return refuse(FLCE_ERR_WORKSPACE, "workspace");
  return aligned(ws, 16) ? FLCE_OK : refuse(FLCE_ERR_ALIGNMENT, "workspace");
}

int cuda_error(cudaError_t e, const char* what) {
  char msg[200];
  snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return refuse(FLCE_ERR_CUDA, msg);
}

// Debug builds: the zeroed word that the kernels flag bad stores in; else NULL.
int debug_status(int** status, cudaStream_t s) {
  *status = nullptr;
#ifdef FLCE_DEBUG
  void* p = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&p, g_debug_status);
  if (e == cudaSuccess) e = cudaMemsetAsync(p, 0, sizeof(int), s);
  if (e != cudaSuccess) return cuda_error(e, "the debug build's status word");
  *status = static_cast<int*>(p);
#else
  (void)s;
#endif
  return FLCE_OK;
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
  NvtxRange range("flce_policy_loss");
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
  k.ratio_lo = static_cast<float>(1.0 - a->clip_low);
  k.ratio_hi = static_cast<float>(1.0 + a->clip_high);
  k.dual = static_cast<float>(a->dual_clip);
  k.log_dual = a->dual_clip > 0.0 ? static_cast<float>(log(a->dual_clip)) : INFINITY;
  k.kl_coef = static_cast<float>(a->kl_coef);
  k.adv_per_token = a->advantage_per_token;
  k.kl = a->kl_estimator;
  k.reduction = a->reduction;
  k.flat = L.flat ? 1 : 0;
  const auto inputs_aligned = [&](int n) {
    return groups_aligned(t, L.flat, a->log_probs, a->ld_log_probs, elem, n) &&
           groups_aligned(t, L.flat, a->old_log_probs, a->ld_old, elem, n) &&
           (a->kl_coef == 0.0 || groups_aligned(t, L.flat, a->ref_log_probs, a->ld_ref, elem, n)) &&
           (!a->advantage_per_token || groups_aligned(t, L.flat, a->advantages, a->ld_advantages, 4, n));
  };
  k.vec = inputs_aligned(4);
  k.vec_mask = t.mask_kind == FLCE_MASK_BYTES && groups_aligned(t, L.flat, t.mask, t.ld_mask, 1, 4);
  k.vec_grad = groups_aligned(t, L.flat, a->grad, a->ld_grad, 4, 4);
  k.octets = L.flat && inputs_aligned(8) && groups_aligned(t, true, a->grad, 0, 4, 8) &&
             (t.mask_kind != FLCE_MASK_BYTES || groups_aligned(t, true, t.mask, 0, 1, 8));
  k.groups = L.groups;
  k.row_groups = L.row_groups;
  k.loss = a->loss;
  k.num_tokens = a->num_tokens;
  k.num_clipped = a->num_clipped;
  k.kl_sum = a->kl_sum;
  k.r_grad = DevRegion{a->grad, span(t, a->ld_grad) * 4};
  k.r_ws = DevRegion{ws, L.total};
  if ((v = debug_status(&k.status, st)) != FLCE_OK) return v;

  if (L.small) {
    v = run_kernel("flce_policy_small", st, [&] { return launch_policy_small(k, a->dtype, st); });
    return v != FLCE_OK ? v : finish_call(k.status, st);
  }
  const int64_t most = std::min<int64_t>(kMaxBlocks, int64_t(sms) * kPolicyBlocksPerSm);
  const int64_t units = k.octets ? token_total(t) / 8 : L.groups;
  // Whole rounds of a block's threads; one block at least, also for a batch of
  // many sequences but few tokens or none.
  k.per = std::max<int64_t>(1, (units + most - 1) / most);
  k.per = (k.per + 255) / 256 * 256;
  const unsigned grid = static_cast<unsigned>(std::max<int64_t>(1, (units + k.per - 1) / k.per));
  k.done = reinterpret_cast<int*>(ws);
  k.counts = reinterpret_cast<long long*>(ws + L.counts_at);
  k.num_counts = L.counts;
  k.partials = reinterpret_cast<PolicyPartial*>(ws + L.partials_at);
  if (L.counts > 0) {
    const int64_t work = a->reduction == FLCE_SEQUENCE_MEAN ? t.sequences : (L.groups + 1023) / 1024;
    const int blocks = static_cast<int>(std::min<int64_t>(work, kMaxBlocks));
    if (a->reduction == FLCE_TOKEN_MEAN) k.num_counts = blocks;
    v = run_kernel("flce_policy_count", st, [&] { return launch_count(k, blocks, st); });
    if (v != FLCE_OK) return v;
  } else {
    const cudaError_t e = cudaMemsetAsync(k.done, 0, sizeof(int), st);
    if (e != cudaSuccess) return cuda_error(e, "cudaMemsetAsync");
  }
  v = run_kernel("flce_policy", st,
                 [&] { return launch_policy(k, a->dtype, L.counts > 0, grid, st); });
  return v != FLCE_OK ? v : finish_call(k.status, st);
}

int flce_preference_workspace_bytes(const flce_preference_args* a, size_t* bytes) {
  const int v = check_preference(a);
  if (v != FLCE_OK) return v;
  if (bytes == nullptr) return refuse(FLCE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = preference_layout(a).total;
  return FLCE_OK;
}

int flce_preference_loss(const flce_preference_args* a, flce_stream_t stream) {
  NvtxRange range("flce_preference_loss");
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
  k.beta = static_cast<float>(a->beta);
  k.smoothing = static_cast<float>(a->label_smoothing);
  k.margin = static_cast<float>(a->margin);
  k.type = a->loss_type;
  k.average = a->average;
  k.loss = a->loss;
  k.chosen = a->chosen_rewards;
  k.rejected = a->rejected_rewards;
  k.flat = contiguous(t, a->log_probs, a->ld_log_probs) && contiguous(t, a->ref_log_probs, a->ld_ref) &&
           contiguous(t, a->grad, a->ld_grad) && contiguous(t, t.mask, t.ld_mask);
  k.vec = groups_aligned(t, k.flat, a->log_probs, a->ld_log_probs, elem, 8) &&
          groups_aligned(t, k.flat, a->ref_log_probs, a->ld_ref, elem, 8) &&
          groups_aligned(t, k.flat, a->grad, a->ld_grad, 4, 8) &&
          (t.mask_kind != FLCE_MASK_BYTES || groups_aligned(t, k.flat, t.mask, t.ld_mask, 1, 8));
  k.r_grad = DevRegion{a->grad, span(t, a->ld_grad) * 4};
  k.r_ws = DevRegion{ws, L.total};
  if ((v = debug_status(&k.status, st)) != FLCE_OK) return v;

  const int64_t pairs = t.sequences / 2;
  if (pairs == 0 && t.packed && t.tokens > 0 && a->grad != nullptr) {
    // no pair writes the tokens outside every sequence
    const cudaError_t e = cudaMemsetAsync(a->grad, 0, static_cast<size_t>(t.tokens) * 4, st);
    if (e != cudaSuccess) return cuda_error(e, "cudaMemsetAsync");
  }
  if (L.small || pairs == 0) {
    v = run_kernel("flce_preference_small", st,
                   [&] { return launch_preference_small(k, a->dtype, st); });
    return v != FLCE_OK ? v : finish_call(k.status, st);
  }
  k.done = reinterpret_cast<int*>(ws);
  k.pair_loss = reinterpret_cast<float*>(ws + L.loss_at);
  // Blocks a pair: enough for two on each SM, while each still has 4096 tokens.
  // (512 pairs of 2 x 8192 tokens: 26 us with one block a pair, 32 us with two.)
  const int64_t a_pair = token_total(t) / pairs;
  // Where there are many pairs of few tokens a warp takes one (cluster 0).
  int cluster = a_pair <= kWarpPairTokens && pairs >= 4 * sms ? 0 : 1;
  while (cluster > 0 && cluster < 8 && pairs * cluster < 2 * sms && a_pair / (cluster * 2) >= 4096) cluster *= 2;
  const cudaError_t e = cudaMemsetAsync(k.done, 0, sizeof(int), st);
  if (e != cudaSuccess) return cuda_error(e, "cudaMemsetAsync");
  v = run_kernel("flce_preference", st, [&] { return launch_preference(k, a->dtype, cluster, st); });
  return v != FLCE_OK ? v : finish_call(k.status, st);
}

int flce_adamw(const flce_adamw_args* a, flce_stream_t stream) {
  NvtxRange range("flce_adamw");
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
  if ((v = debug_status(&k.status, st)) != FLCE_OK) return v;
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
