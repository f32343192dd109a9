// Internal interface of the post-training operators (policy and preference
// losses, AdamW): the host entry points in post_training.cu, the kernels in
// loss_kernels.cu and adamw_kernels.cu. It is not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "flce.h"
#include "kernels.h"

namespace flce {

// Shared with flce.cu.
int require_device(int* sms);   // FLCE_OK on a GB300, with its number of SMs
int run_launch(const char* name, cudaStream_t s, cudaError_t (*f)(void*), void* ctx);
int finish_call(const void* ws, cudaStream_t s);   // debug builds: the bounds check

// run_launch for a callable.
template <class F>
int run_kernel(const char* name, cudaStream_t s, F&& f) {
  using G = typename std::remove_reference<F>::type;
  return run_launch(name, s, [](void* c) { return (*static_cast<G*>(c))(); }, &f);
}

// The tokens of a batch, as flce_tokens with the fields the kernels use.
struct TokenView {
  long long S, cols, N;        // N: packed tokens, or S * cols
  const int* cu;               // packed, else nullptr
  const void* mask;
  long long ld_mask, ignore_index;
  int mask_kind;
};

struct PolicyArgs {
  TokenView t;
  const void* lp;
  const void* old;             // nullable
  const void* ref;             // nullable
  const float* adv;
  float* grad;                 // nullable
  long long ld_lp, ld_old, ld_ref, ld_adv, ld_grad;
  float sign;                  // -1: lp holds -log p
  float lo, hi, log_dual, dual, kl_coef;   // dual: 0 off
  int adv_per_token, kl, reduction;
  float* loss;
  int64_t* num_tokens;
  int64_t* num_clipped;
  float* kl_sum;
  // workspace
  int* status;
  int* done;                   // zeroed before the main kernel
  long long* counts;           // [S]
  double* part_loss;           // [S]
  double* part_kl;
  long long* part_clipped;
  DevRegion r_grad, r_ws;
};

struct PreferenceArgs {
  TokenView t;
  const void* lp;
  const void* ref;             // nullable
  float* grad;                 // nullable
  long long ld_lp, ld_ref, ld_grad;
  float sign;
  float beta, smoothing, margin;
  int type, average;
  float* loss;
  float* chosen;               // nullable
  float* rejected;             // nullable
  int* status;
  int* done;
  double* sums;                // [S]
  long long* counts;           // [S]
  double* pair_loss;           // [S / 2]
  DevRegion r_grad, r_ws;
};

cudaError_t launch_token_count(const PolicyArgs& a, cudaStream_t s);
cudaError_t launch_policy(const PolicyArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_sequence_sum(const PreferenceArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_preference(const PreferenceArgs& a, int dtype, cudaStream_t s);

struct AdamWArgs {
  const float* grad_scale;     // nullable
  float decay, step_size, inv_root_bc2, beta1, beta2, eps;
  // 1 - beta, rounded from the double
  float one_beta1, one_beta2;
  unsigned key;
  int count;
  unsigned first_block;        // of the launch's first tensor among the call's 256-element
                               // blocks, mod 2^32 (it numbers the random bits)
  int* status;                 // debug builds
  flce_adamw_tensor t[FLCE_ADAMW_TABLE];
  unsigned block0[FLCE_ADAMW_TABLE + 1];   // first block of each tensor within the launch
};

// dtype and grad_dtype: flce_dtype; bits: 8 or 32.
cudaError_t launch_adamw(const AdamWArgs& a, int dtype, int grad_dtype, int bits, int sms,
                         cudaStream_t s);
cudaError_t adamw_status(int** status);   // debug builds: a device word for the bounds check

}  // namespace flce
