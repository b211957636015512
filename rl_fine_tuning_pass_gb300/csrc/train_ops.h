// Parameter blocks and launchers of the operators of a fine-tuning step next to the policy loss:
// the preference loss on pairs of sequences, the norm of many gradients, and the AdamW update of
// many tensors.  Host-validated, as in rowpass_internal.h.
#pragma once

#include "rowpass_internal.h"

namespace grpo {

// ---- preference loss -------------------------------------------------------------------
struct PrefParams {
  RowsView x;              // 2 * pairs sequences: the chosen ones first, then the rejected ones
  OutView dx;              // backward, fused
  int64_t pairs;
  const int64_t* idx;
  const uint8_t* mask;     // nullable
  const float* ref_logp;   // [2 * pairs], nullable: 0
  const float* dloss;      // [pairs] backward, fused
  float c;                 // log2(e) / T
  float c_fwd;             // the same in the forward: of 15 bits for bf16 logits
  float c_off;             // (log2(e) / T - c_fwd) / c_fwd: for fp32 logits what c's rounding lost, over c
  float ln2_hi, ln2_lo;    // 1 / T / c_fwd: what ln2 is to the rounded c
  float inv_hi, inv_lo;    // 1 / T
  float T;
  int kind;                // grpo_pref_kind
  bool average;
  float beta, gamma, smoothing, sft;
  float* loss;             // [pairs]
  float* reward;           // [2 * pairs]
  float* seq_logp;         // [2 * pairs]
  float* coef;             // [2 * pairs] output of the forward, input of the backward
  float* logp;             // [2][rows]: rounded, and what the rounding lost
  float* lse;              // [rows] output of the forward, input of the backward
  int32_t* dev_err;        // nullable
};
cudaError_t launch_pref_fwd(int dtype, const PrefParams& p, int64_t rows, int sms, cudaStream_t stream);
cudaError_t launch_pref_bwd(int dtype, bool same_phase, const PrefParams& p, int64_t rows, int sms,
                            cudaStream_t stream);

// ---- many tensors ----------------------------------------------------------------------
// A launch takes its table of tensors as a kernel parameter: no copy to the device, nothing to keep
// alive for a captured graph.  Parameters hold 32,764 bytes, but a call passes them anew, so few
// tensors go by a short table.
constexpr int kNormFew = 32, kNormMany = 1024;
constexpr int kAdamwFew = 24, kAdamwMany = 440;

struct NormTensor {
  const void* grad;
  int64_t n;
};
// first[i]: tensor i's first chunk.  Apart from the rest, so that a search touches few cache lines (among the
// descriptors it cost every CTA some 2 us).
template <int N>
struct NormTable {
  uint32_t first[N];
  NormTensor t[N];
  int count;
  uint32_t chunks;
};
struct NormEntry {
  NormTensor t;
  int32_t bf16;
};

struct NormPartial {
  float hi, lo;  // the sum, as two numbers, of what is in fp32's range squared
  double far;    // and of the rest
};
constexpr int kNormSlots = 8192;  // partial sums
cudaError_t launch_grad_norm(NormEntry* tensors, int64_t count, NormPartial* partial, float* norm, cudaStream_t stream);

constexpr int kAdamwBlock = 256;  // elements that share a scale of the 8-bit states
struct AdamwTensor {
  void* param;
  const void* grad;
  float* master;        // nullable
  void* exp_avg;
  void* exp_avg_sq;
  float2* scale;        // 8-bit states: (first moment's, second moment's root's) of each block
  int64_t n;
  float weight_decay;
  uint32_t ordinal : 24;  // its place in the call's list, for the random bits
  uint32_t param_bf16 : 1, grad_bf16 : 1, aligned : 1;
};
// The device words of grpo_adamw_state.
struct AdamwState {
  int64_t step;
  double beta1_pow, beta2_pow;  // of the steps made; 1 where step == 0, whatever they hold
  uint32_t ticket;
  int32_t reserved;
};
struct AdamwScalars {
  double lr, beta1, beta2;
  const float* lr_dev;   // nullable: lr
  const float* norm;     // nullable: no clipping
  float max_norm;
  float b1, b2, w1, w2;  // beta1, beta2, 1 - beta1, 1 - beta2
  float eps;
  uint32_t seed_lo, seed_hi;
  int stochastic;
  AdamwState* state;
};
template <int N>
struct AdamwTable {
  uint32_t first[N];  // tensor i's first CTA
  AdamwTensor t[N];
  int count;
  uint32_t items;
};
cudaError_t launch_adamw(AdamwTensor* tensors, int64_t count, const AdamwScalars& s, int bits, int sms,
                         cudaStream_t stream);
cudaError_t launch_adamw_moments(const uint8_t* exp_avg, const uint8_t* exp_avg_sq, const float2* scale, int64_t n,
                                 float* m, float* v, cudaStream_t stream);

}  // namespace grpo
