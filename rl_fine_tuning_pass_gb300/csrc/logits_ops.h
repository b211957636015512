// Parameter blocks and launchers of the operators next to the GRPO row pass: the sampler's
// rules on logits, the top log-probs of each row, and the distillation loss on a teacher's
// top log-probs.  Host-validated, as in rowpass_internal.h.
#pragma once

#include "rowpass_internal.h"

namespace grpo {

constexpr int GRPO_DEVERR_DUPLICATE_ID_BIT = 4;

// ---- sampler rules ---------------------------------------------------------------------
// One 32-bit word per column of a tile: generated count in the low bits, whether the column
// occurs in the prompt, and 1 + the position of the column's entry in the bias list.
constexpr int kRuleCountBits = 19;
constexpr uint32_t kRulePrompt = 1u << kRuleCountBits;
constexpr int kRuleBiasShift = kRuleCountBits + 1;
constexpr int64_t kRuleMaxTokens = (int64_t(1) << kRuleCountBits) - 1;
constexpr int64_t kRuleMaxBias = (int64_t(1) << (32 - kRuleBiasShift)) - 1;

struct RulesParams {
  RowsView x;    // logits
  RowsView dy;   // backward: gradient of the processed logits
  OutView out;   // processed logits, or the gradient of the logits
  const int64_t* tokens;
  int64_t tokens_stride;
  int64_t N;
  const int32_t* hist_len;    // [rows], nullable: N
  const int32_t* prompt_len;  // [B], nullable: 0
  const float* repetition;    // [B], nullable
  const float* frequency;     // [B], nullable
  const float* presence;      // [B], nullable
  const int64_t* bias_ids;    // [B][M]
  const float* bias;
  int M;
  const uint32_t* allowed;    // nullable
  int64_t allowed_sb, allowed_sl;  // words
  int32_t* dev_err;
};
// same_phase: every output row starts at the same address mod 16 as the row it is made from
// (the logits' in the forward, the upstream gradient's in the backward).  in_place: they are
// the same memory.
cudaError_t launch_rules(int dtype, bool bwd, bool same_phase, bool in_place, const RulesParams& p, int64_t rows,
                         int sms, cudaStream_t stream);

// ---- top log-probs ---------------------------------------------------------------------
constexpr int kTopkMax = 256;
struct TopkParams {
  RowsView x;
  int K;
  float c;     // log2(e) / T
  float invT;  // 1 / T
  int64_t* ids;
  float* logp;
  float* lse;  // nullable
};
cudaError_t launch_topk(int dtype, const TopkParams& p, int64_t rows, int sms, cudaStream_t stream);

// ---- distillation ----------------------------------------------------------------------
constexpr int kDistillMaxK = 256;
struct DistillParams {
  RowsView x;
  OutView dx;            // backward, fused
  const int64_t* ids;    // [rows][K]
  const float* tlogp;    // [rows][K]
  int K;
  const uint8_t* mask;   // nullable
  const float* dloss;    // backward, fused
  float c;               // log2(e) / T
  float invT, invT_lo;   // 1 / T, and what its rounding left
  float T;
  float beta;
  int tail;
  float* loss;           // forward, fused: outputs; backward: lse and p_rest are inputs
  float* lse;
  float* p_rest;
  int32_t* dev_err;
};
cudaError_t launch_distill_fwd(int dtype, const DistillParams& p, int64_t rows, int sms, cudaStream_t stream);
cudaError_t launch_distill_bwd(int dtype, bool same_phase, const DistillParams& p, int64_t rows, int sms,
                               cudaStream_t stream);
cudaError_t launch_distill_fused(int dtype, bool same_phase, const DistillParams& p, int64_t rows, int sms,
                                 cudaStream_t stream);

}  // namespace grpo
