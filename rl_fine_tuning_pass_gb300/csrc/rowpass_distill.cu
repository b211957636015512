// Distillation kernels (see rowpass_distill.cuh).
#include "rowpass_distill.cuh"

namespace grpo {
cudaError_t launch_distill_fwd(int dtype, const DistillParams& p, int64_t rows, int sms, cudaStream_t stream) {
  return dtype == 1 ? launch_distill_fwd_e<BF16>(p, rows, sms, stream)
                    : launch_distill_fwd_e<F32>(p, rows, sms, stream);
}
cudaError_t launch_distill_bwd(int dtype, bool same_phase, const DistillParams& p, int64_t rows, int sms,
                               cudaStream_t stream) {
  return dtype == 1 ? launch_distill_bwd_e<BF16>(same_phase, p, rows, sms, stream)
                    : launch_distill_bwd_e<F32>(same_phase, p, rows, sms, stream);
}
cudaError_t launch_distill_fused(int dtype, bool same_phase, const DistillParams& p, int64_t rows, int sms,
                                 cudaStream_t stream) {
  return dtype == 1 ? launch_distill_fused_e<BF16>(same_phase, p, rows, sms, stream)
                    : launch_distill_fused_e<F32>(same_phase, p, rows, sms, stream);
}
}  // namespace grpo
