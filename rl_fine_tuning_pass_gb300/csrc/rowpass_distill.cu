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
// Forward, then backward, with the row's results of the forward.
cudaError_t launch_distill_fused(int dtype, bool same_phase, const DistillParams& p, int64_t rows, int sms,
                                 cudaStream_t stream) {
  const cudaError_t e = launch_distill_fwd(dtype, p, rows, sms, stream);
  return e != cudaSuccess ? e : launch_distill_bwd(dtype, same_phase, p, rows, sms, stream);
}
}  // namespace grpo
