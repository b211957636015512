"""GRPO / entropy / selective-log-softmax row pass over LM-head logits, for GB300 (sm_103a).

The compute path is the C-ABI library ``libgrpo_rowpass.so`` (hand-written CUDA kernels,
declared in ``include/grpo_rowpass.h``); this package holds its build step, a thin ctypes
binding with the same function names, autograd wrappers, and the seeded workload
generators.  The library is loaded on first use; importing the package needs no GPU.
"""
from .binding import (  # noqa: F401
    GrpoError,
    distill_topk_bwd,
    distill_topk_fused,
    distill_topk_fwd,
    entropy_from_logits,
    entropy_from_logits_bwd,
    grpo_loss_bwd,
    grpo_loss_fused,
    grpo_loss_fwd,
    grpo_seq_terms,
    load_library,
    process_logits_bwd,
    process_logits_fwd,
    selective_log_softmax_bwd,
    selective_log_softmax_fwd,
    status_string,
    topk_log_softmax,
)
from .autograd import (  # noqa: F401,E402
    distill_topk_loss,
    entropy,
    grpo_loss,
    process_logits,
    selective_log_softmax,
)
