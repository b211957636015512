"""Thin Python binding over the C ABI in ``include/grpo_rowpass.h``.

Argument marshalling only: each function checks tensor devices/dtypes, allocates the
outputs with torch (device memory is torch's job here), and calls the C entry point of
the same name on the current CUDA stream.  Every step of the row pass runs in the CUDA
kernels of ``libgrpo_rowpass.so``; there is no CPU fallback.  A missing library raises
``RuntimeError`` on first use.
"""

from __future__ import annotations

import ctypes
import os
import struct
from array import array
from operator import attrgetter
from typing import Optional

import torch

from .build import LIB_PATH

GRPO_OK, GRPO_ERR_INVALID_ARG, GRPO_ERR_UNSUPPORTED, GRPO_ERR_CUDA = 0, 1, 2, 3
GRPO_FP32, GRPO_BF16 = 0, 1
GRPO_DEVERR_IDX_OUT_OF_RANGE = 1

EXPORTED = ("grpo_loss_fwd", "grpo_loss_bwd", "grpo_loss_fused", "entropy_from_logits",
            "entropy_from_logits_bwd", "selective_log_softmax_fwd", "selective_log_softmax_bwd",
            "grpo_seq_terms", "grpo_vocab_shard_stats", "grpo_vocab_combine", "grpo_loss_bwd_vocab_shard",
            "selective_log_softmax_bwd_vocab_shard", "grpo_fused_linear_workspace_size", "grpo_fused_linear",
            "grpo_fused_linear_noalloc", "grpo_status_string", "process_logits_fwd", "process_logits_bwd",
            "topk_log_softmax", "distill_topk_fwd", "distill_topk_bwd", "distill_topk_fused",
            "preference_loss_fwd", "preference_loss_bwd", "preference_loss_fused", "grad_norm", "adamw_step", "adamw_moments")
GRPO_VOCAB_MAX_WORLD = 64
GRPO_DEVERR_DUPLICATE_ID = 4
GRPO_TOPK_MAX = 256
GRPO_DISTILL_MAX_K = 256
GRPO_PREF_KINDS = {"sigmoid": 0, "hinge": 1, "squared": 2}
GRPO_GRAD_NORM_WORKSPACE = 131072


class GrpoRows(ctypes.Structure):
    """Mirror of ``grpo_rows``."""
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("B", ctypes.c_int64), ("L", ctypes.c_int64), ("V", ctypes.c_int64),
                ("stride_b", ctypes.c_int64), ("stride_l", ctypes.c_int64)]


class GrpoLogitRules(ctypes.Structure):
    """Mirror of ``grpo_logit_rules``."""
    _fields_ = [("tokens", ctypes.c_void_p), ("tokens_stride", ctypes.c_int64), ("N", ctypes.c_int64),
                ("hist_len", ctypes.c_void_p), ("prompt_len", ctypes.c_void_p), ("repetition", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("M", ctypes.c_int64), ("allowed", ctypes.c_void_p),
                ("allowed_stride_b", ctypes.c_int64), ("allowed_stride_l", ctypes.c_int64)]


class GrpoPrefArgs(ctypes.Structure):
    """Mirror of ``grpo_pref_args``."""
    _fields_ = [("T", ctypes.c_double), ("kind", ctypes.c_int32), ("average", ctypes.c_int32), ("beta", ctypes.c_float),
                ("gamma", ctypes.c_float), ("label_smoothing", ctypes.c_float), ("sft_weight", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class GrpoGradTensor(ctypes.Structure):
    """Mirror of ``grpo_grad_tensor``."""
    _fields_ = [("ptr", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class GrpoAdamwTensor(ctypes.Structure):
    """Mirror of ``grpo_adamw_tensor``."""
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("weight_decay", ctypes.c_float), ("reserved", ctypes.c_int32)]


class GrpoAdamwArgs(ctypes.Structure):
    """Mirror of ``grpo_adamw_args``."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("lr_dev", ctypes.c_void_p), ("norm", ctypes.c_void_p),
                ("max_norm", ctypes.c_float), ("state_bits", ctypes.c_int32), ("stochastic", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("seed", ctypes.c_uint64)]


class GrpoError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)}")


_lib = None
_P = ctypes.c_void_p
_F = ctypes.c_float


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load ``libgrpo_rowpass.so`` (once) and declare the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m rl_fine_tuning_pass_gb300.build` "
                           "(or __graft_entry__.build()); the row pass has no fallback")
    lib = ctypes.CDLL(path)
    rows_p = ctypes.POINTER(GrpoRows)
    sig = {
        "grpo_loss_fwd": [rows_p, _P, _P, _P, _P, _P, _F, _F, _F, _F, _P, _P, _P, _P, _P, _P, _P, _P],
        "grpo_loss_bwd": [rows_p, _P, _P, _P, _P, _P, _P, _P, _P, _F, _F, _F, _F, rows_p, _P, _P],
        "grpo_loss_fused": [rows_p, _P, _P, _P, _P, _P, _P, _F, _F, _F, _F, _P, _P, _P, _P, _P, _P, rows_p, _P, _P],
        "entropy_from_logits": [rows_p, _F, _P, _P, _P],
        "entropy_from_logits_bwd": [rows_p, _P, _P, _P, _F, rows_p, _P],
        "grpo_seq_terms": [ctypes.c_int64, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _F, _F, _F, _P, _P, _P, _P, _P, _P],
        "selective_log_softmax_fwd": [rows_p, _P, _F, _P, _P, _P, _P],
        "selective_log_softmax_bwd": [rows_p, _P, _P, _P, _F, rows_p, _P, _P],
        "grpo_vocab_shard_stats": [rows_p, ctypes.c_int64, _P, _P, _F, _P, _P],
        "grpo_vocab_combine": [ctypes.c_int32, _P, _P, ctypes.c_int64, ctypes.c_int64, _P, _P, _P, _P, _P,
                               _F, _F, _F, _F, _P, _P, _P, _P, _P, _P, _P, _P, _P],
        "grpo_loss_bwd_vocab_shard": [rows_p, ctypes.c_int64, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P, _P,
                                      _P, _F, _F, _F, _F, rows_p, _P, _P],
        "selective_log_softmax_bwd_vocab_shard": [rows_p, ctypes.c_int64, ctypes.c_int64, _P, _P, _P, _P, _F,
                                                  rows_p, _P, _P],
        "grpo_fused_linear_workspace_size": [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                             ctypes.POINTER(ctypes.c_uint64)],
        "grpo_fused_linear": [_P, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _P, _P, _P, _P,
                              _P, _P, _F, _F, _F, _F, ctypes.c_int64, _P, ctypes.c_uint64, _P, _P, _P, _P, _P, _P,
                              _P, _P, _P, _P],
        "grpo_fused_linear_noalloc": [_P, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _P, _P,
                                      _P, _P, _P, _P, _F, _F, _F, _F, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P, _P,
                                      _P, _P],
        # descriptors as packed bytes (see _pack_rows), or byref of the structures
        "process_logits_fwd": [_P, _P, _P, _P, _P],
        "process_logits_bwd": [_P, _P, _P, _P, _P, _P],
        "topk_log_softmax": [_P, ctypes.c_int64, _F, _P, _P, _P, _P],
        "distill_topk_fwd": [_P, _P, _P, ctypes.c_int64, _P, _F, _F, ctypes.c_int32, _P, _P, _P, _P, _P],
        "distill_topk_bwd": [_P, _P, _P, ctypes.c_int64, _P, _P, _P, _P, _F, _F, ctypes.c_int32, _P, _P],
        "distill_topk_fused": [_P, _P, _P, ctypes.c_int64, _P, _P, _F, _F, ctypes.c_int32, _P, _P, _P, _P, _P, _P],
        "preference_loss_fwd": [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P],
        "preference_loss_bwd": [_P, _P, _P, _P, _P, _P, ctypes.c_double, _P, _P, _P],
        "preference_loss_fused": [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P],
        "grad_norm": [_P, ctypes.c_int64, _P, _P, ctypes.c_uint64, _P],
        "adamw_step": [_P, ctypes.c_int64, _P, _P, _P],
        "adamw_moments": [_P, _P, _P, ctypes.c_int64, _P, _P, _P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.grpo_status_string.argtypes = [ctypes.c_int]
    lib.grpo_status_string.restype = ctypes.c_char_p
    if path == LIB_PATH:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().grpo_status_string(int(status)).decode()


def rows_of(t: torch.Tensor) -> GrpoRows:
    """Describe a [B, L, V] (or [R, V], read as B=1, L=R) tensor with vocab stride 1."""
    if t.dim() == 2:
        B, L, V = 1, t.shape[0], t.shape[1]
        sb, sl = t.shape[0] * t.stride(0), t.stride(0)
    elif t.dim() == 3:
        B, L, V = t.shape
        sb, sl = t.stride(0), t.stride(1)
    else:
        raise ValueError("logits must be [B, L, V] or [R, V]")
    if V > 0 and t.stride(-1) != 1:
        raise ValueError("the vocabulary dimension must have stride 1")
    if t.dtype == torch.bfloat16:
        dt = GRPO_BF16
    elif t.dtype == torch.float32:
        dt = GRPO_FP32
    else:
        raise TypeError(f"logits dtype {t.dtype} not supported (bf16 or fp32)")
    return GrpoRows(t.data_ptr(), dt, 0, B, L, V, sb, sl)


def _ptr(t: Optional[torch.Tensor], dtype, n: Optional[int], name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    return t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _check(fn: str, st: int):
    if st != GRPO_OK:
        raise GrpoError(fn, st)


def _shape(logits: torch.Tensor):
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if logits.dim() == 3:
        return logits.shape[0], logits.shape[1]
    return 1, logits.shape[0]


def grpo_loss_fwd(logits, idx, adv, *, T, beta, eps_low, eps_high, old_logp=None, ref_logp=None,
                  mask=None, with_kl=True, with_is_clipped=True, with_entropy=False, dev_err=None):
    """GRPO forward; returns a dict with loss, logp, lse (+ kl, is_clipped, entropy)."""
    B, L = _shape(logits)
    R = B * L
    dev = logits.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"loss": torch.empty(R, **f32), "logp": torch.empty(R, **f32), "lse": torch.empty(R, **f32)}
    out["kl"] = torch.empty(R, **f32) if with_kl else None
    out["is_clipped"] = torch.empty(R, dtype=torch.uint8, device=dev) if with_is_clipped else None
    out["entropy"] = torch.empty(R, **f32) if with_entropy else None
    x = rows_of(logits)
    st = load_library().grpo_loss_fwd(
        ctypes.byref(x), _ptr(idx, torch.int64, R, "idx"), _ptr(old_logp, torch.float32, R, "old_logp"),
        _ptr(ref_logp, torch.float32, R, "ref_logp"), _ptr(adv, torch.float32, B, "adv"),
        _ptr(mask, torch.uint8, R, "mask"), float(T), float(beta), float(eps_low), float(eps_high),
        out["loss"].data_ptr(), out["logp"].data_ptr(), out["lse"].data_ptr(),
        _ptr(out["kl"], torch.float32, R, "kl"), _ptr(out["is_clipped"], torch.uint8, R, "is_clipped"),
        _ptr(out["entropy"], torch.float32, R, "entropy"), _ptr(dev_err, torch.int32, 1, "dev_err"),
        _stream(dev))
    _check("grpo_loss_fwd", st)
    return {k: v for k, v in out.items() if v is not None}


def grpo_loss_bwd(logits, idx, adv, dloss, logp, lse, *, T, beta, eps_low, eps_high, old_logp=None,
                  ref_logp=None, mask=None, dlogits=None, dev_err=None):
    """GRPO backward; returns dlogits (allocated [B, L, V] like logits unless given;
    pass ``dlogits=logits`` for an in-place backward)."""
    B, L = _shape(logits)
    R = B * L
    if dlogits is None:
        dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    x, dx = rows_of(logits), rows_of(dlogits)
    st = load_library().grpo_loss_bwd(
        ctypes.byref(x), _ptr(idx, torch.int64, R, "idx"), _ptr(old_logp, torch.float32, R, "old_logp"),
        _ptr(ref_logp, torch.float32, R, "ref_logp"), _ptr(adv, torch.float32, B, "adv"),
        _ptr(mask, torch.uint8, R, "mask"), _ptr(dloss, torch.float32, R, "dloss"),
        _ptr(logp, torch.float32, R, "logp"), _ptr(lse, torch.float32, R, "lse"), float(T), float(beta),
        float(eps_low), float(eps_high), ctypes.byref(dx), _ptr(dev_err, torch.int32, 1, "dev_err"),
        _stream(logits.device))
    _check("grpo_loss_bwd", st)
    return dlogits


def grpo_loss_fused(logits, idx, adv, dloss, *, T, beta, eps_low, eps_high, old_logp=None, ref_logp=None,
                    mask=None, with_kl=True, with_is_clipped=True, with_entropy=False, dlogits=None, dev_err=None):
    """GRPO forward and backward in one pass (dloss known in advance); returns the forward's
    dict plus "dlogits"."""
    B, L = _shape(logits)
    R = B * L
    dev = logits.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"loss": torch.empty(R, **f32), "logp": torch.empty(R, **f32), "lse": torch.empty(R, **f32)}
    out["kl"] = torch.empty(R, **f32) if with_kl else None
    out["is_clipped"] = torch.empty(R, dtype=torch.uint8, device=dev) if with_is_clipped else None
    out["entropy"] = torch.empty(R, **f32) if with_entropy else None
    if dlogits is None:
        dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    x, dx = rows_of(logits), rows_of(dlogits)
    st = load_library().grpo_loss_fused(
        ctypes.byref(x), _ptr(idx, torch.int64, R, "idx"), _ptr(old_logp, torch.float32, R, "old_logp"),
        _ptr(ref_logp, torch.float32, R, "ref_logp"), _ptr(adv, torch.float32, B, "adv"),
        _ptr(mask, torch.uint8, R, "mask"), _ptr(dloss, torch.float32, R, "dloss"), float(T), float(beta),
        float(eps_low), float(eps_high), out["loss"].data_ptr(), out["logp"].data_ptr(), out["lse"].data_ptr(),
        _ptr(out["kl"], torch.float32, R, "kl"), _ptr(out["is_clipped"], torch.uint8, R, "is_clipped"),
        _ptr(out["entropy"], torch.float32, R, "entropy"), ctypes.byref(dx),
        _ptr(dev_err, torch.int32, 1, "dev_err"), _stream(dev))
    _check("grpo_loss_fused", st)
    res = {k: v for k, v in out.items() if v is not None}
    res["dlogits"] = dlogits
    return res


def entropy_from_logits(logits, *, T=1.0, return_lse=False):
    """Per-row entropy [B*L] fp32 (and lse [B*L] when return_lse)."""
    B, L = _shape(logits)
    out = torch.empty(B * L, dtype=torch.float32, device=logits.device)
    lse = torch.empty(B * L, dtype=torch.float32, device=logits.device) if return_lse else None
    x = rows_of(logits)
    st = load_library().entropy_from_logits(ctypes.byref(x), float(T), out.data_ptr(),
                                            None if lse is None else lse.data_ptr(), _stream(logits.device))
    _check("entropy_from_logits", st)
    return (out, lse) if return_lse else out


def entropy_from_logits_bwd(logits, dentropy, lse, entropy, *, T=1.0, dlogits=None):
    """dlogits of sum_r dentropy_r * H_r (allocated like logits unless given)."""
    B, L = _shape(logits)
    R = B * L
    if dlogits is None:
        dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    x, dx = rows_of(logits), rows_of(dlogits)
    st = load_library().entropy_from_logits_bwd(
        ctypes.byref(x), _ptr(dentropy, torch.float32, R, "dentropy"), _ptr(lse, torch.float32, R, "lse"),
        _ptr(entropy, torch.float32, R, "entropy"), float(T), ctypes.byref(dx), _stream(logits.device))
    _check("entropy_from_logits_bwd", st)
    return dlogits


def selective_log_softmax_fwd(logits, idx, *, T=1.0, dev_err=None):
    """Returns (logp, lse), each [B*L] fp32."""
    B, L = _shape(logits)
    R = B * L
    logp = torch.empty(R, dtype=torch.float32, device=logits.device)
    lse = torch.empty(R, dtype=torch.float32, device=logits.device)
    x = rows_of(logits)
    st = load_library().selective_log_softmax_fwd(
        ctypes.byref(x), _ptr(idx, torch.int64, R, "idx"), float(T), logp.data_ptr(), lse.data_ptr(),
        _ptr(dev_err, torch.int32, 1, "dev_err"), _stream(logits.device))
    _check("selective_log_softmax_fwd", st)
    return logp, lse


def selective_log_softmax_bwd(logits, idx, dlogp, lse, *, T=1.0, dlogits=None, dev_err=None):
    """Returns dlogits of sum_r dlogp_r * logp_r (allocated like logits unless given)."""
    B, L = _shape(logits)
    R = B * L
    if dlogits is None:
        dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    x, dx = rows_of(logits), rows_of(dlogits)
    st = load_library().selective_log_softmax_bwd(
        ctypes.byref(x), _ptr(idx, torch.int64, R, "idx"), _ptr(dlogp, torch.float32, R, "dlogp"),
        _ptr(lse, torch.float32, R, "lse"), float(T), ctypes.byref(dx), _ptr(dev_err, torch.int32, 1, "dev_err"),
        _stream(logits.device))
    _check("selective_log_softmax_bwd", st)
    return dlogits


def grpo_seq_terms(logp, adv, dloss, *, B, L, beta, eps_low, eps_high, old_logp=None, ref_logp=None, mask=None):
    """Sequence-level GRPO terms; returns dict(loss, kl, dlogp [B*L], seq_ratio [B],
    seq_is_clipped [B]).  Feed dlogp to selective_log_softmax_bwd for the dlogits."""
    R = B * L
    dev = logp.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"loss": torch.empty(R, **f32), "kl": torch.empty(R, **f32), "dlogp": torch.empty(R, **f32),
           "seq_ratio": torch.empty(B, **f32), "seq_is_clipped": torch.empty(B, dtype=torch.uint8, device=dev)}
    st = load_library().grpo_seq_terms(
        B, L, _ptr(logp, torch.float32, R, "logp"), _ptr(old_logp, torch.float32, R, "old_logp"),
        _ptr(ref_logp, torch.float32, R, "ref_logp"), _ptr(adv, torch.float32, B, "adv"),
        _ptr(mask, torch.uint8, R, "mask"), _ptr(dloss, torch.float32, R, "dloss"), float(beta), float(eps_low),
        float(eps_high), out["loss"].data_ptr(), out["kl"].data_ptr(), out["dlogp"].data_ptr(),
        out["seq_ratio"].data_ptr(), out["seq_is_clipped"].data_ptr(), _stream(dev))
    _check("grpo_seq_terms", st)
    return out


# ---------------------------------------------------------------------------
# vocabulary-parallel form (each rank holds a column shard of every row)
# ---------------------------------------------------------------------------

def grpo_vocab_shard_stats(logits_shard, vocab_start, *, T=1.0, idx=None, mask=None):
    """Per-row statistic (a, s, u, x_sel) of one vocabulary shard: [B*L, 4] fp32."""
    B, L = _shape(logits_shard)
    R = B * L
    stats = torch.empty(R, 4, dtype=torch.float32, device=logits_shard.device)
    x = rows_of(logits_shard)
    st = load_library().grpo_vocab_shard_stats(
        ctypes.byref(x), int(vocab_start), _ptr(idx, torch.int64, R, "idx"), _ptr(mask, torch.uint8, R, "mask"),
        float(T), stats.data_ptr(), _stream(logits_shard.device))
    _check("grpo_vocab_shard_stats", st)
    return stats


def grpo_vocab_combine(stats_all, vocab_starts, B, L, *, T=1.0, idx=None, adv=None, grpo=False, beta=0.0,
                       eps_low=0.2, eps_high=0.2, old_logp=None, ref_logp=None, mask=None, with_entropy=True,
                       with_p_rest=True, dev_err=None):
    """Merge gathered shard statistics [world, B*L, 4] (rank order) into the full rows'
    outputs: dict with lse (+ entropy), and with idx given logp and p_rest, and with
    grpo=True the GRPO terms (loss, kl, is_clipped)."""
    world = int(stats_all.shape[0])
    R = B * L
    dev = stats_all.device
    if stats_all.dtype != torch.float32 or tuple(stats_all.shape) != (world, R, 4) or not stats_all.is_contiguous():
        raise ValueError("stats_all must be a contiguous [world, B*L, 4] float32 tensor")
    if not stats_all.is_cuda:
        raise ValueError("stats_all must be a CUDA tensor")
    starts = (ctypes.c_int64 * (world + 1))(*[int(v) for v in vocab_starts])
    if len(vocab_starts) != world + 1:
        raise ValueError("vocab_starts needs world + 1 entries")
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"lse": torch.empty(R, **f32), "entropy": torch.empty(R, **f32) if with_entropy else None,
           "logp": None, "p_rest": None, "loss": None, "kl": None, "is_clipped": None}
    if idx is not None:
        out["logp"] = torch.empty(R, **f32)
        out["p_rest"] = torch.empty(R, **f32) if with_p_rest else None
    if grpo:
        out["loss"], out["kl"] = torch.empty(R, **f32), torch.empty(R, **f32)
        out["is_clipped"] = torch.empty(R, dtype=torch.uint8, device=dev)
    p = lambda k, dt=torch.float32: _ptr(out[k], dt, R, k)
    st = load_library().grpo_vocab_combine(
        world, stats_all.data_ptr(), starts, B, L, _ptr(idx, torch.int64, R, "idx"),
        _ptr(old_logp, torch.float32, R, "old_logp"), _ptr(ref_logp, torch.float32, R, "ref_logp"),
        _ptr(adv, torch.float32, B, "adv"), _ptr(mask, torch.uint8, R, "mask"), float(T), float(beta),
        float(eps_low), float(eps_high), p("loss"), p("logp"), p("lse"), p("kl"), p("is_clipped", torch.uint8),
        p("entropy"), p("p_rest"), _ptr(dev_err, torch.int32, 1, "dev_err"), _stream(dev))
    _check("grpo_vocab_combine", st)
    return {k: v for k, v in out.items() if v is not None}


def grpo_loss_bwd_vocab_shard(logits_shard, vocab_start, vocab_total, idx, adv, dloss, logp, lse, p_rest, *, T,
                              beta, eps_low, eps_high, old_logp=None, ref_logp=None, mask=None, dlogits=None,
                              dev_err=None):
    """This shard's columns of the GRPO dlogits (allocated like logits_shard unless given)."""
    B, L = _shape(logits_shard)
    R = B * L
    if dlogits is None:
        dlogits = torch.empty(logits_shard.shape, dtype=logits_shard.dtype, device=logits_shard.device)
    x, dx = rows_of(logits_shard), rows_of(dlogits)
    st = load_library().grpo_loss_bwd_vocab_shard(
        ctypes.byref(x), int(vocab_start), int(vocab_total), _ptr(idx, torch.int64, R, "idx"),
        _ptr(old_logp, torch.float32, R, "old_logp"), _ptr(ref_logp, torch.float32, R, "ref_logp"),
        _ptr(adv, torch.float32, B, "adv"), _ptr(mask, torch.uint8, R, "mask"), _ptr(dloss, torch.float32, R, "dloss"),
        _ptr(logp, torch.float32, R, "logp"), _ptr(lse, torch.float32, R, "lse"),
        _ptr(p_rest, torch.float32, R, "p_rest"), float(T), float(beta), float(eps_low), float(eps_high),
        ctypes.byref(dx), _ptr(dev_err, torch.int32, 1, "dev_err"), _stream(logits_shard.device))
    _check("grpo_loss_bwd_vocab_shard", st)
    return dlogits


def selective_log_softmax_bwd_vocab_shard(logits_shard, vocab_start, vocab_total, idx, dlogp, lse, p_rest, *,
                                          T=1.0, dlogits=None, dev_err=None):
    """This shard's columns of the selective-log-softmax dlogits."""
    B, L = _shape(logits_shard)
    R = B * L
    if dlogits is None:
        dlogits = torch.empty(logits_shard.shape, dtype=logits_shard.dtype, device=logits_shard.device)
    x, dx = rows_of(logits_shard), rows_of(dlogits)
    st = load_library().selective_log_softmax_bwd_vocab_shard(
        ctypes.byref(x), int(vocab_start), int(vocab_total), _ptr(idx, torch.int64, R, "idx"),
        _ptr(dlogp, torch.float32, R, "dlogp"), _ptr(lse, torch.float32, R, "lse"),
        _ptr(p_rest, torch.float32, R, "p_rest"), float(T), ctypes.byref(dx),
        _ptr(dev_err, torch.int32, 1, "dev_err"), _stream(logits_shard.device))
    _check("selective_log_softmax_bwd_vocab_shard", st)
    return dlogits


# ---------------------------------------------------------------------------
# the GRPO loss on top of the LM head (hidden states and head weight)
# ---------------------------------------------------------------------------

def grpo_fused_linear_workspace_size(H, V, chunk_rows):
    out = ctypes.c_uint64(0)
    _check("grpo_fused_linear_workspace_size",
           load_library().grpo_fused_linear_workspace_size(int(H), int(V), int(chunk_rows), ctypes.byref(out)))
    return int(out.value)


def grpo_fused_linear(hidden, weight, idx, adv, dloss, *, B, L, T, beta, eps_low, eps_high, old_logp=None,
                      ref_logp=None, mask=None, chunk_rows=2048, with_grad_hidden=True, grad_weight=None,
                      with_grad_weight=True, with_entropy=True, workspace=None, dev_err=None):
    """GRPO loss on top of the LM head, in chunks of rows: dict with the forward outputs
    (loss, logp, lse, kl, is_clipped, entropy), grad_hidden [B*L, H] fp32 and grad_weight
    [V, H] fp32 (accumulated into the given tensor, else into zeros).  The chunks hold only
    unmasked rows.  chunk_rows trades workspace (one chunk's 16-bit exponentials / dlogits,
    statistics and gathered hidden rows, ~2.1 V + 2 H bytes a row, plus 128 MiB) for speed:
    with V = 151936, H = 1024 and 16384 rows (11180 unmasked), chunks of 2048 rows took
    8.9 ms on GB300."""
    R, H = hidden.shape
    V = weight.shape[0]
    if R != B * L:
        raise ValueError("hidden must be [B*L, H]")
    for name, t in (("hidden", hidden), ("weight", weight)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.shape[-1] != H:
            raise ValueError(f"{name} must be a contiguous CUDA bf16 tensor with H columns")
    dev = hidden.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"loss": torch.empty(R, **f32), "logp": torch.empty(R, **f32), "lse": torch.empty(R, **f32),
           "kl": torch.empty(R, **f32), "is_clipped": torch.empty(R, dtype=torch.uint8, device=dev),
           "entropy": torch.empty(R, **f32) if with_entropy else None,
           "grad_hidden": torch.empty(R, H, **f32) if with_grad_hidden else None}
    if with_grad_weight and grad_weight is None:
        grad_weight = torch.zeros(V, H, **f32)
    out["grad_weight"] = grad_weight if with_grad_weight else None
    chunk = max(1, min(int(chunk_rows), R)) if R else 1
    need = grpo_fused_linear_workspace_size(H, V, chunk)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    st = load_library().grpo_fused_linear(
        hidden.data_ptr(), weight.data_ptr(), B, L, H, V, _ptr(idx, torch.int64, R, "idx"),
        _ptr(old_logp, torch.float32, R, "old_logp"), _ptr(ref_logp, torch.float32, R, "ref_logp"),
        _ptr(adv, torch.float32, B, "adv"), _ptr(mask, torch.uint8, R, "mask"), _ptr(dloss, torch.float32, R, "dloss"),
        float(T), float(beta), float(eps_low), float(eps_high), chunk, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), out["loss"].data_ptr(), out["logp"].data_ptr(),
        out["lse"].data_ptr(), out["kl"].data_ptr(), out["is_clipped"].data_ptr(),
        _ptr(out["entropy"], torch.float32, R, "entropy"), _ptr(out["grad_hidden"], torch.float32, R * H, "grad_hidden"),
        _ptr(out["grad_weight"], torch.float32, V * H, "grad_weight"), _ptr(dev_err, torch.int32, 1, "dev_err"),
        _stream(dev))
    _check("grpo_fused_linear", st)
    return {k: v for k, v in out.items() if v is not None}


# ---------------------------------------------------------------------------
# the sampler's rules on logits; a teacher's top log-probs; distillation from them
# ---------------------------------------------------------------------------

# A decode step calls these for microseconds of GPU work, so their marshalling is kept short:
# descriptors are packed with ``struct`` (0.3 us; a ctypes structure takes 1.2 us), and the
# stream and device are asked of torch's C layer (0.1 us each; torch.cuda's objects take 2 us),
# where torch has one: a CPU build does not, and can still import this module.
_ROWS = struct.Struct("=Qiiqqqqq")
_RULES = struct.Struct("=QqqQQQQQQQqQqq")
assert _ROWS.size == ctypes.sizeof(GrpoRows) and _RULES.size == ctypes.sizeof(GrpoLogitRules)
_DTYPES = {torch.bfloat16: GRPO_BF16, torch.float32: GRPO_FP32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", lambda: torch.cuda.current_device())


def _pack_rows(t: torch.Tensor):
    """(packed grpo_rows, B, L, V) of a [B, L, V] (or [R, V], read as B=1, L=R) tensor."""
    shape, stride, dt = t.shape, t.stride(), _DTYPES.get(t.dtype)
    if dt is None or not t.is_cuda or not 2 <= len(shape) <= 3 or stride[-1] != 1:
        if not t.is_cuda:
            raise ValueError("logits must be a CUDA tensor")
        rows_of(t)  # raises, but for a tensor whose vocabulary stride does not matter
        stride = (*stride[:-1], 1)
    if len(shape) == 3:
        B, L, V = shape
        sb, sl, _ = stride
    else:
        (L, V), B = shape, 1
        sl = stride[0]
        sb = L * sl
    return _ROWS.pack(t.data_ptr(), dt, 0, B, L, V, sb, sl), B, L, V


def _on(t: Optional[torch.Tensor], dtype, n: Optional[int], name: str, dev):
    """``_ptr`` for a tensor that has to be on the logits' device (0 for None)."""
    if t is None:
        return 0
    if t.dtype is dtype and t.device == dev and t.is_contiguous() and (n is None or t.numel() == n):
        return t.data_ptr()
    _ptr(t, dtype, n, name)
    raise ValueError(f"{name} must be on {dev}, got {t.device}")


def _like(t: Optional[torch.Tensor], logits: torch.Tensor, name: str):
    """A second [B, L, V] tensor of the call (allocated like the logits if None) and its
    descriptor."""
    if t is None:
        t = torch.empty_like(logits) if logits.is_contiguous() else \
            torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    elif t.device != logits.device:
        raise ValueError(f"{name} must be on {logits.device}, got {t.device}")
    return t, _pack_rows(t)[0]


def _call(fn: str, dev, *args):
    """Call the C entry point with the device's current stream, on that device."""
    f = getattr(_lib or load_library(), fn)
    index = dev.index
    if _raw_device() == index:
        st = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            st = f(*args, _raw_stream(index))
    if st != GRPO_OK:
        raise GrpoError(fn, st)


def _rules(B, L, V, dev, tokens, hist_len, prompt_len, repetition, frequency, presence, bias_ids, bias, allowed):
    tk = ts = N = ids = bs = M = al = sb = sl = 0
    if tokens is not None:
        if tokens.dim() != 2 or tokens.shape[0] != B or tokens.dtype != torch.int64 or tokens.device != dev:
            raise ValueError(f"tokens must be a [B, N] int64 tensor on {dev}")
        ts, one = tokens.stride()
        N = tokens.shape[1]
        if N > 1 and one != 1:
            raise ValueError("tokens must have stride 1 along a sequence")
        tk = tokens.data_ptr()
    elif hist_len is not None or prompt_len is not None or repetition is not None or frequency is not None \
            or presence is not None:
        raise ValueError("penalties and history lengths need tokens")
    f32 = torch.float32
    hist = _on(hist_len, torch.int32, B * L, "hist_len", dev)
    prompt = _on(prompt_len, torch.int32, B, "prompt_len", dev)
    rep = _on(repetition, f32, B, "repetition", dev)
    freq = _on(frequency, f32, B, "frequency", dev)
    pres = _on(presence, f32, B, "presence", dev)
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    if bias_ids is not None:
        shape = bias_ids.shape
        if len(shape) != 2 or shape[0] != B or bias.shape != shape:
            raise ValueError("bias_ids and bias must be [B, M]")
        ids = _on(bias_ids, torch.int64, None, "bias_ids", dev)
        bs = _on(bias, f32, None, "bias", dev)
        M = shape[1]
    if allowed is not None:
        words = (V + 31) // 32
        shape, stride = allowed.shape, allowed.stride()
        if len(shape) == 2 and shape[0] == B * L:
            sb, sl = L * stride[0], stride[0]
        elif len(shape) == 3 and shape[0] == B and shape[1] == L:
            sb, sl = stride[0], stride[1]
        else:
            raise ValueError("allowed must be [B*L, W] or [B, L, W]")
        if allowed.dtype != torch.int32 or allowed.device != dev:
            raise ValueError(f"allowed must be an int32 tensor on {dev}")
        if shape[-1] < words or (words > 1 and stride[-1] != 1):
            raise ValueError(f"allowed needs {words} words a row, with stride 1")
        al = allowed.data_ptr()
    return _RULES.pack(tk, ts, N, hist, prompt, rep, freq, pres, ids, bs, M, al, sb, sl)


def process_logits_fwd(logits, *, tokens=None, hist_len=None, prompt_len=None, repetition=None, frequency=None,
                       presence=None, bias_ids=None, bias=None, allowed=None, out=None, dev_err=None):
    """The sampler's rules on [B, L, V] logits: penalties for the tokens [B, N] of each row's
    history (the first hist_len[b*L + l] of its sequence, of which the first prompt_len[b]
    count for repetition only), biases [B, M] on the columns bias_ids [B, M], and a bitmask of
    the allowed columns, int32 [B*L, ceil(V / 32)] or [B, L, ceil(V / 32)] (expanded views
    too).  A decode batch is [B, 1, V].  Returns the processed logits, allocated like logits
    unless given; ``out=logits`` works in place and touches only what the rules change."""
    x, B, L, V = _pack_rows(logits)
    dev = logits.device
    out, y = _like(out, logits, "out")
    q = _rules(B, L, V, dev, tokens, hist_len, prompt_len, repetition, frequency, presence, bias_ids, bias, allowed)
    _call("process_logits_fwd", dev, x, q, y, _on(dev_err, torch.int32, 1, "dev_err", dev))
    return out


def process_logits_bwd(logits, dout, *, tokens=None, hist_len=None, prompt_len=None, repetition=None, frequency=None,
                       presence=None, bias_ids=None, bias=None, allowed=None, dlogits=None, dev_err=None):
    """Gradient of the logits of process_logits_fwd from that of its output (dlogits allocated
    like logits unless given; ``dlogits=dout`` works in place)."""
    x, B, L, V = _pack_rows(logits)
    dev = logits.device
    _, dy = _like(dout, logits, "dout")
    dlogits, dx = _like(dlogits, logits, "dlogits")
    q = _rules(B, L, V, dev, tokens, hist_len, prompt_len, repetition, frequency, presence, bias_ids, bias, allowed)
    _call("process_logits_bwd", dev, x, dy, q, dx, _on(dev_err, torch.int32, 1, "dev_err", dev))
    return dlogits


def topk_log_softmax(logits, K, *, T=1.0):
    """The K largest log-probs of each row: (ids [B*L, K] int64, logp [B*L, K] fp32, lse [B*L]
    fp32), by falling logit, ties by rising column.  1 <= K <= min(V, 256)."""
    x, B, L, _ = _pack_rows(logits)
    dev = logits.device
    R, K = B * L, max(-1, min(int(K), 1 << 30))   # what the C side refuses stays refused in its 64 bits
    n = max(0, min(K, GRPO_TOPK_MAX))
    ids = torch.empty((R, n), dtype=torch.int64, device=dev)
    logp = torch.empty((R, n), dtype=torch.float32, device=dev)
    lse = torch.empty(R, dtype=torch.float32, device=dev)
    _call("topk_log_softmax", dev, x, K, float(T), ids.data_ptr(), logp.data_ptr(), lse.data_ptr())
    return ids, logp, lse


def _list_of(ids, teacher_logp, R, dev):
    shape = ids.shape
    if len(shape) != 2 or shape[0] != R or teacher_logp.shape != shape:
        raise ValueError("ids and teacher_logp must be [B*L, K]")
    return (_on(ids, torch.int64, None, "ids", dev), _on(teacher_logp, torch.float32, None, "teacher_logp", dev),
            shape[1])


def distill_topk_fwd(logits, ids, teacher_logp, *, T=1.0, beta=0.0, tail=False, mask=None, dev_err=None):
    """Divergence of each row's softmax(logits / T) from a teacher's top log-probs (ids and
    teacher_logp [B*L, K], K <= 256): dict with loss, lse and p_rest, each [B*L] fp32.
    beta 0: KL(teacher | student), 1: KL(student | teacher), between: the mixture's.  tail:
    the teacher's mass outside its list is one more bucket (needed at beta 1); without it, and in
    rows whose unlisted logits are all -inf, the teacher is renormalised over the list."""
    x, B, L, _ = _pack_rows(logits)
    R, dev = B * L, logits.device
    pi, pt, K = _list_of(ids, teacher_logp, R, dev)
    loss = torch.empty(R, dtype=torch.float32, device=dev)
    lse, p_rest = torch.empty_like(loss), torch.empty_like(loss)
    _call("distill_topk_fwd", dev, x, pi, pt, K, _on(mask, torch.uint8, R, "mask", dev), float(T), float(beta),
          bool(tail),
          loss.data_ptr(), lse.data_ptr(), p_rest.data_ptr(), _on(dev_err, torch.int32, 1, "dev_err", dev))
    return {"loss": loss, "lse": lse, "p_rest": p_rest}


def distill_topk_bwd(logits, ids, teacher_logp, dloss, lse, p_rest, *, T=1.0, beta=0.0, tail=False, mask=None,
                     dlogits=None):
    """dlogits of sum_r dloss_r * loss_r, with lse and p_rest of distill_topk_fwd (allocated
    like logits unless given; ``dlogits=logits`` works in place)."""
    x, B, L, _ = _pack_rows(logits)
    R, dev = B * L, logits.device
    dlogits, dx = _like(dlogits, logits, "dlogits")
    pi, pt, K = _list_of(ids, teacher_logp, R, dev)
    f32 = torch.float32
    _call("distill_topk_bwd", dev, x, pi, pt, K, _on(mask, torch.uint8, R, "mask", dev),
          _on(dloss, f32, R, "dloss", dev), _on(lse, f32, R, "lse", dev), _on(p_rest, f32, R, "p_rest", dev),
          float(T), float(beta), bool(tail), dx)
    return dlogits


def distill_topk_fused(logits, ids, teacher_logp, dloss, *, T=1.0, beta=0.0, tail=False, mask=None, dlogits=None,
                       dev_err=None):
    """distill_topk_fwd and distill_topk_bwd in one call, for loss weights dloss known in
    advance; returns the forward's dict plus "dlogits"."""
    x, B, L, _ = _pack_rows(logits)
    R, dev = B * L, logits.device
    dlogits, dx = _like(dlogits, logits, "dlogits")
    pi, pt, K = _list_of(ids, teacher_logp, R, dev)
    loss = torch.empty(R, dtype=torch.float32, device=dev)
    lse, p_rest = torch.empty_like(loss), torch.empty_like(loss)
    _call("distill_topk_fused", dev, x, pi, pt, K, _on(mask, torch.uint8, R, "mask", dev),
          _on(dloss, torch.float32, R, "dloss", dev), float(T), float(beta), bool(tail), loss.data_ptr(), lse.data_ptr(),
          p_rest.data_ptr(), dx, _on(dev_err, torch.int32, 1, "dev_err", dev))
    return {"loss": loss, "lse": lse, "p_rest": p_rest, "dlogits": dlogits}


# ---------------------------------------------------------------------------
# preference loss on pairs; the norm of many gradients
# ---------------------------------------------------------------------------

_PREF_ARGS = struct.Struct("=diiffffi4x")
assert _PREF_ARGS.size == ctypes.sizeof(GrpoPrefArgs)


def _pref(logits, idx, ref_logp, mask, T, beta, kind, label_smoothing, gamma, average, sft_weight):
    """(rows, idx, ref, mask, args) for the C call, the number of pairs and of rows."""
    x, B, L, _ = _pack_rows(logits)
    if logits.dim() != 3 or B % 2:
        raise ValueError("logits must be [2 P, L, V]: the chosen sequences, then the rejected ones")
    if kind not in GRPO_PREF_KINDS:
        raise ValueError(f"kind must be one of {', '.join(GRPO_PREF_KINDS)}, got {kind!r}")
    dev = logits.device
    args = _PREF_ARGS.pack(T, GRPO_PREF_KINDS[kind], bool(average), beta, gamma, label_smoothing, sft_weight, 0)
    return (x, _on(idx, torch.int64, B * L, "idx", dev), _on(ref_logp, torch.float32, B, "ref_logp", dev),
            _on(mask, torch.uint8, B * L, "mask", dev), args), B // 2, B * L


def _pref_out(P, R, dev):
    # tensors of their own, not parts of one: autograd keeps some of them, and a caller may change the
    # others in place
    f32 = dict(dtype=torch.float32, device=dev)
    # (logp: with a second row of what its rounding lost, for the sums)
    reward, lse = torch.empty(2 * P, **f32), torch.empty(R, **f32)
    out = {"loss": torch.empty(P, **f32), "reward": reward, "seq_logp": torch.empty_like(reward),
           "coef": torch.empty_like(reward), "logp": torch.empty(2 * R, **f32)[:R], "lse": lse}
    return out, [t.data_ptr() for t in out.values()]


def preference_loss_fwd(logits, idx, *, T=1.0, beta=0.1, kind="sigmoid", label_smoothing=0.0, gamma=0.0,
                        average=False, sft_weight=0.0, ref_logp=None, mask=None, dev_err=None):
    """Preference loss of P pairs from [2P, L, V] logits (the chosen sequences, then the rejected
    ones): dict with loss [P], reward, seq_logp and coef [2P] (coef is what the backward needs),
    logp and lse [2P*L].  kind: "sigmoid" (with label_smoothing), "hinge" or "squared";
    average: mean log-probs instead of sums; ref_logp [2P]: the reference policy's, summed or
    averaged alike; sft_weight: of the chosen sequence's mean negative log-prob."""
    a, P, R = _pref(logits, idx, ref_logp, mask, T, beta, kind, label_smoothing, gamma, average, sft_weight)
    dev = logits.device
    out, at = _pref_out(P, R, dev)
    _call("preference_loss_fwd", dev, *a, *at, _on(dev_err, torch.int32, 1, "dev_err", dev))
    return out


def preference_loss_bwd(logits, idx, dloss, coef, lse, *, T=1.0, mask=None, dlogits=None, dev_err=None):
    """dlogits of sum_i dloss_i * loss_i, with coef and lse of preference_loss_fwd (allocated like
    logits unless given; ``dlogits=logits`` works in place)."""
    x, B, L, _ = _pack_rows(logits)
    dev, f32 = logits.device, torch.float32
    if logits.dim() != 3 or B % 2:
        raise ValueError("logits must be [2 P, L, V]: the chosen sequences, then the rejected ones")
    dlogits, dx = _like(dlogits, logits, "dlogits")
    _call("preference_loss_bwd", dev, x, _on(idx, torch.int64, B * L, "idx", dev),
          _on(mask, torch.uint8, B * L, "mask", dev), _on(dloss, f32, B // 2, "dloss", dev),
          _on(coef, f32, B, "coef", dev), _on(lse, f32, B * L, "lse", dev), float(T), dx,
          _on(dev_err, torch.int32, 1, "dev_err", dev))
    return dlogits


def preference_loss_fused(logits, idx, dloss, *, T=1.0, beta=0.1, kind="sigmoid", label_smoothing=0.0, gamma=0.0,
                          average=False, sft_weight=0.0, ref_logp=None, mask=None, dlogits=None, dev_err=None):
    """preference_loss_fwd and preference_loss_bwd in one call, for loss weights dloss [P] known in
    advance; returns the forward's dict plus "dlogits"."""
    a, P, R = _pref(logits, idx, ref_logp, mask, T, beta, kind, label_smoothing, gamma, average, sft_weight)
    dev = logits.device
    dlogits, dx = _like(dlogits, logits, "dlogits")
    out, at = _pref_out(P, R, dev)
    x, pi, pr, pm, args = a
    _call("preference_loss_fused", dev, x, pi, pr, pm, _on(dloss, torch.float32, P, "dloss", dev), args, *at, dx,
          _on(dev_err, torch.int32, 1, "dev_err", dev))
    out["dlogits"] = dlogits
    return out


_ptrs_of, _numels_of, _devices_of = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.get_device
_dtype_of = attrgetter("dtype")
_contiguous, _NONE = torch.Tensor.is_contiguous, type(None)


def grad_dtypes(grads, dev):
    """The dtypes of contiguous tensors on ``dev`` (a model has hundreds: one sweep an attribute)."""
    index = dev.index if dev.type == "cuda" else -2
    if list(map(_devices_of, grads)).count(index) != len(grads):
        raise ValueError(f"gradients must be CUDA tensors on {dev if index >= 0 else 'one device'}")
    if not all(map(_contiguous, grads)):
        raise ValueError("gradients must be contiguous")
    return list(map(_dtype_of, grads))


def dtype_words(dtypes):
    try:
        if dtypes and dtypes.count(dtypes[0]) == len(dtypes):
            return array("Q", [_DTYPES[dtypes[0]]]) * len(dtypes)
        return array("Q", [_DTYPES[d] for d in dtypes])
    except KeyError as e:
        raise TypeError(f"gradient dtype {e} not supported (bf16 or fp32)") from None


def norm_of_table(pointers, counts, words, dev, norm=None):
    n = len(pointers)
    table = array("Q", bytes(24 * n))
    table[0::3], table[1::3], table[2::3] = pointers, counts, words
    work = torch.empty(GRPO_GRAD_NORM_WORKSPACE, dtype=torch.uint8, device=dev)
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=dev)
    _call("grad_norm", dev, table.buffer_info()[0], n, _on(norm, torch.float32, 1, "norm", dev), work.data_ptr(),
          GRPO_GRAD_NORM_WORKSPACE)
    return norm


def grad_norm(grads, *, norm=None):
    """sqrt of the sum of squares over all elements of the tensors (contiguous, bf16 or fp32; None is
    passed over): a 0-dim fp32 tensor (allocated unless given).  Right for every finite input; inf or
    NaN where an element is."""
    grads = list(grads)
    if _NONE in set(map(type, grads)):
        grads = [g for g in grads if g is not None]
    if not grads:
        raise ValueError("grad_norm needs a tensor")
    dev = grads[0].device
    words = dtype_words(grad_dtypes(grads, dev))
    return norm_of_table(array("Q", map(_ptrs_of, grads)), array("Q", map(_numels_of, grads)), words, dev, norm)
