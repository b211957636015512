"""The sampler-rules, top-log-probs and distillation entry points on the CPU: bad arguments are
refused on the host before any launch (fake device addresses are never dereferenced), and the
Python functions refuse tensors that the library cannot take."""
import ctypes
import math

import pytest
import torch

from rl_fine_tuning_pass_gb300 import autograd as ag
from rl_fine_tuning_pass_gb300 import binding
from rl_fine_tuning_pass_gb300.build import build

FAKE = 0x7F0000100000
FAR = FAKE + (1 << 20)
OK, INV, UNS = binding.GRPO_OK, binding.GRPO_ERR_INVALID_ARG, binding.GRPO_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load_library()


def rows(ptr=FAKE, dtype=binding.GRPO_BF16, B=2, L=3, V=64, sb=None, sl=None):
    sl = V if sl is None else sl
    return binding.GrpoRows(ptr, dtype, 0, B, L, V, L * sl if sb is None else sb, sl)


def rules(**kw):
    q = binding.GrpoLogitRules()
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def fwd(lib, q, x=None, y=None, err=None):
    return lib.process_logits_fwd(ctypes.byref(x or rows()), None if q is None else ctypes.byref(q),
                                  ctypes.byref(y or rows(FAR)), err, None)


def bwd(lib, q, x=None, dy=None, dx=None):
    return lib.process_logits_bwd(ctypes.byref(x or rows()), ctypes.byref(dy or rows(FAKE + (1 << 16))),
                                  ctypes.byref(q), ctypes.byref(dx or rows(FAR)), None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=3), INV), (dict(N=-1), INV), (dict(N=3, tokens=FAKE + 4), INV),
    (dict(N=3, tokens=FAKE, tokens_stride=-3), INV), (dict(N=1 << 19, tokens=FAKE), UNS),
    (dict(N=3, tokens=FAKE, hist_len=FAKE + 2), INV), (dict(N=3, tokens=FAKE, prompt_len=FAKE + 1), INV),
    (dict(N=3, tokens=FAKE, repetition=FAKE + 2), INV), (dict(N=3, tokens=FAKE, frequency=FAKE + 2), INV),
    (dict(N=3, tokens=FAKE, presence=FAKE + 2), INV), (dict(M=-1), INV), (dict(M=2), INV),
    (dict(M=2, bias_ids=FAKE), INV), (dict(M=2, bias=FAKE), INV), (dict(M=1 << 12, bias_ids=FAKE, bias=FAKE), UNS),
    (dict(allowed=FAKE + 2), INV), (dict(allowed=FAKE, allowed_stride_b=-1), INV),
    (dict(allowed=FAKE, allowed_stride_l=-1), INV), (dict(allowed=FAKE, allowed_stride_b=1 << 60), INV),
])
def test_rules_refused(lib, kw, want):
    assert fwd(lib, rules(**kw)) == want
    assert bwd(lib, rules(**kw)) == want


def test_rules_tensors_refused(lib):
    assert fwd(lib, None) == INV
    q = rules()
    assert fwd(lib, q, err=FAKE + 1) == INV
    assert fwd(lib, q, y=rows(FAKE + 64)) == INV                       # overlaps the logits in part
    assert fwd(lib, q, y=rows(FAR, V=32)) == INV
    assert fwd(lib, q, y=rows(FAR, sl=16)) == INV                      # rows of the output overlap
    assert fwd(lib, q, x=rows(dtype=9)) == INV
    assert bwd(lib, q, dy=rows(FAKE + (1 << 16), V=63)) == INV
    assert bwd(lib, q, dy=rows(FAKE + (1 << 16), dtype=binding.GRPO_FP32)) == INV
    assert bwd(lib, q, dx=rows(FAKE + 64)) == INV                      # overlaps the logits in part
    assert bwd(lib, q, dx=rows(FAKE + (1 << 16) + 64)) == INV          # overlaps the gradient in part
    assert fwd(lib, q, x=rows(None, B=0), y=rows(None, B=0)) == OK     # no rows: nothing launched


def test_topk_refused(lib):
    def call(x=None, K=4, T=1.0, ids=FAR, logp=FAR, lse=FAR):
        return lib.topk_log_softmax(ctypes.byref(x or rows()), K, T, ids, logp, lse, None)
    assert call(K=0) == INV
    assert call(K=65) == INV                      # more than the vocabulary
    assert call(x=rows(V=1000), K=257) == UNS
    assert call(T=0.0) == INV and call(T=math.nan) == INV
    assert call(ids=None) == INV and call(ids=FAR + 4) == INV
    assert call(logp=None) == INV and call(lse=FAR + 2) == INV
    assert call(x=rows(None, B=0), ids=None, logp=None, lse=None) == OK


def test_distill_refused(lib):
    def three(x=None, ids=FAR, tl=FAR, K=4, T=1.0, beta=0.0, tail=0, dx=None, s=FAR, dloss=FAR):
        xr, dr = x or rows(), dx or rows(FAR)
        return (lib.distill_topk_fwd(ctypes.byref(xr), ids, tl, K, None, T, beta, tail, s, s, s, None, None),
                lib.distill_topk_bwd(ctypes.byref(xr), ids, tl, K, None, dloss, s, s, T, beta, tail, ctypes.byref(dr),
                                     None),
                lib.distill_topk_fused(ctypes.byref(xr), ids, tl, K, None, dloss, T, beta, tail, s, s, s,
                                       ctypes.byref(dr), None, None))
    for kw, want in [(dict(K=0), INV), (dict(K=257), UNS), (dict(T=0.0), INV), (dict(T=math.inf), INV),
                     (dict(beta=-0.1), INV), (dict(beta=1.1), INV), (dict(beta=math.nan), INV),
                     (dict(beta=1.0, tail=0), INV), (dict(ids=None), INV), (dict(ids=FAR + 4), INV),
                     (dict(tl=None), INV), (dict(tl=FAR + 1), INV), (dict(s=None), INV), (dict(s=FAR + 2), INV),
                     (dict(x=rows(V=0)), INV)]:
        assert three(**kw) == (want,) * 3, kw
    for kw in (dict(dloss=None), dict(dx=rows(FAKE + 64)), dict(dx=rows(FAR, V=63)), dict(dx=rows(FAR, sl=8))):
        assert three(**kw)[1:] == (INV, INV), kw
    assert three(x=rows(None, B=0), dx=rows(None, B=0), ids=None, tl=None, s=None, dloss=None) == (OK,) * 3


def test_python_functions_refuse_cpu_tensors():
    x = torch.randn(2, 3, 8, requires_grad=True)
    ids, tl = torch.zeros(6, 2, dtype=torch.int64), torch.zeros(6, 2)
    with pytest.raises(ValueError, match="CUDA"):
        ag.process_logits(x)
    with pytest.raises(ValueError, match="CUDA"):
        binding.topk_log_softmax(x, 2)
    with pytest.raises(ValueError, match="CUDA"):
        ag.distill_topk_loss(x, ids, tl)


@pytest.mark.parametrize("kw,match", [
    (dict(tokens=torch.zeros(3, 4, dtype=torch.int64)), "tokens"),
    (dict(tokens=torch.zeros(2, 4, dtype=torch.int32)), "tokens"),
    (dict(tokens=torch.zeros(4, 2, dtype=torch.int64).t()), "stride 1"),
    (dict(repetition=torch.ones(2)), "need tokens"), (dict(hist_len=torch.ones(6)), "need tokens"),
    (dict(bias_ids=torch.zeros(2, 3, dtype=torch.int64)), "go together"),
    (dict(bias=torch.zeros(2, 3)), "go together"),
    (dict(bias_ids=torch.zeros(2, 3, dtype=torch.int64), bias=torch.zeros(2, 4)), r"\[B, M\]"),
    (dict(allowed=torch.zeros(5, 2, dtype=torch.int32)), "allowed"),
    (dict(allowed=torch.zeros(6, 1, dtype=torch.int32)), "2 words"),
    (dict(allowed=torch.zeros(6, 2, dtype=torch.int64)), "int32"),
    (dict(allowed=torch.zeros(6, 4, dtype=torch.int32)[:, ::2]), "stride 1"),
])
def test_python_rules_refused(kw, match):
    full = dict.fromkeys(("tokens", "hist_len", "prompt_len", "repetition", "frequency", "presence", "bias_ids",
                          "bias", "allowed"))
    with pytest.raises(ValueError, match=match):
        binding._rules(2, 3, 64, torch.device("cpu"), **{**full, **kw})


def described(*args, **kw):
    return binding.GrpoLogitRules.from_buffer_copy(binding._rules(*args, **kw))


def test_rules_are_packed_as_the_c_structure():
    t = lambda *n, dt=torch.float32: torch.zeros(*n, dtype=dt)  # noqa: E731
    kw = dict(tokens=t(2, 9, dt=torch.int64)[:, :7], hist_len=t(6, dt=torch.int32), prompt_len=t(2, dt=torch.int32),
              repetition=t(2), frequency=t(2), presence=t(2), bias_ids=t(2, 5, dt=torch.int64), bias=t(2, 5),
              allowed=t(2, 3, 4, dt=torch.int32))
    q = described(2, 3, 64, torch.device("cpu"), **kw)
    for name, v in kw.items():
        assert getattr(q, name) == v.data_ptr(), name
    assert (q.tokens_stride, q.N, q.M, q.allowed_stride_b, q.allowed_stride_l) == (9, 7, 5, 12, 4)


def test_expanded_masks_are_described_by_their_strides():
    full = dict.fromkeys(("tokens", "hist_len", "prompt_len", "repetition", "frequency", "presence", "bias_ids",
                          "bias"))
    one = torch.zeros(1, 1, 2, dtype=torch.int32)
    q = described(2, 3, 64, torch.device("cpu"), allowed=one.expand(2, 3, 2), **full)
    assert (q.allowed_stride_b, q.allowed_stride_l) == (0, 0)
    q = described(2, 3, 64, torch.device("cpu"), allowed=torch.zeros(6, 5, dtype=torch.int32), **full)
    assert (q.allowed_stride_b, q.allowed_stride_l) == (15, 5)
