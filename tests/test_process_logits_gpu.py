"""process_logits_fwd / _bwd against the fp64 oracle.

Tolerance: a value is formed by at most five fp32 operations (penalty division or product,
frequency FMA, presence, bias), each off by at most 2^-24 of a partial sum no larger than
``size`` (the sum of the terms' magnitudes), and rounded once: 5 * 2^-24 * size plus half a step
of the output type.  The gradient is one operation: 2^-24 of the value plus half a step.
"""
import numpy as np
import pytest
import torch

import rl_fine_tuning_pass_gb300 as rl
from logits_ops_util import DEV, HALF, close, f64, place, randn, same_bits, untouched
from oracle import logits_ops_oracle as lo
from rl_fine_tuning_pass_gb300 import binding as rp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


def make_rules(B, L, V, seed, N=40, M=6, mask=True, penalties=True, growing=True):
    """Rules on the host: histories with repeats, empty places and a shared hot token; biases
    with a column listed twice and an unused entry; masks from nothing to all allowed."""
    g = np.random.default_rng(seed)
    k = {}
    if penalties:
        hot = g.integers(0, V, 4)
        tokens = np.where(g.random((B, N)) < 0.4, hot[g.integers(0, 4, (B, N))], g.integers(0, V, (B, N)))
        tokens[g.random((B, N)) < 0.05] = -1
        first = g.integers(0, max(1, N - L), B)
        hist = np.minimum(N, first[:, None] + np.arange(L)) if growing else g.integers(0, N + 1, (B, L))
        k.update(tokens=tokens, hist_len=hist.reshape(-1).astype(np.int32), prompt_len=first.astype(np.int32),
                 repetition=(1.0 + g.random(B)).astype(np.float32), frequency=g.normal(size=B).astype(np.float32),
                 presence=g.normal(size=B).astype(np.float32))
    if M:
        ids = g.integers(0, V, (B, M))
        ids[:, -1] = -1
        if M > 2:
            ids[:, 1] = ids[:, 0]
        k.update(bias_ids=ids, bias=g.normal(size=(B, M)).astype(np.float32) * 3)
    if mask:
        W = (V + 31) // 32
        bits = g.random((B * L, W * 32)) < g.choice([0.02, 0.5, 0.97, 1.0], B * L)[:, None]
        bits[0] = False                                  # nothing allowed
        k["allowed"] = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
    return k


def on_gpu(k):
    return {n: torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for n, v in k.items()}


def check(x, k, out_layout="dense", what="", dev=None):
    """Forward and backward of GPU logits x under host rules k."""
    B, L, V = x.shape
    d = on_gpu(k) if dev is None else dev
    half = HALF[x.dtype]
    out, buf = place(torch.zeros(B, L, V, dtype=x.dtype), out_layout)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert rp.process_logits_fwd(x, **d, out=out, dev_err=err) is out
    y, size = lo.process_logits(f64(x), L, **k)
    close(out, y, 5 * 2.0 ** -24 * size + half * np.abs(np.where(np.isfinite(y), y, 0)), what + " out")
    untouched(buf, out)
    dy = randn(B, L, V, seed=5).to(x.dtype).to(DEV)
    dx, buf = place(torch.zeros(B, L, V, dtype=x.dtype), out_layout)
    rp.process_logits_bwd(x, dy, **d, dlogits=dx, dev_err=err)
    want = lo.process_logits_bwd(f64(x), f64(dy), L, **{n: v for n, v in k.items()
                                                      if n not in ("frequency", "presence", "bias", "bias_ids")})
    close(dx, want, (2.0 ** -24 + half) * np.abs(want), what + " dlogits")
    untouched(buf, dx)
    return out, dx, int(err.item())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 32, 33, 64, 1003, 16384, 16400, 32003])
def test_vocabularies(dtype, V):
    x, _ = place((randn(2, 3, V, seed=V) * 3).to(dtype), "dense")
    assert check(x, make_rules(2, 3, V, V), what=f"V={V}")[2] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["cut", "odd", "phase"])
@pytest.mark.parametrize("out_layout", ["dense", "odd", "phase"])
def test_layouts(dtype, layout, out_layout):
    x, _ = place((randn(3, 5, 2051, seed=1) * 3).to(dtype), layout)
    check(x, make_rules(3, 5, 2051, 2), out_layout, f"{layout}->{out_layout}")


@pytest.mark.parametrize("part", ["penalties", "bias", "mask", "nothing", "all"])
@pytest.mark.parametrize("growing", [True, False])
def test_each_rule_alone(part, growing):
    x, _ = place((randn(2, 9, 515, seed=3) * 3).to(torch.bfloat16), "dense")
    k = make_rules(2, 9, 515, 4, M=6 if part in ("bias", "all") else 0, mask=part in ("mask", "all"),
                   penalties=part in ("penalties", "all"), growing=growing)
    check(x, k, what=part)


@pytest.mark.parametrize("name", ["repetition", "frequency", "presence", "hist_len", "prompt_len"])
@pytest.mark.parametrize("only", [True, False])
def test_optional_arrays(name, only):
    k = make_rules(2, 6, 300, 7, mask=False)
    if only:   # this one alone, with the tokens
        k = {n: v for n, v in k.items() if n in ("tokens", name)}
    else:
        del k[name]
    x, _ = place((randn(2, 6, 300, seed=3) * 3), "dense")
    check(x, k, what=name)


@pytest.mark.parametrize("N", [0, 1, 2, 255, 256, 257, 5000])
def test_history_lengths(N):
    V = 777
    x, _ = place((randn(2, 1, V, seed=9) * 3).to(torch.bfloat16), "dense")
    k = make_rules(2, 1, V, N, N=max(N, 1), mask=False)
    if N == 0:
        k["tokens"], k["hist_len"] = k["tokens"][:, :0], np.zeros(2, np.int32)
    check(x, k, what=f"N={N}")


@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 70])
def test_runs_of_rows(L):
    """Growing, standing and falling histories along a sequence, some of them empty."""
    B, V = 3, 1030
    k = make_rules(B, L, V, L, N=90, mask=False)
    h = k["hist_len"].reshape(B, L)
    h[1] = 17
    h[2] = np.arange(L)[::-1] % 23
    x, _ = place((randn(B, L, V, seed=2) * 3).to(torch.bfloat16), "dense")
    check(x, k, what=f"L={L}")
    x, _ = place((randn(B, L, V, seed=2) * 3), "odd")
    check(x, k, "phase", what=f"L={L} odd")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["dense", "odd"])
def test_in_place_equals_out_of_place(dtype, layout):
    x, buf = place((randn(3, 4, 1003, seed=11) * 3).to(dtype), layout)
    for k in (make_rules(3, 4, 1003, 1), make_rules(3, 4, 1003, 2, mask=False), make_rules(3, 4, 1003, 3, M=0)):
        d = on_gpu(k)
        y, _ = place(x.cpu(), layout)
        want = rp.process_logits_fwd(x, **d)
        rp.process_logits_fwd(y, **d, out=y)
        same_bits(y, want, "in place")
        dy = randn(3, 4, 1003, seed=5).to(dtype).to(DEV)
        want = rp.process_logits_bwd(x, dy, **d)
        dx = dy.clone()
        rp.process_logits_bwd(x, dx, **d, dlogits=dx)
        same_bits(dx, want, "in place over dout")
        with pytest.raises(rp.GrpoError):       # not over the logits
            rp.process_logits_bwd(x, dy, **d, dlogits=x)
    untouched(buf, x)


def test_forbidden_places_hold_anything():
    """NaN, infinities and the type's lowest value in forbidden columns, in the logits and in
    the gradient, leave -inf and +0.0 there and change nothing else; allowed ones pass through."""
    V = 203
    x = randn(1, 4, V, seed=1).to(torch.bfloat16)
    bad = [float("nan"), float("inf"), float("-inf"), torch.finfo(torch.bfloat16).min, 0.0, -0.0]
    x[0, :, :6] = torch.tensor(bad)
    x[0, :, 100:106] = torch.tensor(bad)
    bits = np.ones((4, 224), bool)
    bits[:, :6] = False
    k = make_rules(1, 4, V, 3, mask=False)
    k["tokens"][0, :12] = np.r_[0:6, 100:106]
    k["hist_len"][:] = [0, 12, 20, 40]
    k["allowed"] = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
    d = on_gpu(k)
    xg = x.to(DEV)
    out = rp.process_logits_fwd(xg, **d)
    assert bool((out[0, :, :6] == float("-inf")).all())
    y, size = lo.process_logits(f64(xg), 4, **k)
    size = np.where(np.isfinite(size), size, 0)
    # the lowest bf16 value times a penalty above 1 is past (2 - 2^-8) 2^127, where bf16 rounds
    # to infinity
    y = np.where(np.abs(y) >= (2 - 2.0 ** -8) * 2.0 ** 127, np.copysign(np.inf, y), y)
    close(out, y, 5 * 2.0 ** -24 * size + 2.0 ** -8 * np.abs(np.where(np.isfinite(y), y, 0)), "out")
    dy = randn(1, 4, V, seed=2).to(torch.bfloat16).to(DEV)
    dy[0, :, :6] = torch.tensor(bad)
    dx = rp.process_logits_bwd(xg, dy, **d)
    assert int((dx[0, :, :6].contiguous().view(torch.int16) != 0).sum()) == 0


def test_ids_and_lengths_out_of_range():
    """Ids past the vocabulary and lengths past the tokens set the error bit; the rest of the
    row is as without them."""
    V = 130
    x, _ = place(randn(2, 3, V, seed=1), "dense")
    for name, at, value in [("tokens", (0, 0), V), ("tokens", (1, 1), 1 << 40), ("bias_ids", (1, 0), V + 3),
                            ("hist_len", 2, 41), ("hist_len", 4, -3), ("hist_len", 1, np.iinfo(np.int32).max),
                            ("hist_len", 0, np.iinfo(np.int32).min)]:
        k = make_rules(2, 3, V, 8, mask=False)
        k["prompt_len"][:] = 0
        k["hist_len"][:] = 40
        k[name][at] = value
        assert check(x, k, what=name)[2] == rp.GRPO_DEVERR_IDX_OUT_OF_RANGE
    k = make_rules(2, 3, V, 8, mask=False)
    k["prompt_len"][:] = [-5, 1 << 20]          # a prompt length is only compared
    assert check(x, k, what="prompt_len")[2] == 0


def test_more_touched_columns_than_are_listed():
    """Histories that touch most columns of a tile."""
    V = 9000
    x, _ = place((randn(2, 3, V, seed=1) * 2).to(torch.bfloat16), "odd")
    k = make_rules(2, 3, V, 1, N=20000, growing=False)
    k["hist_len"][:] = [20000, 19000, 2500, 0, 2000, 2300]
    check(x, k, "phase", "many touched")
    y = x.clone()
    rp.process_logits_fwd(y, **on_gpu(k), out=y)
    same_bits(y, rp.process_logits_fwd(x, **on_gpu(k)), "in place")


def test_shared_histories_and_masks():
    """One history and one mask for every sequence, as expanded views."""
    B, L, V = 3, 4, 515
    k = make_rules(1, 1, V, 1)
    k["allowed"] = make_rules(1, 2, V, 1)["allowed"][1:]
    x, _ = place((randn(B, L, V, seed=4) * 2).to(torch.bfloat16), "dense")
    wide = {n: np.repeat(v, B, 0) for n, v in k.items() if n not in ("hist_len", "allowed")}
    wide["allowed"] = np.repeat(k["allowed"], B * L, 0)
    d = on_gpu(wide)
    d["tokens"] = on_gpu(k)["tokens"].expand(B, -1)
    d["allowed"] = on_gpu(k)["allowed"][None].expand(B, L, -1)
    assert d["tokens"].stride(0) == 0 and d["allowed"].stride(0) == 0
    check(x, wide, dev=d)


def test_large_vocabulary_and_far_rows():
    """Every column of a vocabulary of 600001, and rows more than 2^31 elements apart."""
    V = 600001
    x, _ = place((randn(1, 2, V, seed=6) * 2).to(torch.bfloat16), "dense")
    check(x, make_rules(1, 2, V, 5, N=3000), what="V=600001")
    V, far = 40, (1 << 31) + 24
    buf = torch.empty(far + 64, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(buf, (2, 1, V), (far, V, 1))
    x.copy_(randn(2, 1, V, seed=7))
    k = make_rules(2, 1, V, 5)
    d = on_gpu(k)
    want = rp.process_logits_fwd(x.clone(), **d)
    rp.process_logits_fwd(x, **d, out=x)
    same_bits(x.clone(), want, "far rows")


def test_counts_are_exact_and_results_repeat():
    """One token thousands of times: the count is exact, and two calls give the same bits."""
    V, N = 5000, 60000
    tokens = np.full((1, N), 4321)
    tokens[0, ::7] = np.arange(len(tokens[0, ::7])) % V
    k = dict(tokens=tokens, frequency=np.array([2.0 ** -10], np.float32), repetition=np.array([1.5], np.float32),
             prompt_len=np.array([10], np.int32))
    x, _ = place(randn(1, 1, V, seed=6), "dense")
    a, da, _ = check(x, k)
    b, db, _ = check(x, k)
    same_bits(a, b, "out")
    same_bits(da, db, "dlogits")


def test_autograd_and_other_streams():
    B, L, V = 2, 3, 301
    k = make_rules(B, L, V, 3)
    d = on_gpu(k)
    x = (randn(B, L, V, seed=1) * 2).to(DEV).requires_grad_(True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w = randn(B, L, V, seed=2).to(DEV)
    with torch.cuda.stream(s):
        y = rl.process_logits(x, **d)
        (y.masked_fill(y.isinf(), 0.0) * w).sum().backward()
    torch.cuda.current_stream().wait_stream(s)
    same_bits(y.detach(), rp.process_logits_fwd(x.detach(), **d), "y")
    dy = torch.where(torch.isinf(y.detach()), 0.0, w)
    same_bits(x.grad, rp.process_logits_bwd(x.detach(), dy, **d), "grad")
    x.grad = None
    k.pop("allowed")
    rl.process_logits(x, **on_gpu(k)).sum().backward()      # an expanded gradient of ones
    want = lo.process_logits_bwd(f64(x), np.ones((B * L, V)), L, tokens=k["tokens"], hist_len=k["hist_len"],
                                 repetition=k["repetition"])
    close(x.grad, want, 2.0 ** -23 * np.abs(want), "grad of the sum")
    x.grad = None                                            # without a repetition penalty the logits are not kept
    few = {n: v for n, v in on_gpu(k).items() if n != "repetition"}
    h = x * 1.0
    y = rl.process_logits(h, **few)
    with torch.no_grad():
        h.zero_()
    y.sum().backward()
    assert bool((x.grad == 1.0).all())
    with pytest.raises(RuntimeError):                        # no second derivative is offered
        g, = torch.autograd.grad(rl.process_logits(x, **d).sum(), x, create_graph=True)
        g.sum().backward()


def test_captured_and_replayed():
    """Both passes in a CUDA graph follow the lengths, masks and logits of the replay."""
    B, L, V = 2, 5, 1003
    k = make_rules(B, L, V, 3)
    d = on_gpu(k)
    x = (randn(B, L, V, seed=1) * 2).to(torch.bfloat16).to(DEV)
    dy = randn(B, L, V, seed=2).to(torch.bfloat16).to(DEV)
    out, dx = torch.empty_like(x), torch.empty_like(x)

    def both(o, g):
        rp.process_logits_fwd(x, **d, out=o)
        rp.process_logits_bwd(x, dy, **d, dlogits=g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both(out, dx)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(out, dx)
    for n in range(2):
        x.copy_(randn(B, L, V, seed=10 + n))
        d["hist_len"].sub_(n).clamp_(min=0)
        d["allowed"].bitwise_not_()
        graph.replay()
        a, b = torch.empty_like(x), torch.empty_like(x)
        both(a, b)
        same_bits(out, a, "out")
        same_bits(dx, b, "dlogits")
