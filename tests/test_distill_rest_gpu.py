"""Rows whose columns outside the teacher's list hold no mass at all: nothing is left for a bucket
of the rest, and the teacher is renormalised over its list.  Tolerances as in
test_distill_topk_gpu.py."""
import numpy as np
import pytest
import torch

import rl_fine_tuning_pass_gb300 as rl
from logits_ops_util import DEV, f64, randn
from oracle import logits_ops_oracle as lo
from rl_fine_tuning_pass_gb300 import binding as rp
from test_distill_topk_gpu import EPS, WAYS, check

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("beta,tail", WAYS)
@pytest.mark.parametrize("V", [1, 7, 255])
def test_every_column_listed(dtype, beta, tail, V):
    """A student equal to its teacher has neither a loss nor a gradient; another one has both."""
    x = (randn(1, 4, V, seed=V) * 3).to(dtype)
    ids = torch.stack([torch.randperm(V, generator=torch.Generator().manual_seed(r)) for r in range(4)])
    T = float(np.float32(0.7))
    lp = torch.log_softmax(x[0].double() / T, 1).gather(1, ids).float()
    w = torch.ones(4)
    out, dl, err = check(x.to(DEV), ids, lp, T, beta, tail, dloss=w, what="equal")
    assert err == 0 and bool((out["p_rest"] == 0).all())
    # the loss and the gradient within the bounds of their terms: G = 0, each q log q below 1/2
    assert bool((out["loss"].abs() <= 2.0 ** -20 * V + 1e-7).all())
    assert bool((dl.float().abs() <= 2 * EPS * 4 / T).all())
    check(x.to(DEV), ids, torch.log_softmax(randn(4, V, seed=3) * 2, 1), T, beta, tail, what="other")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("beta,tail", WAYS)
@pytest.mark.parametrize("R,V", [(3, 700), (3, 151936), (1200, 5001), (1, 300007)])
def test_nothing_allowed_outside_the_list(dtype, beta, tail, R, V):
    """Every unlisted column is -inf, in every launch shape; a row beside them has a rest."""
    K = 12
    g = torch.Generator().manual_seed(V)
    x = torch.full((1, R, V), float("-inf"))
    ids = torch.randperm(V, generator=g)[:K].repeat(R, 1)
    x.scatter_(2, ids[None], randn(1, R, K, seed=1) * 3)
    x[0, 0, ids[0, 4]] = float("-inf")
    if R > 1:
        x[0, R // 2] = randn(V, seed=2)
    lp = torch.log_softmax(randn(R, K, seed=3) * 2, 1) - 1e-3 * torch.rand(R, 1, generator=g)
    lp[0, 4] = float("-inf")
    ids[:, 7], lp[:, 7] = -1, float("nan")       # its column stays without a listing: -inf as well
    x[0, :, torch.randperm(V, generator=torch.Generator().manual_seed(V))[7]] = float("-inf")
    x, lp = x.to(dtype), lp.contiguous()
    if R <= 3:
        assert check(x.to(DEV), ids, lp, 0.9, beta, tail, what="no rest")[2] == 0
        return
    rows = torch.tensor([0, 1, R // 2, R - 1])
    d = lambda t: t.to(DEV)  # noqa: E731
    w = torch.ones(R)
    how = dict(T=0.9, beta=beta, tail=tail)
    f = rp.distill_topk_fwd(d(x), d(ids), d(lp), **how)
    dl = rp.distill_topk_bwd(d(x), d(ids), d(lp), d(w), f["lse"], f["p_rest"], **how)
    u = rp.distill_topk_fused(d(x), d(ids), d(lp), d(w), **how)
    few, fdl, _ = check(d(x[:, rows]), ids[rows], lp[rows], 0.9, beta, tail, dloss=w[rows], what="no rest")
    at = rows.to(DEV)
    for a, b in ((f["loss"][at], few["loss"]), (u["loss"][at], few["loss"]), (dl[0, at], fdl[0]),
                 (u["dlogits"][0, at], fdl[0])):
        assert bool(((a.float() - b.float()).abs() <= 1e-5 + (2.0 ** -7) * b.float().abs()).all())
    assert bool(f["loss"].isfinite().all()) and bool(dl.isfinite().all()) and bool(u["dlogits"].isfinite().all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("beta,tail", WAYS)
def test_a_grammar_bound_step(dtype, beta, tail):
    """Student and teacher under one mask, some positions with fewer allowed tokens than the list is
    long: rules, the teacher's list, the divergence and its gradient back through the rules."""
    B, L, V, K = 2, 3, 1003, 20
    R = B * L
    x = (randn(B, L, V, seed=1) * 2).to(dtype).to(DEV).requires_grad_(True)
    t = (x.detach().float().cpu() + 0.5 * randn(B, L, V, seed=2)).to(dtype).to(DEV)
    bits = np.random.default_rng(3).random((R, (V + 31) // 32 * 32)) < 0.5
    for r, n in ((0, 8), (2, 1), (3, 20), (5, 21)):
        bits[r] = False
        bits[r, 17 * np.arange(n) + r] = True
    allowed = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32)).to(DEV)
    y = rl.process_logits(x, allowed=allowed)
    ids, lp, _ = rl.topk_log_softmax(rl.process_logits_fwd(t, allowed=allowed), K)
    div, p_rest = rl.distill_topk_loss(y, ids, lp, beta=beta, tail=tail)
    div.sum().backward()
    assert bool(div.isfinite().all()) and bool(x.grad.isfinite().all())
    few = torch.tensor([0, 2, 3])
    assert bool((p_rest[few.to(DEV)] == 0).all()) and int((p_rest == 0).sum()) == 3
    o = lo.distill_topk(f64(y), ids.cpu().numpy(), lp.cpu().numpy(), 1.0, float(np.float32(beta)), tail, None, np.ones(R))
    got = div.detach().double().cpu().numpy()
    assert np.all(np.abs(got - o["loss"]) <= EPS * o["G"] + 2.0 ** -20 * o["terms"] + 1e-7)
    # each element: the passes' 2 EPS of |g| (|G_k| + (2 + G) p) <= 8 G + 8, and half a step of the type
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    tol = 16 * EPS * (1 + o["G"][:, None]) + 2 * half * np.abs(o["dlogits"])
    assert np.all(np.abs(f64(x.grad) - o["dlogits"]) <= tol)
    assert int((f64(x.grad)[~bits[:, :V]] != 0).sum()) == 0
    assert abs(got[2]) <= 1e-6                       # one token left: both give it everything
