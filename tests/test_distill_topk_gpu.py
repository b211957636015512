"""distill_topk_fwd / _bwd / _fused against the fp64 oracle.

Tolerances.  The student's bucket masses come from a sum of V exponentials in fp32: a thread adds
at most a few hundred terms one after another (2^-24 each), the exponent's FMA and the rounded
log2(e) / T move a term by up to 2^-24 |z - max| log2(e) < 2^-18 relative, so a mass is within
EPS = 2e-5 of itself, and lse within 2e-5 + 2^-23 |lse|.  Then
  loss:    sum_b |dL/dlog p_b| EPS = G EPS, plus 2^-20 of the terms' magnitudes (logs and products)
  p_rest:  EPS p_rest
  dlogits: with g = dloss / T, at an unlisted column |g| p_j (2 |F| + G + 1) 2 EPS, at a listed one
           |g| (|G_k| + (2 + G) p_k) 2 EPS (G_k = p_k * a log-ratio, off by p_k EPS (1 + the ratio);
           bounded below through G and the loss terms), plus half a step of the output type.
G, F and the terms come from the oracle.
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
EPS = 2e-5
WAYS = [(0.0, False), (0.0, True), (0.3, False), (0.5, True), (1.0, True)]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


def teacher(x, K, seed, noise=0.7, unused=True):
    """ids and log-probs [R, K] of the top of logits near x (host tensors)."""
    B, L, V = x.shape
    t = (x.double() + noise * randn(B, L, V, seed=seed).double()).reshape(-1, V)
    top = t.topk(K, dim=1)
    ids, lp = top.indices, (top.values - torch.logsumexp(t, 1, keepdim=True)).float()
    if unused and K > 2:
        ids[1::3, K // 2] = -1
        lp[1::3, K // 2] = float("nan")
    return ids.contiguous(), lp.contiguous()


def tolerances(o, x, ids, dloss, T, half):
    R, V = x.shape
    with np.errstate(over="ignore", invalid="ignore"):   # rows that are not read: nothing allowed
        p = np.exp(x / T - o["lse"][:, None])
    p = np.nan_to_num(p, nan=0.0, posinf=0.0)
    g = np.abs(np.nan_to_num(dloss)) / T
    t = {"loss": EPS * o["G"] + 2.0 ** -20 * o["terms"] + 1e-7, "lse": EPS + 2.0 ** -23 * np.abs(o["lse"]),
         "p_rest": EPS * o["p_rest"] + 1e-30}
    col = p * (2 * o["F"] + o["G"] + 1)[:, None]
    for r in range(R):
        for i in ids[r]:
            if 0 <= i < V:
                # |G_k| <= |d_k| T / dloss + p_k |S|
                d = abs(o["dlogits"][r, i]) / g[r] if g[r] > 0 else 0.0
                col[r, i] = d + (3 + 2 * o["G"][r]) * p[r, i]
    t["dlogits"] = 2 * EPS * g[:, None] * col + half * np.abs(np.nan_to_num(o["dlogits"])) + 2.0 ** -126
    return t


def check(x, ids, lp, T=1.0, beta=0.0, tail=False, mask=None, dloss=None, out_layout="dense", what=""):
    B, L, V = x.shape
    R = B * L
    T = float(np.float32(T))
    if dloss is None:
        dloss = randn(R, seed=99)
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    how = dict(T=T, beta=beta, tail=tail, mask=d(mask))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = rp.distill_topk_fwd(x, d(ids), d(lp), **how, dev_err=err)
    dl, buf = place(torch.zeros(B, L, V, dtype=x.dtype), out_layout)
    rp.distill_topk_bwd(x, d(ids), d(lp), d(dloss), out["lse"], out["p_rest"], **how, dlogits=dl)
    xs = f64(x)
    o = lo.distill_topk(xs, ids.numpy(), lp.numpy(), T, float(np.float32(beta)), tail,
                        None if mask is None else mask.numpy(), dloss.double().numpy())
    tol = tolerances({k: np.nan_to_num(v) for k, v in o.items()}, xs, ids.numpy(), dloss.double().numpy(), T,
                     HALF[x.dtype])
    for k in ("loss", "lse", "p_rest"):
        close(out[k], o[k], tol[k], f"{what} {k}")
    close(dl, o["dlogits"], tol["dlogits"], f"{what} dlogits")
    untouched(buf, dl)
    fl, fbuf = place(torch.zeros(B, L, V, dtype=x.dtype), out_layout)
    fused = rp.distill_topk_fused(x, d(ids), d(lp), d(dloss), **how, dlogits=fl, dev_err=err)
    for k in ("loss", "lse", "p_rest"):
        close(fused[k], o[k], tol[k], f"{what} fused {k}")
    close(fused["dlogits"], o["dlogits"], tol["dlogits"], f"{what} fused dlogits")
    untouched(fbuf, fl)
    return out, dl, int(err.item())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("beta,tail", WAYS)
@pytest.mark.parametrize("V,K", [(1, 1), (7, 7), (9, 4), (64, 1), (512, 8), (1003, 256), (5001, 64), (32003, 100)])
def test_sizes(dtype, beta, tail, V, K):
    x = (randn(2, 3, V, seed=V) * 2).to(dtype)
    ids, lp = teacher(x, K, 1)
    assert check(x.to(DEV), ids, lp, 0.8, beta, tail, what=f"V={V} K={K}")[2] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["cut", "odd", "phase"])
@pytest.mark.parametrize("out_layout", ["dense", "odd", "phase"])
def test_layouts(dtype, layout, out_layout):
    x, _ = place((randn(3, 4, 2051, seed=1) * 2).to(dtype), layout)
    ids, lp = teacher(x.cpu(), 33, 2)
    check(x, ids, lp, 1.0, 0.4, True, out_layout=out_layout, what=f"{layout}->{out_layout}")


@pytest.mark.parametrize("beta,tail", WAYS)
def test_long_rows(beta, tail):
    for dtype, V in ((torch.bfloat16, 151936), (torch.float32, 151935), (torch.bfloat16, 300007)):
        x = (randn(1, 3, V, seed=V) * 2).to(dtype)
        x[0, 1, 5] += 20.0
        ids, lp = teacher(x, 64, 3)
        check(x.to(DEV), ids, lp, 1.0, beta, tail, what=f"V={V}")


@pytest.mark.parametrize("R", [5, 180, 400, 1200])
@pytest.mark.parametrize("dtype,V,layout", [(torch.bfloat16, 70003, "cut"), (torch.float32, 40001, "odd")])
def test_row_counts(R, dtype, V, layout):
    """Batches of every split of rows over CTAs (clusters in the forward, parts in the backward),
    masked rows among them: some rows against the oracle, every row against the rows alone."""
    x, _ = place((randn(1, R, V, seed=R) * 2).to(dtype), layout)
    ids, lp = teacher(x.cpu(), 20, 1)
    ids[:, 0] = torch.where(ids[:, 1] != 0, 0, ids[:, 0])                # the first column
    ids[:, 2] = torch.where((ids != V - 1).all(1), V - 1, ids[:, 2])     # and the last one
    dup = torch.tensor([len(set(r.tolist()) - {-1}) < int((r >= 0).sum()) for r in ids])
    ids[dup] = torch.arange(20)                                          # no column twice
    mask = (torch.arange(R) % 7 != 3).to(torch.uint8)
    w = randn(R, seed=3)
    d = lambda t: t.to(DEV)  # noqa: E731
    how = dict(T=0.8, beta=0.5, tail=True)
    f = rp.distill_topk_fwd(x, d(ids), d(lp), **how, mask=d(mask))
    dl = rp.distill_topk_bwd(x, d(ids), d(lp), d(w), f["lse"], f["p_rest"], **how, mask=d(mask))
    fused = rp.distill_topk_fused(x, d(ids), d(lp), d(w), **how, mask=d(mask))
    rows = np.unique(np.r_[0, 3, R // 2, R - 1, np.arange(0, R, 97)])
    at = torch.from_numpy(rows)
    xs, T = f64(x[0, at.to(DEV)]), float(np.float32(0.8))
    o = lo.distill_topk(xs, ids[at].numpy(), lp[at].numpy(), T, 0.5, True, mask[at].numpy(), w[at].double().numpy())
    tol = tolerances(o, xs, ids[at].numpy(), w[at].double().numpy(), T, HALF[dtype])
    for out, grad in ((f, dl), (fused, fused["dlogits"])):
        for k in ("loss", "lse", "p_rest"):
            close(out[k][at.to(DEV)], o[k], tol[k], k)
        close(grad[0, at.to(DEV)], o["dlogits"], tol["dlogits"], "dlogits")
    # every row: the fused and the separate passes agree (two sums, each within its bound of the row)
    big = fused["dlogits"][0].float().abs().amax(1, keepdim=True).clamp(min=1e-30)
    assert bool(((fused["dlogits"][0].float() - dl[0].float()).abs() <= big * (4 * HALF[dtype] + 2e-4)).all())
    assert bool(((fused["loss"] - f["loss"]).abs() <= 1e-4 * (1 + f["loss"].abs())).all())


@pytest.mark.parametrize("beta,tail", WAYS)
def test_confident_students(beta, tail):
    """The list holds all but a sliver of the student's mass, or nearly none of it."""
    V, K = 4000, 16
    x = randn(1, 6, V, seed=5)
    for r, up in enumerate((8.0, 16.0, 30.0, 60.0, 83.0)):
        x[0, r, 100:100 + K] += up
    x[0, 5, 3000] += 30.0
    ids = torch.arange(100, 100 + K).repeat(6, 1)
    lp = torch.log_softmax(randn(6, K + 1, seed=6) * 2, 1)[:, :K].contiguous()
    check(x.to(DEV), ids, lp, 1.0, beta, tail, what="confident")


def test_masks_zero_weights_and_unused_slots():
    x = (randn(2, 4, 700, seed=1) * 2).to(torch.bfloat16)
    ids, lp = teacher(x, 9, 4)
    mask = torch.tensor([1, 0, 1, 1, 1, 1, 0, 1], dtype=torch.uint8)
    dloss = torch.tensor([1.0, 5.0, 0.0, -0.0, -2.0, 1e-30, 1.0, 0.5])
    ids[4] = -1                                  # nothing listed
    bad = x.clone()
    bad[0, 1] = float("nan")                     # a masked row's logits are not read
    for beta, tail in WAYS:
        out, dl, err = check(bad.to(DEV), ids, lp, 0.9, beta, tail, mask, dloss, what=f"masked {beta} {tail}")
        assert err == 0
        flat = dl.reshape(8, -1)
        for r in (1, 2, 3, 6):
            assert int((flat[r].view(torch.int16) != 0).sum()) == 0, f"row {r} is not +0.0"
        for k in ("loss", "lse", "p_rest"):
            assert int((out[k][[1, 6]].view(torch.int32) != 0).sum()) == 0
        if tail:
            assert abs(float(out["loss"][4])) < 1e-6


@pytest.mark.parametrize("V", [100, 300007])
def test_ids_out_of_range_and_listed_twice(V):
    x = randn(1, 5, V, seed=1)
    for beta, tail in WAYS:
        ids, lp = teacher(x, 6, 4, unused=False)
        assert check(x.to(DEV), ids, lp, 1.0, beta, tail)[2] == 0
        ids[1, 2] = V
        assert check(x.to(DEV), ids, lp, 1.0, beta, tail)[2] == rp.GRPO_DEVERR_IDX_OUT_OF_RANGE
        ids[3, 5] = ids[3, 0]
        assert check(x.to(DEV), ids, lp, 1.0, beta, tail)[2] == \
            rp.GRPO_DEVERR_IDX_OUT_OF_RANGE | rp.GRPO_DEVERR_DUPLICATE_ID
        ids[1, 2] = 1 << 40
        check(x.to(DEV), ids, lp, 1.0, beta, tail)


def test_columns_that_share_a_place_in_the_filter():
    """Columns a multiple of 262144 apart, one of each pair listed."""
    V = 3 * 262144 + 5
    x = randn(1, 2, V, seed=3)
    lp = torch.log_softmax(randn(2, 6, seed=1), 1)[:, :5].contiguous()
    ids = torch.tensor([[0, 262144 + 7, 2 * 262144 + 9, V - 1, 5]] * 2)
    ids[1, 0] = 262144 + 5
    x[0, :, 262144] = 9.0
    x[0, :, 7] = 9.0
    for beta, tail in WAYS:
        for dtype in (torch.float32, torch.bfloat16):
            assert check(x.to(dtype).to(DEV), ids, lp, 1.0, beta, tail)[2] == 0


@pytest.mark.parametrize("beta,tail", WAYS)
def test_infinities_and_nan(beta, tail):
    """-inf logits have no mass; NaN and +inf make the row NaN; a listed column without mass."""
    V, K = 300, 5
    x = randn(1, 4, V, seed=2)
    x[0, 0, 50:] = float("-inf")
    x[0, 1, 7] = float("nan")
    x[0, 2, 8] = float("inf")
    ids, lp = teacher(torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=-50.0), K, 1, unused=False)
    ids[3, 0] = 60 if 60 not in ids[3].tolist() else ids[3, 0]
    d = lambda t: t.to(DEV)  # noqa: E731
    w = torch.ones(4, device=DEV)
    out = rp.distill_topk_fused(d(x), d(ids), d(lp), w, beta=beta, tail=tail)
    for k in ("loss", "lse", "p_rest"):
        assert bool(out[k][1:3].isnan().all()), k
    assert bool(out["dlogits"][0, 1:3].isnan().all())
    keep = [0, 3]
    check(d(x[:, keep]), ids[keep], lp[keep], 1.0, beta, tail, what="-inf")
    if beta == 0.0:   # a teacher's token that the student gives no mass: infinite, with a finite gradient
        x[0, 0, int(ids[0, 0])] = float("-inf")
        out = rp.distill_topk_fused(d(x), d(ids), d(lp), w, beta=beta, tail=tail)
        assert float(out["loss"][0]) == float("inf") and bool(out["dlogits"][0, 0].isfinite().all())


@pytest.mark.parametrize("beta,tail", WAYS)
def test_listed_columns_without_mass(beta, tail):
    """Listed columns whose student logit is -inf: no part of the loss but the teacher's, no NaN in
    the row; forward, backward and fused."""
    x = randn(1, 3, 500, seed=2)
    ids, lp = teacher(x, 7, 1, unused=False)
    lp[:, 3] = float("-inf")                 # the teacher gives it none either
    x[0, 0, int(ids[0, 3])] = float("-inf")
    x[0, 1, int(ids[1, 3])] = -1e30
    check(x.to(DEV), ids, lp, 0.7, beta, tail, what="no mass")
    if beta < 1.0 and beta > 0.0:            # the mixture is finite where only the student has none
        lp[:, 3] = -2.0 - torch.arange(3.0)
        x[0, 2, int(ids[2, 3])] = float("-inf")
        check(x.to(DEV), ids, lp, 0.7, beta, tail, what="teacher's mass only")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_columns_at_the_lowest_value(dtype):
    """Columns set to the type's lowest value have no mass, listed ones among them; whole threads
    may meet nothing else."""
    V, K = 9001, 12
    x = (randn(1, 4, V, seed=2) * 2).to(dtype)
    x[0, 0, 20:] = torch.finfo(dtype).min
    x[0, 1, :-3] = torch.finfo(dtype).min
    x[0, 2, ::2] = torch.finfo(dtype).min
    ids, lp = teacher(randn(1, 4, V, seed=9), K, 1)
    ids[0, :2] = torch.tensor([3, 4])
    for beta, tail in ((0.3, False), (0.5, True)):
        check(x.to(DEV), ids, lp, 1.0, beta, tail, what="lowest")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_and_repeats(dtype):
    x = (randn(2, 5, 3001, seed=1) * 2).to(dtype)
    ids, lp = (t.to(DEV) for t in teacher(x, 20, 2))
    w = randn(10, seed=3).to(DEV)
    xg = x.to(DEV)
    how = dict(T=0.9, beta=0.5, tail=True)
    f = rp.distill_topk_fwd(xg, ids, lp, **how)
    want = rp.distill_topk_bwd(xg, ids, lp, w, f["lse"], f["p_rest"], **how)
    same_bits(rp.distill_topk_bwd(xg, ids, lp, w, f["lse"], f["p_rest"], **how), want, "repeat")
    y = xg.clone()
    rp.distill_topk_bwd(y, ids, lp, w, f["lse"], f["p_rest"], **how, dlogits=y)
    same_bits(y, want, "in place")
    a = rp.distill_topk_fused(xg, ids, lp, w, **how)
    y = xg.clone()
    b = rp.distill_topk_fused(y, ids, lp, w, **how, dlogits=y)
    for k in a:
        same_bits(a[k], b[k], f"fused in place {k}")


def test_far_rows():
    far, V = (1 << 31) + 24, 700
    buf = torch.empty(far + 1024, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(buf, (2, 1, V), (far, V, 1))
    x.copy_(randn(2, 1, V, seed=3))
    ids, lp = teacher(x.cpu(), 10, 1)
    check(x, ids, lp, 1.0, 0.5, True)


def test_autograd_against_the_oracle_and_differences():
    x = (randn(2, 3, 401, seed=4) * 2).to(DEV).requires_grad_(True)
    ids, lp = teacher(x.detach().cpu(), 12, 5)
    w = randn(6, seed=6)
    loss, p_rest = rl.distill_topk_loss(x, ids.to(DEV), lp.to(DEV), T=0.8, beta=0.3, tail=True)
    assert not p_rest.requires_grad
    (loss * w.to(DEV)).sum().backward()
    T = float(np.float32(0.8))
    xs = f64(x)
    o = lo.distill_topk(xs, ids.numpy(), lp.numpy(), T, float(np.float32(0.3)), True, None, w.double().numpy())
    close(x.grad, o["dlogits"], tolerances(o, xs, ids.numpy(), w.double().numpy(), T, 2.0 ** -24)["dlogits"], "grad")
    h = 1e-5
    e = randn(6, 401, seed=8).double().numpy()
    up, dn = (lo.distill_topk(xs + s * h * e, ids.numpy(), lp.numpy(), T, 0.3, True)["loss"] for s in (1, -1))
    along = ((up - dn) * w.double().numpy()).sum() / (2 * h)
    assert abs(along - (x.grad.double().cpu().numpy().reshape(6, -1) * e).sum()) < 1e-3 * abs(along) + 1e-4
    x.grad = None
    rl.distill_topk_loss(x, ids.to(DEV), lp.to(DEV))[0].sum().backward()   # an expanded gradient
    assert bool(x.grad.isfinite().all())
    with pytest.raises(RuntimeError):                                      # no second derivative is offered
        g, = torch.autograd.grad(rl.distill_topk_loss(x, ids.to(DEV), lp.to(DEV))[0].sum(), x, create_graph=True)
        g.sum().backward()


@pytest.mark.parametrize("dtype,V", [(torch.float32, 100003), (torch.bfloat16, 151936)])
@pytest.mark.parametrize("R", [1, 3, 40, 200])
def test_few_rows_in_place(R, V, dtype):
    # a row that several CTAs would share: none may read a listed logit that another has overwritten
    x = (randn(1, R, V, seed=R) * 2).to(dtype).to(DEV)
    ids, lp, _ = rp.topk_log_softmax(x, 256)
    lp = (lp - 0.5).contiguous()
    w = randn(R, seed=3).to(DEV)
    how = dict(T=0.9, beta=0.3, tail=True)
    f = rp.distill_topk_fwd(x, ids, lp, **how)
    want = rp.distill_topk_bwd(x, ids, lp, w, f["lse"], f["p_rest"], **how)
    for _ in range(20):
        y = x.clone()
        rp.distill_topk_bwd(y, ids, lp, w, f["lse"], f["p_rest"], **how, dlogits=y)
        same_bits(y, want, "dlogits")


def test_captured_and_replayed():
    x = (randn(2, 5, 3001, seed=1) * 2).to(torch.bfloat16)
    ids, lp = (t.to(DEV) for t in teacher(x, 20, 2))
    w = randn(10, seed=3).to(DEV)
    xg = x.to(DEV)
    how = dict(T=0.9, beta=0.5, tail=True)

    def step():
        f = rp.distill_topk_fwd(xg, ids, lp, **how)
        f["dlogits"] = rp.distill_topk_bwd(xg, ids, lp, w, f["lse"], f["p_rest"], **how)
        return f, rp.distill_topk_fused(xg, ids, lp, w, **how)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in range(2):
        xg.copy_(randn(2, 5, 3001, seed=20 + n))
        graph.replay()
        want = step()
        for a, b in zip(got, want):
            for k in b:
                same_bits(a[k], b[k], k)
