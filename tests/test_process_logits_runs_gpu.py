"""The sampler's rules on batches whose CTAs take runs of several rows (up to eight): the history
that follows a run, the ring of stages, masks in the stages.  Some rows against the fp64 oracle,
and every row against calls of few rows, whose CTAs take one row each."""
import numpy as np
import pytest
import torch

from logits_ops_util import DEV, HALF, close, f64, place, randn, same_bits, untouched
from oracle import logits_ops_oracle as lo
from rl_fine_tuning_pass_gb300 import binding as rp
from test_process_logits_gpu import make_rules, on_gpu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


def rows_of(k, b, l0, l1, L):
    """The rules of rows [l0, l1) of sequence b as a batch of one sequence."""
    q = {n: v[b:b + 1] for n, v in k.items() if n not in ("hist_len", "allowed")}
    if "hist_len" in k:
        q["hist_len"] = k["hist_len"][b * L + l0:b * L + l1]
    if "allowed" in k:
        q["allowed"] = k["allowed"][b * L + l0:b * L + l1]
    return q


def check_runs(x, dy, k, rows, out_layout="dense"):
    """x, dy: GPU [B, L, V]; k: rules on the host; rows: (b, l) compared with the oracle."""
    B, L, V = x.shape
    d, half = on_gpu(k), HALF[x.dtype]
    out, obuf = place(torch.zeros(B, L, V, dtype=x.dtype), out_layout)
    dx, dbuf = place(torch.zeros(B, L, V, dtype=x.dtype), out_layout)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    rp.process_logits_fwd(x, **d, out=out, dev_err=err)
    rp.process_logits_bwd(x, dy, **d, dlogits=dx, dev_err=err)
    assert int(err.item()) == 0
    untouched(obuf, out)
    untouched(dbuf, dx)
    for b, l in rows:
        q = rows_of(k, b, l, l + 1, L)
        y, size = lo.process_logits(f64(x[b:b + 1, l]), 1, **q)
        close(out[b:b + 1, l], y, 5 * 2.0 ** -24 * size + half * np.abs(np.where(np.isfinite(y), y, 0)), f"out {b},{l}")
        want = lo.process_logits_bwd(f64(x[b:b + 1, l]), f64(dy[b:b + 1, l]), 1,
                                     **{n: v for n, v in q.items() if n not in ("frequency", "presence", "bias", "bias_ids")})
        close(dx[b:b + 1, l], want, (2.0 ** -24 + half) * np.abs(want), f"dlogits {b},{l}")
    step = 300
    for b in range(B):
        for l0 in range(0, L, step):
            l1 = min(L, l0 + step)
            q = {n: (v[b:b + 1] if n not in ("hist_len", "allowed") else v[b * L + l0:b * L + l1]) for n, v in d.items()}
            xs = x[b:b + 1, l0:l1].contiguous()
            same_bits(out[b:b + 1, l0:l1], rp.process_logits_fwd(xs, **q), f"rows {b}, {l0}..")
            same_bits(dx[b:b + 1, l0:l1], rp.process_logits_bwd(xs, dy[b:b + 1, l0:l1].contiguous(), **q), f"dlogits {b}, {l0}..")
    y = x.clone()
    same_bits(rp.process_logits_fwd(y, **d, out=y), out, "in place")
    g = dy.clone()
    same_bits(rp.process_logits_bwd(x, g, **d, dlogits=g), dx, "in place over dout")


def lengths(kind, L, N, g):
    """Histories along a sequence."""
    if kind == "growing":
        return np.minimum(N, np.arange(L) + 3)
    if kind == "standing and falling":
        return np.where(np.arange(L) % 5 < 3, N // 2, N // 2 - np.arange(L) % 7)
    if kind == "jumping":      # past the tokens that are held ready, and back
        return (np.arange(L) * 293) % (N + 1)
    return g.integers(0, N + 1, L)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("layout,out_layout", [("dense", "dense"), ("odd", "odd"), ("cut", "phase")])
@pytest.mark.parametrize("B,L,V", [(3, 900, 1032), (3, 1700, 1030), (2, 7000, 517), (2, 1000, 9001)])
def test_runs(dtype, mask, layout, out_layout, B, L, V):
    g = np.random.default_rng(L + V)
    N = L + 40
    k = make_rules(B, L, V, L + V, N=N, mask=mask)
    for b, kind in enumerate(("growing", "jumping", "standing and falling")[:B]):
        k["hist_len"].reshape(B, L)[b] = lengths(kind, L, N, g)
    x, _ = place((randn(B, L, V, seed=2) * 3).to(dtype), layout)
    dy, _ = place(randn(B, L, V, seed=5).to(dtype), layout if layout != "cut" else "dense")
    rows = [(b, int(l)) for b in range(B) for l in np.r_[0:9, L // 2:L // 2 + 5, L - 3:L]]
    check_runs(x, dy, k, rows, out_layout)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("order", ["growing", "any"])
def test_touched_columns_past_the_list_within_a_run(dtype, mask, order):
    """Histories that come to touch more columns of a tile than are listed, row after row."""
    B, L, V, N = 1, 6000, 4096, 2600
    k = make_rules(B, L, V, 3, N=N, mask=mask)
    g = np.random.default_rng(4)
    k["tokens"][0] = g.permutation(V)[:N]
    # rows around the list's length, one token more each, over and over
    k["hist_len"][:] = (2040 + np.arange(L) % 24) if order == "growing" else g.integers(1900, N + 1, L)
    x = (randn(B, L, V, seed=1) * 2).to(dtype).to(DEV)
    dy = randn(B, L, V, seed=2).to(dtype).to(DEV)
    check_runs(x, dy, k, [(0, int(l)) for l in np.r_[0:40, 3000:3010, L - 8:L]])


@pytest.mark.parametrize("part", ["penalties", "bias", "mask", "nothing"])
def test_one_rule_in_runs(part):
    B, L, V = 2, 2500, 2056
    k = make_rules(B, L, V, 4, N=L, M=6 if part == "bias" else 0, mask=part == "mask", penalties=part == "penalties")
    x = (randn(B, L, V, seed=1) * 2).to(torch.bfloat16).to(DEV)
    dy = randn(B, L, V, seed=2).to(torch.bfloat16).to(DEV)
    check_runs(x, dy, k, [(b, l) for b in range(B) for l in (0, 1, 7, 8, 1000, L - 1)])


def test_bad_tokens_met_within_a_run():
    """An id past the vocabulary that comes in at a run's later row sets the error bit."""
    B, L, V = 1, 6000, 1032
    k = make_rules(B, L, V, 4, N=L, mask=False)
    k["hist_len"][:] = np.minimum(np.arange(L), 3005)
    k["tokens"][0, 3003] = V
    x = randn(B, L, V, seed=1).to(torch.bfloat16).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = rp.process_logits_fwd(x, **on_gpu(k), dev_err=err)
    assert int(err.item()) == rp.GRPO_DEVERR_IDX_OUT_OF_RANGE
    k["tokens"][0, 3003] = -1
    err.zero_()
    same_bits(rp.process_logits_fwd(x, **on_gpu(k), dev_err=err), y, "skipped")
    assert int(err.item()) == 0


def test_runs_captured_and_replayed():
    B, L, V = 2, 2500, 2056
    k = make_rules(B, L, V, 4, N=L, mask=True)
    d = on_gpu(k)
    x = (randn(B, L, V, seed=1) * 2).to(torch.bfloat16).to(DEV)
    dy = randn(B, L, V, seed=2).to(torch.bfloat16).to(DEV)
    out, dx = torch.empty_like(x), torch.empty_like(x)

    def both(o, g):
        rp.process_logits_fwd(x, **d, out=o)
        rp.process_logits_bwd(x, dy, **d, dlogits=g)
    both(out, dx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(out, dx)
    for n in range(2):
        d["hist_len"].add_(300 * n).clamp_(max=L)
        d["allowed"].bitwise_not_()
        graph.replay()
        a, b = torch.empty_like(x), torch.empty_like(x)
        both(a, b)
        same_bits(out, a, "out")
        same_bits(dx, b, "dlogits")
