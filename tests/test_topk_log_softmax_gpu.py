"""topk_log_softmax against the fp64 oracle: ids exactly, log-probs within 1e-5 + 1e-5 |value|
(fp32: x c - a is off by 2^-24 of at most |z - max| log2 e, ln s by 2^-23 |ln s| and the sum's
own error of some 2^-20, as in the other forward passes)."""
import numpy as np
import pytest
import torch

from logits_ops_util import DEV, close, f64, place, randn, same_bits
from oracle import logits_ops_oracle as lo
from rl_fine_tuning_pass_gb300 import binding as rp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


def check(x, K, T=1.0, what=""):
    ids, logp, lse = rp.topk_log_softmax(x, K, T=T)
    o_ids, o_logp, o_lse = lo.topk_log_softmax(f64(x), K, float(np.float32(T)))
    got = ids.cpu().numpy()
    bad = np.nonzero((got != o_ids).any(1))[0]
    assert len(bad) == 0, f"{what}: row {bad[0]}: {got[bad[0]]} for {o_ids[bad[0]]}"
    close(logp, o_logp, 1e-5 + 1e-5 * np.abs(np.nan_to_num(o_logp)), what + " logp")
    close(lse, o_lse, 1e-5 + 1e-5 * np.abs(np.nan_to_num(o_lse, neginf=0, posinf=0)), what + " lse")
    return ids, logp, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,K", [(1, 1), (2, 2), (7, 3), (8, 8), (33, 32), (255, 255), (256, 256), (257, 256),
                                 (1003, 20), (4099, 128), (32000, 64), (50001, 5), (151936, 1), (151936, 256)])
def test_sizes(dtype, V, K):
    x, _ = place((randn(2, 2, V, seed=V) * 3).to(dtype), "dense")
    check(x, K, 0.7, f"V={V} K={K}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["cut", "odd", "phase"])
@pytest.mark.parametrize("R", [(1, 1), (3, 7), (2, 400)])
def test_layouts_and_row_counts(dtype, layout, R):
    x, _ = place((randn(*R, 3001, seed=1) * 3).to(dtype), layout)
    check(x, 37, 1.0, layout)


def rows_of_kind(kind, V, g):
    n = torch.arange(V, dtype=torch.float32)
    if kind == "constant":
        return torch.full((V,), 1.5)
    if kind == "two values":
        return (n % 3 == 0).float()
    if kind == "rising":
        return n / 64
    if kind == "falling":
        return -n / 64
    if kind == "few allowed":
        return torch.where(torch.rand(V, generator=g) < 10 / V, torch.randn(V, generator=g), -torch.inf)
    if kind == "one allowed, last":
        return torch.where(n == V - 1, 2.0, -torch.inf)
    if kind == "block":       # the largest side by side, at the end
        return torch.randn(V, generator=g) + 50.0 * (n >= V - 300)
    if kind == "zeros of both signs":
        return torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)
    if kind == "lowest":
        return torch.full((V,), torch.finfo(torch.bfloat16).min)
    if kind == "tiny":
        return torch.randn(V, generator=g) * 1e-39
    if kind == "ties at the border":
        return torch.where(torch.rand(V, generator=g) < 0.02, 3.0, torch.randn(V, generator=g).clamp(max=2.0))
    if kind == "one thread's columns":   # a stride at which one thread may meet all the large ones
        return torch.randn(V, generator=g) + 30.0 * (n % 2048 < 8)
    raise ValueError(kind)


KINDS = ["constant", "two values", "rising", "falling", "few allowed", "one allowed, last", "block",
         "zeros of both signs", "lowest", "tiny", "ties at the border", "one thread's columns"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,K", [(300, 17), (20011, 64), (151936, 200)])
def test_hard_rows(dtype, kind, V, K):
    g = torch.Generator().manual_seed(V)
    r = rows_of_kind(kind, V, g)
    x = torch.stack([r, torch.randn(V, generator=g), r.flip(0)])[None].to(dtype).to(DEV)
    check(x, K, 1.0, kind)


def test_hard_rows_among_many():
    """The same in a batch large enough for the launch of many rows."""
    g = torch.Generator().manual_seed(3)
    V = 40003
    x = torch.stack([rows_of_kind(KINDS[i % len(KINDS)], V, g) if i % 7 == 0 else torch.randn(V, generator=g) * 2
                     for i in range(1400)])
    rows = np.unique(np.r_[np.arange(0, 1400, 7)[:60], np.arange(0, 1400, 131)])
    for dtype in (torch.bfloat16, torch.float32):
        xd = x.to(dtype).to(DEV)
        ids, logp, lse = rp.topk_log_softmax(xd, 50)
        o_ids, o_logp, o_lse = lo.topk_log_softmax(f64(xd[torch.from_numpy(rows).to(DEV)]), 50, 1.0)
        assert np.array_equal(ids.cpu().numpy()[rows], o_ids)
        at = torch.from_numpy(rows).to(DEV)
        close(logp[at], o_logp, 1e-5 + 1e-5 * np.abs(o_logp), "logp")


@pytest.mark.parametrize("R,V,dtype", [(400, 140003, torch.float32), (310, 600011, torch.bfloat16),
                                       (1, 2200003, torch.float32), (2, 2200003, torch.bfloat16)])
@pytest.mark.parametrize("K", [7, 200])
def test_rows_whose_chunks_are_several_steps(R, V, dtype, K):
    # the row as a whole, and (few rows) the parts of a cluster
    g = torch.Generator(device=DEV).manual_seed(V)
    x = (torch.randn(R, V, generator=g, device=DEV) * 3).to(dtype)
    x[0] = torch.arange(V, device=DEV) / 64    # rising: the largest come last, in one thread's chunks or a few
    ids, logp, lse = rp.topk_log_softmax(x, K)
    for r in {0, R // 2, R - 1}:
        o_ids, o_logp, o_lse = lo.topk_log_softmax(f64(x[r:r + 1]), K, 1.0)
        assert np.array_equal(ids[r:r + 1].cpu().numpy(), o_ids)
        close(logp[r:r + 1], o_logp, 1e-5 + 1e-5 * np.abs(o_logp), "logp")
        close(lse[r:r + 1], o_lse, 1e-5 + 1e-5 * np.abs(o_lse), "lse")


def test_rows_without_log_probs():
    """NaN, +inf, all -inf: ids 0..K-1 and NaN log-probs; the lse says why."""
    x = randn(1, 6, 500, seed=1)
    x[0, 0, 77] = float("nan")
    x[0, 1, 499] = float("inf")
    x[0, 2] = float("-inf")
    x[0, 3, :490] = float("-inf")
    x[0, 4, 0] = float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        ids, logp, lse = rp.topk_log_softmax(x.to(dtype).to(DEV), 9)
        for r in (0, 1, 2, 4):
            assert ids[r].tolist() == list(range(9)) and bool(logp[r].isnan().all())
        assert float(lse[2]) == float("-inf") and bool(lse[[0, 1, 4]].isnan().all())
        check(x[:, [3, 5]].to(dtype).to(DEV), 9)


@pytest.mark.parametrize("R", [1, 20, 70, 150, 400])
def test_masked_rows_at_every_split(R):
    """Rows left with a few columns (and fewer than K), at the row counts of each number of CTAs."""
    V, K = 33003, 30
    g = torch.Generator().manual_seed(R)
    x = torch.randn(1, R, V, generator=g)
    x[0, ::3] = torch.where(torch.rand(x[0, ::3].shape, generator=g) < 12 / V, x[0, ::3], -torch.inf)
    x[0, ::3, V - 1] = 1.0
    rows = np.unique(np.r_[0, np.arange(0, R, 37), R - 1])
    for dtype in (torch.bfloat16, torch.float32):
        xd = x.to(dtype).to(DEV)
        ids, logp, _ = rp.topk_log_softmax(xd, K)
        o_ids, o_logp, _ = lo.topk_log_softmax(f64(xd[0, torch.from_numpy(rows).to(DEV)]), K, 1.0)
        assert np.array_equal(ids.cpu().numpy()[rows], o_ids)
        close(logp[torch.from_numpy(rows).to(DEV)], o_logp, 1e-5 + 1e-5 * np.abs(np.nan_to_num(o_logp, neginf=0)),
              "logp")


@pytest.mark.parametrize("T", [0.05, 1.0, 50.0])
def test_temperatures(T):
    x, _ = place(randn(1, 5, 7001, seed=2) * 4, "dense")
    check(x, 33, T)


def test_no_rows_and_repeats():
    ids, logp, lse = rp.topk_log_softmax(torch.empty(2, 0, 64, device=DEV), 5)
    assert ids.shape == (0, 5) and logp.shape == (0, 5) and lse.shape == (0,)
    for shape in ((1, 1, 151936), (4, 500, 8003)):
        x = (torch.randn(*shape, generator=torch.Generator().manual_seed(1)) * 2).to(torch.bfloat16).to(DEV)
        a, b = rp.topk_log_softmax(x, 100), rp.topk_log_softmax(x, 100)
        for u, v in zip(a, b):
            same_bits(u, v, "repeat")


def test_far_rows():
    far, V = (1 << 31) + 24, 700
    buf = torch.empty(far + 1024, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(buf, (2, 1, V), (far, V, 1))
    x.copy_(randn(2, 1, V, seed=3))
    check(x, 10)


def test_captured_replayed_and_on_two_streams():
    xs = [(randn(2, 3, 9001, seed=s) * 2).to(torch.bfloat16).to(DEV) for s in (1, 2)]
    want = [rp.topk_log_softmax(x, 40, T=0.9) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for x, s in zip(xs, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(rp.topk_log_softmax(x, 40, T=0.9))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for u, v in zip(a, b):
            same_bits(u, v, "streams")
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rp.topk_log_softmax(x, 40, T=0.9)
    for src, w in zip(xs[::-1], want[::-1]):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(out, w):
            same_bits(u, v, "replay")
