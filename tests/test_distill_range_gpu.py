"""The distillation where the student's mass of the rest, or of a listed column, is below what fp32
can hold: log-ratios stay finite and the unlisted columns' gradient -g q_rest p_j / p_rest keeps its
size.  Tolerances as in test_distill_topk_gpu.py: they come from the 64-bit oracle, whose masses
reach e^-700."""
import numpy as np
import pytest
import torch

from logits_ops_util import DEV, HALF, close, f64, place, randn, same_bits
from oracle import logits_ops_oracle as lo
from rl_fine_tuning_pass_gb300 import binding as rp
from test_distill_topk_gpu import WAYS, check, teacher, tolerances

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
# the lift of the list over the rest, in units of T; 87.3 + log(V) / 2 is where p_rest leaves fp32's
# normal numbers, 103 + where it is 0
UPS = (84.0, 88.0, 92.0, 95.0, 97.0, 100.0, 103.0, 110.0, 120.0, 200.0, 600.0)


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


def teacher_of_four(R):
    return torch.arange(100, 104).repeat(R, 1), torch.tensor([[0.5, 0.2, 0.15, 0.1]]).log().repeat(R, 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("beta,tail", WAYS)
@pytest.mark.parametrize("V,T", [(4000, 1.0), (4000, 0.05), (30011, 0.6), (151936, 1.0)])
@pytest.mark.parametrize("whole", [True, False])
def test_confident_students(dtype, beta, tail, V, T, whole):
    """The whole list, or its first column alone, far above everything else."""
    x = randn(1, len(UPS), V, seed=5) * T
    for r, up in enumerate(UPS):
        x[0, r, 100:104 if whole else 101] += up * T
    ids, lp = teacher_of_four(len(UPS))
    check(x.to(dtype).to(DEV), ids, lp, T, beta, tail, what="confident")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("beta,tail", WAYS)
def test_biases_of_a_hundred(dtype, beta, tail):
    """+100 and -100, the biases that choose and ban a token: on a listed column, on an unlisted one,
    on all listed, on all others, at two temperatures."""
    V = 2051
    x = (randn(1, 8, V, seed=7) * 2)
    ids, lp = teacher(x, 9, 8, unused=False)
    at = lambda r, k: int(ids[r, k])  # noqa: E731
    x[0, 0, at(0, 0)] += 100.0
    x[0, 1, at(1, 0)] -= 100.0
    x[0, 2, ids[2]] -= 100.0
    x[0, 3, ids[3]] += 100.0
    x[0, 4] -= 100.0
    x[0, 4, ids[4]] += 100.0
    x[0, 5, at(5, 2)] -= 100.0
    x[0, 5, at(5, 3)] += 100.0
    unlisted = next(j for j in range(V) if j not in set(ids[6].tolist()))
    x[0, 6, unlisted] += 100.0
    x[0, 7, ids[7, :4]] += 100.0
    x[0, 7, ids[7, 4:]] -= 500.0
    for T in (1.0, 0.5):
        check(x.to(dtype).to(DEV), ids, lp, T, beta, tail, what=f"T={T}")


@pytest.mark.parametrize("beta,tail", WAYS)
@pytest.mark.parametrize("gap", [88.0, 104.0, 110.0, 150.0, 500.0])
def test_listed_columns_far_below(beta, tail, gap):
    """A teacher's token that the student has put far down: its part of the loss is q (log q + gap)."""
    x = randn(1, 3, 600, seed=3)
    ids, lp = teacher(x, 6, 2, unused=False)
    for r in range(3):
        x[0, r, int(ids[r, 2 * r])] -= gap
    check(x.to(DEV), ids, lp, 1.0, beta, tail, what=f"gap {gap}")


@pytest.mark.parametrize("beta,tail", WAYS)
@pytest.mark.parametrize("layout,out_layout", [("odd", "dense"), ("cut", "phase")])
def test_layouts_and_weights(beta, tail, layout, out_layout):
    """Rows out of phase, with columns listed in the row's ends, and large and small weights."""
    V = 4099
    x = randn(2, 3, V, seed=6)
    ids = torch.tensor([[0, 1, V - 1, V - 2, 700, 2050]]).repeat(6, 1)
    x[..., ids[0]] += torch.tensor([90.0, 97.0, 105.0, 130.0, 60.0, 300.0]).reshape(2, 3, 1)
    lp = torch.log_softmax(randn(6, 7, seed=2), 1)[:, :6].contiguous()
    for dtype in (torch.bfloat16, torch.float32):
        v, _ = place(x.to(dtype), layout)
        check(v, ids, lp, 1.0, beta, tail, dloss=torch.tensor([1e20, -1e10, 1.0, -1e-10, 1e5, 1e-20]),
              out_layout=out_layout, what="weights")


@pytest.mark.parametrize("dtype,V", [(torch.float32, 100003), (torch.bfloat16, 151936)])
@pytest.mark.parametrize("R", [1, 40, 700])
def test_row_counts_and_in_place(R, V, dtype):
    """Every split of rows over CTAs, a long list, gradients over the logits."""
    K = 256
    g = torch.Generator(device=DEV).manual_seed(R)
    x = torch.randn(1, R, V, generator=g, device=DEV)
    ids = torch.rand(R, V, generator=g, device=DEV).topk(K, dim=1).indices
    x.scatter_add_(2, ids[None], (80.0 + 40.0 * torch.rand(1, R, 1, generator=g, device=DEV)).expand(1, R, K))
    x = x.to(dtype)
    lp = torch.log_softmax(torch.randn(R, K, generator=g, device=DEV), 1) - 0.05
    w = torch.randn(R, generator=g, device=DEV)
    rows = torch.tensor(sorted({0, R // 3, R - 1}))
    at = rows.to(DEV)
    for beta in (0.0, 0.5):
        how = dict(T=0.9, beta=beta, tail=True)
        f = rp.distill_topk_fwd(x, ids, lp, **how)
        dl = rp.distill_topk_bwd(x, ids, lp, w, f["lse"], f["p_rest"], **how)
        u = rp.distill_topk_fused(x, ids, lp, w, **how)
        xs, T = f64(x[0, at]), float(np.float32(0.9))
        ws = w[at].double().cpu().numpy()
        o = lo.distill_topk(xs, ids[at].cpu().numpy(), lp[at].cpu().numpy(), T, beta, True, None, ws)
        tol = tolerances(o, xs, ids[at].cpu().numpy(), ws, T, HALF[dtype])
        for out, grad in ((f, dl), (u, u["dlogits"])):
            close(out["loss"][at], o["loss"], tol["loss"], "loss")
            close(grad[0, at], o["dlogits"], tol["dlogits"], "dlogits")
        y = x.clone()
        same_bits(rp.distill_topk_bwd(y, ids, lp, w, f["lse"], f["p_rest"], **how, dlogits=y)[0, :40], dl[0, :40],
                  "in place")


@pytest.mark.parametrize("beta", [0.0, 0.5, 1.0])
def test_masks_of_the_lowest_value_outside_the_list(beta):
    """Unlisted columns at the type's lowest value are a rest of hardly any mass: the loss is finite
    or, where its terms leave fp32, infinite; the gradient is finite, and the mixture's is that of
    the definition."""
    V = 1003
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.full((1, 2, V), torch.finfo(dtype).min)
        ids = torch.tensor([[5, 900, 17], [0, V - 1, 3]])
        for r in range(2):
            x[0, r, ids[r]] = torch.tensor([1.0, 0.5, -2.0])
        lp = torch.tensor([[0.6, 0.2, 0.1]]).log().repeat(2, 1)
        x = x.to(dtype).to(DEV)
        how = dict(T=0.5, beta=beta, tail=True)
        w = torch.ones(2, device=DEV)
        f = rp.distill_topk_fwd(x, ids.to(DEV), lp.to(DEV), **how)
        dl = rp.distill_topk_bwd(x, ids.to(DEV), lp.to(DEV), w, f["lse"], f["p_rest"], **how)
        u = rp.distill_topk_fused(x, ids.to(DEV), lp.to(DEV), w, **how)
        assert not bool(f["loss"].isnan().any()) and bool(dl.isfinite().all()) and bool(u["dlogits"].isfinite().all())
        if beta == 0.0:      # -q_rest, spread evenly over the unlisted columns
            rest = torch.ones(2, V, dtype=torch.bool).scatter_(1, ids, False).to(DEV)
            for grad in (dl, u["dlogits"]):
                got = grad[0][rest].double()
                want = -(1 - 0.9) / 0.5 / (V - 3)
                assert bool(((got / want - 1).abs() <= 1e-4 + HALF[dtype]).all())
