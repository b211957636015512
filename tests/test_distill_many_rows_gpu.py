"""The distillation forward on batches of more rows than are resident at once (over twenty rows per
SM), whose launch has 256 streaming threads: some rows against the fp64 oracle, all against calls of
few rows."""
import numpy as np
import pytest
import torch

from logits_ops_util import DEV, HALF, close, f64, place, randn
from oracle import logits_ops_oracle as lo
from rl_fine_tuning_pass_gb300 import binding as rp
from test_distill_topk_gpu import WAYS, tolerances

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


@pytest.mark.parametrize("dtype,layout", [(torch.bfloat16, "dense"), (torch.bfloat16, "odd"), (torch.float32, "cut")])
@pytest.mark.parametrize("beta,tail", WAYS)
def test_many_rows(dtype, layout, beta, tail):
    R, V, K = 21 * torch.cuda.get_device_properties(0).multi_processor_count, 5003, 33
    x, _ = place((randn(2, R // 2, V, seed=1) * 2).to(dtype), layout)
    R = 2 * (R // 2)
    ids, lp, _ = rp.topk_log_softmax((x.float() + 0.5 * randn(2, R // 2, V, seed=2).to(DEV)).contiguous(), K)
    ids[1::3, K // 2] = -1
    mask = (torch.arange(R, device=DEV) % 7 != 3).to(torch.uint8)
    w = randn(R, seed=3).to(DEV)
    T = float(np.float32(0.8))
    how = dict(T=T, beta=beta, tail=tail)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    f = rp.distill_topk_fwd(x, ids, lp, **how, mask=mask, dev_err=err)
    dl = rp.distill_topk_bwd(x, ids, lp, w, f["lse"], f["p_rest"], **how, mask=mask).reshape(R, V)
    u = rp.distill_topk_fused(x, ids, lp, w, **how, mask=mask, dev_err=err)
    assert int(err.item()) == 0
    at = torch.from_numpy(np.unique(np.r_[0:8, R // 2 - 4:R // 2 + 4, R - 8:R, np.arange(0, R, 331)]))
    flat = x.reshape(R, V)
    xs, g, c = f64(flat[at.to(DEV)]), w[at.to(DEV)].double().cpu().numpy(), lambda t: t[at.to(DEV)].cpu().numpy()
    o = lo.distill_topk(xs, c(ids), c(lp), T, float(np.float32(beta)), tail, c(mask), g)
    tol = tolerances(o, xs, c(ids), g, T, HALF[dtype])
    for out, grad in ((f, dl), (u, u["dlogits"].reshape(R, V))):
        for k in ("loss", "lse", "p_rest"):
            close(out[k][at.to(DEV)], o[k], tol[k], k)
        close(grad[at.to(DEV)], o["dlogits"], tol["dlogits"], "dlogits")
    for r0 in range(0, R, 400):       # the launch of few rows
        r = slice(r0, min(R, r0 + 400))
        few = rp.distill_topk_fwd(flat[r].contiguous(), ids[r], lp[r], **how, mask=mask[r])
        for k in ("loss", "lse", "p_rest"):
            assert bool(((few[k] - f[k][r]).abs() <= 1e-4 * (1 + f[k][r].abs())).all()), k
