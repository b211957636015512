"""The preference loss at temperatures other than 1, where log2(e) / T is a number of its own in every pass.

* The fused call is the forward and then the backward: equal bit by bit, whatever T.
* Against the oracle with the tolerances of ``test_preference_gpu.check``, for bf16 logits too.
"""
import numpy as np
import pytest
import torch

import rl_fine_tuning_pass_gb300 as rl
from logits_ops_util import DEV, f64, place, same_bits, untouched
from oracle import train_ops_oracle as to
from rl_fine_tuning_pass_gb300 import binding as rp
from test_preference_gpu import check, make

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


@pytest.mark.parametrize("T", [1.0, 0.75, 0.9, 1.3])
@pytest.mark.parametrize("dtype,layout", [(F32, "dense"), (BF16, "dense"), (F32, "cut"), (BF16, "phase")])
@pytest.mark.parametrize("P,L,V", [(2, 21, 2503), (2, 300, 16600), (40, 7, 7001)])
def test_fused_is_the_forward_and_then_the_backward(T, dtype, layout, P, L, V):
    x, _, idx, how, w, _ = make(P, L, V, dtype, layout, seed=9)
    w = w.to(DEV)
    args = dict(T=T, beta=0.3, label_smoothing=0.1)
    two = rl.preference_loss_fwd(x, idx, **args, **how)
    two["dlogits"] = rl.preference_loss_bwd(x, idx, w, two["coef"], two["lse"], T=T, mask=how["mask"])
    one = rl.preference_loss_fused(x, idx, w, **args, **how)
    assert one.keys() == two.keys()
    for k in two:
        same_bits(one[k], two[k], k)


@pytest.mark.parametrize("T", [0.7, 0.9, 1.3])
@pytest.mark.parametrize("P,L,V,layout,args", [
    (2, 9, 1003, "odd", dict(label_smoothing=0.1, gamma=0.5)),
    (3, 21, 4096, "cut", dict(kind="hinge", beta=0.3)),
    (2, 19, 2051, "phase", dict(kind="squared", beta=0.5)),
    (2, 33, 520, "dense", dict(average=True, beta=2.0, sft_weight=0.3)),
    (2, 3, 32003, "odd", dict()),
])
@pytest.mark.parametrize("fused", [False, True])
def test_bf16_against_the_oracle(T, P, L, V, layout, args, fused):
    args = dict(args, T=T)
    x, buf, idx, how, w, ohow = make(P, L, V, BF16, layout, seed=P + L, average=args.get("average", False))
    f32 = {k: float(np.float32(v)) if isinstance(v, float) and k != "T" else v for k, v in args.items()}
    o = to.preference(f64(x), idx.cpu().numpy(), L, dloss=w.double().numpy(), **f32, **ohow)
    dx, dbuf = place(torch.zeros(2 * P, L, V, dtype=BF16), layout)
    if fused:
        out = rl.preference_loss_fused(x, idx, w.to(DEV), dlogits=dx, **args, **how)
    else:
        out = rl.preference_loss_fwd(x, idx, **args, **how)
        rl.preference_loss_bwd(x, idx, w.to(DEV), out["coef"], out["lse"], T=T, mask=how["mask"], dlogits=dx)
    check(out, o, P, L, BF16, f32, dx)
    untouched(buf, x)
    untouched(dbuf, dx)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [0.7, 0.9, 1.0, 1.3])
@pytest.mark.parametrize("L,V", [(2048, 4096), (700, 32003)])
def test_errors_do_not_add_up_over_a_sequence(dtype, T, L, V):
    """What errs the same way on every token: 1e-8 of the second order of c's correction, 1e-8 of what is left of the
    exponential's mean error, 1e-9 of the logarithm, and of the sums' roundings, which are each below 1e-7
    of the sum and not alike, their mean over some 1000 rows: 3e-8 in all, and 6e-8 is allowed.  A sequence's sum may
    be off by as much a token, and by a half step of what it is rounded to."""
    beta = 0.25
    g = torch.Generator(device=DEV).manual_seed(int(T * 10) + L)
    x = torch.randn(2, L, V, generator=g, device=DEV) * 2
    idx = torch.randint(0, V, (2, L), generator=g, device=DEV)
    known = torch.rand(2, L, 1, generator=g, device=DEV) < 0.5
    x = x.scatter_add_(2, idx[..., None], known * 12.0).to(dtype)
    lse, logp = torch.empty(2, L, dtype=torch.float64, device=DEV), torch.empty(2, L, dtype=torch.float64, device=DEV)
    for b in range(2):
        for l in range(0, L, 256):
            z = x[b, l:l + 256].double() / T
            lse[b, l:l + 256] = torch.logsumexp(z, 1)
            logp[b, l:l + 256] = z.gather(1, idx[b, l:l + 256, None])[:, 0] - lse[b, l:l + 256]
    S = logp.sum(1)
    ref = S.float() + torch.tensor([1.5, -2.0], device=DEV)
    out = rl.preference_loss_fwd(x, idx.reshape(-1), T=T, beta=beta, ref_logp=ref)
    off = out["lse"].double() - lse.reshape(-1)
    # the stored values' own roundings are not alike either: half a step of 2^-20 for 8 to 16, over 2 L rows
    noise = 5 * 2.0 ** -21 / (2 * L) ** 0.5
    assert abs(float(off.mean())) <= 6e-8 + noise
    assert abs(float((out["logp"].double() - logp.reshape(-1)).mean())) <= 6e-8 + noise
    sums = (out["seq_logp"].double() - S).abs()
    assert bool((sums <= L * 6e-8 + 2.0 ** -24 * S.abs()).all()), (sums / L).tolist()
    want = beta * (S - ref.double())
    rewards = (out["reward"].double() - want).abs()
    assert bool((rewards <= beta * L * 6e-8 + 2.0 ** -24 * want.abs()).all()), (rewards / (beta * L)).tolist()


@pytest.mark.parametrize("dtype,tol", [(BF16, 3e-9), (F32, 6e-9)])
def test_the_mean_error_of_a_log_prob(dtype, tol):
    """What is added for the exponential's mean error is a number of two digits, so it is within some 1e-9 of the mean
    over temperatures and spreads; 32768 errors of 4e-8 each leave 2e-10.  The log-probs in both their rows."""
    L, V, off = 2048, 4096, []
    g = torch.Generator(device=DEV).manual_seed(3)
    for T in (0.7, 0.9, 1.0, 1.3):
        for spread in (1.0, 2.0):
            x = (torch.randn(2, L, V, generator=g, device=DEV) * spread).to(dtype)
            idx = torch.randint(0, V, (2 * L,), generator=g, device=DEV)
            logp = rl.preference_loss_fwd(x, idx, T=T)["logp"]
            both = logp.double() + torch.as_strided(logp, (2 * L,), (1,), 2 * L).double()
            z = x.view(-1, V).double() / T
            off.append(both - (z.gather(1, idx[:, None])[:, 0] - torch.logsumexp(z, 1)))
            del x, z
    assert abs(float(torch.cat(off).mean())) <= tol


@pytest.mark.parametrize("T", [1.0, 1.3])
def test_the_mean_error_of_rows_of_one_large_logit(T):
    """Whose exponentials lie next to their row's offset: as far off as others.  6e-9 (between what is added and the
    exponential's mean error), and 4096 errors of 4e-8 leave 6e-10."""
    L, V = 2048, 700
    g = torch.Generator(device=DEV).manual_seed(8)
    x = torch.randn(2, L, V, generator=g, device=DEV) * 2
    idx = torch.randint(0, V, (2, L), generator=g, device=DEV)
    x.scatter_add_(2, idx[..., None], torch.full((2, L, 1), 14.0, device=DEV))
    logp = rl.preference_loss_fwd(x, idx.reshape(-1), T=T)["logp"]
    both = logp.double() + torch.as_strided(logp, (2 * L,), (1,), 2 * L).double()
    z = x.view(-1, V).double() / T
    off = both - (z.gather(1, idx.view(-1, 1))[:, 0] - torch.logsumexp(z, 1))
    assert abs(float(off.mean())) <= 8e-9
