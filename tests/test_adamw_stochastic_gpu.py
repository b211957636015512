"""Stochastic rounding of bf16 parameters without a master copy: by the bits that the header promises, and with the
expectation kept.

The parameter before its rounding is known within fp32's roundings (the tolerance of test_adamw_gpu.check_step, some
units of 2^-24 of it).  With `low` its place between two bf16 numbers, in 2^16-ths of their distance, it goes up where
low + bits >= 2^16: certain where that sum is farther from 2^16 than the tolerance.
"""
import numpy as np
import pytest
import torch

import rl_fine_tuning_pass_gb300 as rl
from logits_ops_util import DEV
from oracle import train_ops_oracle as to
from rl_fine_tuning_pass_gb300 import binding as rp
from test_adamw_gpu import BETAS, EPS, F24, make, snapshot, start

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("g_dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 1])
def test_each_parameter_is_rounded_by_its_bits(bits, g_dtype, shift):
    sizes = [1, 257, 2049, 0, 33333, 4096 * 3]
    params, grads = make(sizes, BF16, g_dtype, seed=bits + shift, shift=shift)
    opt = rl.AdamW(params, lr=1e-3, betas=BETAS, eps=EPS, weight_decay=0.1, state_bits=bits, stochastic=True,
                   seed=2 ** 63 + 98765)
    start(opt)
    ups = sure = total = 0
    for _ in range(2):
        before = snapshot(opt)
        opt.step(grads)
        step, wd, lr = opt.state_dict()["step"], float(np.float32(0.1)), 1e-3
        for i, (p, g) in enumerate(zip(opt.params, grads)):
            n = p.numel()
            if n == 0:
                continue
            m0, v0, g64 = before["m"][i], before["v"][i], g.detach().double().cpu().numpy()
            if bits == 8:
                s = before["s"][i]
                m0, v0 = to.decode_m(m0, s[:, 0]), to.decode_r(v0, s[:, 1]).astype(np.float64) ** 2
            want, m, v, size = to.adamw(before["p"][i], g64, m0.astype(np.float64), v0.astype(np.float64), step=step, lr=lr,
                                        betas=BETAS, eps=EPS, weight_decay=wd)
            alpha, den = lr / (1 - BETAS[0] ** step), np.sqrt(v / (1 - BETAS[1] ** step)) + EPS
            change = np.abs(want - before["p"][i])
            tol = F24 * (np.abs(want) + change) + 28 * F24 * alpha * size / den + 4 * F24 * lr * wd * np.abs(before["p"][i])
            apart = 2.0 ** (np.floor(np.log2(np.abs(want))) - 7)           # of bf16 numbers there
            down = np.floor(np.abs(want) / apart)
            low, unsure = (np.abs(want) / apart - down) * 65536, tol / apart * 65536 + 1
            _, r = to.random_bits(opt.seed, step, i, n)
            at = low + r
            known = (np.abs(at - 65536) > unsure) & (low > unsure) & (low < 65536 - unsure)
            expect = np.sign(want) * (down + (at >= 65536)) * apart
            got = p.detach().double().cpu().numpy()
            assert np.array_equal(got[known], expect[known]), f"tensor {i}: {(got[known] != expect[known]).sum()}"
            ups, sure, total = ups + int((at >= 65536)[known].sum()), sure + int(known.sum()), total + n
    assert sure >= 0.98 * total and 0.4 * sure < ups < 0.6 * sure


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("part", [0.02, 0.3, 0.9])
def test_small_updates_are_kept_on_average(bits, part):
    """A first step moves every parameter by lr: `part` of the distance 2^-8 of the bf16 numbers below 1."""
    n, lr = 100_003, part * 2.0 ** -8
    for stochastic in (True, False):
        p = torch.ones(n, dtype=BF16, device=DEV)
        opt = rl.AdamW([p], lr=lr, betas=BETAS, eps=EPS, weight_decay=0.0, state_bits=bits, stochastic=stochastic, seed=5)
        opt.step([torch.ones(n, device=DEV)])
        moved = (1.0 - p.double()) * 256
        if not stochastic:
            assert bool((moved == (1.0 if part > 0.5 else 0.0)).all())
            continue
        assert bool(((moved == 0) | (moved == 1)).all())
        assert abs(float(moved.mean()) - part) <= 5 * (part * (1 - part) / n) ** 0.5 + 1e-5
