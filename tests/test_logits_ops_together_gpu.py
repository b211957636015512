"""The operators in the order a training step uses them: a teacher's top log-probs, the policy's
logits under the sampler's rules, the GRPO loss and the distillation loss on the processed
logits, and the gradient of their sum back through the rules; against the fp64 oracles."""
import numpy as np
import pytest
import torch

import oracle
import rl_fine_tuning_pass_gb300 as rl
from logits_ops_util import DEV, HALF, f64, randn
from oracle import logits_ops_oracle as lo
from rl_fine_tuning_pass_gb300 import binding as rp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_training_step(dtype):
    B, L, V, K, P = 2, 7, 1003, 12, 9
    R = B * L
    T = float(np.float32(0.9))
    g = np.random.default_rng(1)
    x = (randn(B, L, V, seed=1) * 2).to(dtype).to(DEV).requires_grad_(True)
    teacher_logits = (x.detach().float().cpu() + 0.5 * randn(B, L, V, seed=2)).to(dtype).to(DEV)
    k = dict(tokens=g.integers(0, V, (B, P + L)), prompt_len=np.full(B, P, np.int32),
             hist_len=np.tile(P + np.arange(L), B).astype(np.int32), repetition=np.array([1.3, 1.0], np.float32),
             frequency=np.array([0.2, 0.5], np.float32), presence=np.array([0.1, 0.0], np.float32),
             bias_ids=np.array([[3, 5], [8, -1]]), bias=np.array([[1.0, -2.0], [0.5, 0.0]], np.float32))
    d = {n: torch.from_numpy(v).to(DEV) for n, v in k.items()}
    idx = torch.from_numpy(k["tokens"][:, P:].reshape(-1).copy()).to(DEV)
    adv = torch.tensor([0.7, -0.4], device=DEV)

    ids, tlp, _ = rl.topk_log_softmax(teacher_logits, K, T=T)
    y = rl.process_logits(x, **d)
    y.retain_grad()
    loss, aux = rl.grpo_loss(y, idx, adv, T=T)
    div, _ = rl.distill_topk_loss(y, ids, tlp, T=T, beta=0.5, tail=True)
    (loss.sum() / R + 0.3 * div.sum() / R).backward()

    o_ids, o_tlp, _ = lo.topk_log_softmax(f64(teacher_logits), K, T)
    assert np.array_equal(ids.cpu().numpy(), o_ids)
    ys = f64(y)                                      # the processed logits as rounded to the type
    oy, size = lo.process_logits(f64(x), L, **k)
    assert np.all(np.abs(ys - oy) <= 5 * 2.0 ** -24 * size + HALF[dtype] * np.abs(oy))
    w = np.full(R, float(np.float32(1.0 / R)))
    odl, _ = oracle.grpo_loss_bwd(ys, idx.cpu().numpy(), None, None, oracle.per_row(adv.cpu().numpy(), L), None, w, T,
                                  0.0, float(np.float32(0.2)), float(np.float32(0.2)))
    o = lo.distill_topk(ys, o_ids, tlp.cpu().numpy(), T, 0.5, True, None, 0.3 * w)
    assert np.all(np.abs(div.detach().double().cpu().numpy() - o["loss"]) <= 2e-5 * o["G"] + 1e-6)
    dy = odl + o["dlogits"]
    want = lo.process_logits_bwd(f64(x), dy, L, tokens=k["tokens"], hist_len=k["hist_len"], repetition=k["repetition"])
    # each loss's gradient is rounded to the type, then their sum, then the product with the
    # penalty: four half steps of the parts' magnitudes, and 5e-5 of them for the fp32 sums
    part = np.abs(odl) + np.abs(o["dlogits"])
    slope = np.where(dy != 0, np.abs(want) / np.maximum(np.abs(dy), 1e-300), 1.5)
    got = f64(x.grad)
    assert np.all(np.abs(got - want) <= (4 * HALF[dtype] + 5e-5) * part * np.maximum(slope, 1.0) + 1e-9)


def test_a_decode_step():
    """A batch of single rows: rules in place, then the log-probs to return and the sampled
    token's, from the processed logits; a row left with one column has log-prob 0 there."""
    B, V, K = 5, 4001, 10
    x = (randn(B, 1, V, seed=3) * 2).to(torch.bfloat16).to(DEV)
    bits = np.ones((B, (V + 31) // 32 * 32), bool)
    bits[2] = False
    bits[2, 4000] = True
    k = dict(tokens=np.random.default_rng(2).integers(0, V, (B, 50)), frequency=np.full(B, 0.5, np.float32),
             allowed=np.packbits(bits, axis=1, bitorder="little").view(np.int32))
    oy, size = lo.process_logits(f64(x), 1, **k)
    rl.process_logits_fwd(x, **{n: torch.from_numpy(v).to(DEV) for n, v in k.items()}, out=x)
    ids, logp, lse = rl.topk_log_softmax(x, K)
    o_ids, o_logp, _ = lo.topk_log_softmax(f64(x), K, 1.0)
    assert np.array_equal(ids.cpu().numpy(), o_ids)
    assert ids[2, 0] == 4000 and abs(float(logp[2, 0])) < 1e-6 and float(logp[2, 1]) == float("-inf")
    lp, lse2 = rl.selective_log_softmax_fwd(x, ids[:, 0].contiguous(), T=1.0)
    assert bool(((lp - logp[:, 0]).abs() <= 1e-5).all())


def test_gradients_captured_and_replayed():
    B, L, V, K, N = 2, 5, 1003, 12, 9
    x = (randn(B, L, V, seed=1) * 2).to(DEV).requires_grad_(True)
    tokens = torch.from_numpy(np.random.default_rng(2).integers(0, V, (B, N))).to(DEV)
    rep = torch.tensor([1.3, 0.8], device=DEV)
    ids, tlp, _ = rl.topk_log_softmax(x.detach(), K)

    def step():
        y = rl.process_logits(x, tokens=tokens, repetition=rep)
        div, _ = rl.distill_topk_loss(y, ids, tlp, beta=0.5, tail=True)
        return torch.autograd.grad(div.sum(), x)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in range(2):
        with torch.no_grad():
            x.copy_(randn(B, L, V, seed=20 + n))
        graph.replay()
        assert torch.equal(got, step())
