"""AdamW on parameters that are seen as another type of the same memory."""
import pytest
import torch

import rl_fine_tuning_pass_gb300 as rl
from logits_ops_util import DEV, same_bits
from rl_fine_tuning_pass_gb300 import binding as rp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


@pytest.mark.parametrize("was,now,shape", [(BF16, F32, (16,)), (F32, BF16, (8, 8))])
def test_another_type_over_the_same_bytes_changes_nothing(was, now, shape):
    p = torch.nn.Parameter(torch.randn(32, device=DEV).to(was))
    opt = rl.AdamW([p], lr=0.1)
    opt.step([torch.ones(32, device=DEV)])
    p.data = p.data.view(now).view(shape)
    kept, state = p.data.clone(), opt.state_dict()
    with pytest.raises(ValueError, match="another size"):
        opt.step([torch.ones(shape, device=DEV)])
    same_bits(p.data, kept, "parameter")
    now = opt.state_dict()
    assert now["step"] == state["step"] == 1
    same_bits(now["exp_avg"], state["exp_avg"], "state")


def test_a_parameter_that_becomes_bf16_keeps_its_values():
    """With master copies, beside another bf16 parameter: the first step moves it from where it is."""
    p, q = (torch.nn.Parameter(torch.full((40,), 3.0, device=DEV).to(t)) for t in (F32, BF16))
    g = [torch.ones(40, device=DEV)] * 2
    opt = rl.AdamW([p, q], lr=0.25, weight_decay=0.0, master=True)
    for _ in range(4):
        opt.step(g)                                    # gradients of one sign and size move by lr a step
    assert bool(((p.data - 2.0).abs() < 1e-5).all())
    p.data = p.data.bfloat16()
    opt.step(g)
    # lr times m / sqrt(v), both within a few roundings of 1; 1.75 and 1 bf16 steps of 2^-7
    for t, x in ((p, 1.75), (q, 1.75)):
        assert bool(((t.data.float() - x).abs() <= 2.0 ** -7).all())
    assert bool(((opt.views(opt.master)[0] - 1.75).abs() < 1e-2).all())
    same_bits(p.data, opt.views(opt.master)[0].bfloat16(), "its master copy's rounding")
