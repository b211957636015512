"""AdamW's table follows what a parameter is now, on the CPU: the C call is replaced by one that notes the table
it would have been given, and the checks that ask for CUDA tensors are left out."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from rl_fine_tuning_pass_gb300 import AdamW
from rl_fine_tuning_pass_gb300 import binding as rp

F32, BF16 = torch.float32, torch.bfloat16
CHECK = AdamW._check_params


@pytest.fixture
def calls(monkeypatch):
    """Tables of the calls made: for each tensor its address, number of elements, parameter's and gradient's type."""
    seen = []

    def note(name, dev, table, count, args, state):
        assert name == "adamw_step"
        rows = (rp.GrpoAdamwTensor * count).from_buffer_copy(
            ctypes.string_at(table, count * ctypes.sizeof(rp.GrpoAdamwTensor)))
        seen.append([SimpleNamespace(param=t.param, n=t.n, types=(t.param_dtype, t.grad_dtype), master=t.master)
                     for t in rows])
    monkeypatch.setattr(rp, "_call", note)
    monkeypatch.setattr(rp, "grad_dtypes", lambda grads, dev: [g.dtype for g in grads])
    monkeypatch.setattr(AdamW, "_check_params", lambda self: None)
    return seen


@pytest.mark.parametrize("was,now,shape", [(BF16, F32, (16,)), (F32, BF16, (64,))])
def test_another_type_over_the_same_bytes_is_another_size(calls, was, now, shape):
    p = torch.nn.Parameter(torch.zeros(32, dtype=was))
    opt = AdamW([p])
    opt.step([torch.zeros(32, dtype=was)])
    assert calls[-1][0].n == 32
    p.data = p.data.view(now)
    assert p.shape == shape and p.data_ptr() == calls[-1][0].param
    with pytest.raises(ValueError, match="another size"):
        opt.step([torch.zeros(shape, dtype=now)])
    assert len(calls) == 1


def test_another_type_of_the_same_width_is_noticed(calls, monkeypatch):
    p = torch.nn.Parameter(torch.zeros(32, dtype=BF16))
    opt = AdamW([p])
    monkeypatch.setattr(AdamW, "_check_params", CHECK)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    opt.step([torch.zeros(32, dtype=BF16)])
    p.data = p.data.view(torch.float16)
    with pytest.raises(TypeError, match="not supported"):
        opt.step([torch.zeros(32)])
    assert len(calls) == 1


def test_as_many_elements_of_another_type_are_followed(calls):
    memory = torch.zeros(32)
    p = torch.nn.Parameter(memory)
    opt = AdamW([p])
    opt.step([torch.zeros(32)])
    p.data = memory.view(BF16)[:32]
    opt.step([torch.zeros(32)])
    first, second = calls[0][0], calls[1][0]
    assert first.param == second.param and first.n == second.n == 32
    assert first.types == (rp.GRPO_FP32, rp.GRPO_FP32) and second.types == (rp.GRPO_BF16, rp.GRPO_FP32)
