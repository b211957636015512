"""AdamW's table follows what a parameter is now, on the CPU: the C call is replaced by one that notes the table
it would have been given, and the checks that ask for CUDA tensors are left out."""
import copy
import ctypes
import pickle
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
        seen.append([SimpleNamespace(param=t.param, n=t.n, types=(t.param_dtype, t.grad_dtype), master=t.master,
                                     states=(t.exp_avg, t.exp_avg_sq, t.scale))
                     for t in rows])
    monkeypatch.setattr(rp, "_call", note)
    monkeypatch.setattr(rp, "grad_dtypes", lambda grads, dev: [g.dtype for g in grads])
    monkeypatch.setattr(AdamW, "_check_params", lambda self: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
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


def test_a_parameter_that_becomes_bf16_takes_its_master_copy_anew(calls):
    """Not what its slot was filled with at the start, or left with when it was bf16 before."""
    memory = torch.full((32,), 3.0)
    p, q = torch.nn.Parameter(memory), torch.nn.Parameter(torch.ones(32, dtype=BF16))
    opt = AdamW([p, q], master=True)
    g = [torch.zeros(32), torch.zeros(32)]
    opt.step(g)
    assert calls[-1][0].master is None and calls[-1][1].master == opt.views(opt.master)[1].data_ptr()
    for value in (5.0, 7.0):
        opt.views(opt.master)[1].fill_(value + 0.001)           # the other's copy is the update's
        p.data = memory.view(BF16)[:32].fill_(value)
        opt.step(g)
        assert calls[-1][0].master == opt.views(opt.master)[0].data_ptr()
        assert bool((opt.views(opt.master)[0] == value).all())
        assert bool((opt.views(opt.master)[1] == value + 0.001).all())
        p.data = memory
        opt.step(g)
        assert calls[-1][0].master is None


def test_the_first_parameter_that_becomes_bf16_gets_a_master_copy(calls):
    memory = torch.zeros(300)
    p = torch.nn.Parameter(memory)
    opt = AdamW([p], master=True)
    assert opt.master is None
    p.data = memory.view(BF16)[:300].fill_(2.0)
    opt.step([torch.zeros(300)])
    assert calls[-1][0].master == opt.master.data_ptr() and bool((opt.views(opt.master)[0] == 2).all())
    other = AdamW([p])                                          # without
    other.step([torch.zeros(300)])
    assert other.master is None and calls[-1][0].master is None


def test_another_type_is_refused_while_a_graph_is_captured(calls, monkeypatch):
    memory = torch.zeros(32)
    p = torch.nn.Parameter(memory)
    opt = AdamW([p], master=True)
    p.data = memory.view(BF16)[:32]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="before the capture"):
        opt.step([torch.zeros(32)])
    assert not calls


@pytest.mark.parametrize("way", [copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o))])
def test_a_copy_has_states_of_its_own(calls, way):
    """Also where a parameter lies at the address that the original's had, as in a program that loads a saved one."""
    p = torch.nn.Parameter(torch.zeros(300))
    opt = AdamW([p], state_bits=8)
    other = way(opt)
    other.params[0].data = p.data
    other.step([torch.zeros(300)])
    assert calls[-1][0].param == p.data_ptr()
    assert calls[-1][0].states == tuple(t.data_ptr() for t in (other.exp_avg, other.exp_avg_sq, other.scale))
    assert other.exp_avg.data_ptr() != opt.exp_avg.data_ptr()


def test_without_master_copies_there_is_none_to_reset(calls):
    p = torch.nn.Parameter(torch.ones(30, dtype=BF16))
    AdamW([p]).reset_master()
    opt = AdamW([p, torch.nn.Parameter(torch.ones(30))], master=True)
    p.data.fill_(4.0)
    opt.reset_master()
    assert bool((opt.views(opt.master)[0] == 4).all())
