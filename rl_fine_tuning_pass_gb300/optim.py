"""AdamW over many tensors at once: the update that takes a loss's gradients to the parameters.

``AdamW`` holds what a program keeps between steps (the states, in 32 or 8 bits, fp32 master copies
and the step count, all on the GPU) and marshals; the update is the C entry point ``adamw_step``.
"""

from __future__ import annotations

import ctypes
import struct
from array import array

import torch

from . import binding as rp

BLOCK = 256   # elements that share a scale of the 8-bit states; each tensor's slot is whole blocks

_WORDS = ctypes.sizeof(rp.GrpoAdamwTensor) // 8
_ARGS = struct.Struct("=ddddQQfiiiQ")
assert _ARGS.size == ctypes.sizeof(rp.GrpoAdamwArgs) and _WORDS == 9


class AdamW:
    """AdamW with decoupled weight decay for CUDA tensors (contiguous, fp32 or bf16, on one device).

    params        tensors to update, in place
    lr            a float, or a one-element fp32 CUDA tensor (read by the update, so that a captured
                  step follows it); may be set between steps
    weight_decay  one value, or one for each tensor
    state_bits    32, or 8: moments in 8-bit codes, 256 of a tensor's elements to a pair of scales
    master        keep an fp32 copy of bf16 parameters, which are then its rounding (one that becomes bf16
                  later has it from its next step on)
    stochastic    round what is kept in few bits (the second moment's codes, bf16 parameters without
                  a master copy) up or down by random bits, so that changes below its precision
                  are kept on average.  Default: with 8-bit states
    seed          of those random bits, which depend on it, the step and the element alone

    ``exp_avg``, ``exp_avg_sq`` (fp32, or uint8 codes), ``scale`` and ``master`` are flat buffers in
    which each tensor's slot is whole blocks of 256; ``views`` gives a tensor's part of such a buffer.
    They are written in place and stay where they are.
    """

    def __init__(self, params, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32,
                 master=False, stochastic=None, seed=0):
        self.params = list(params)
        if not self.params:
            raise ValueError("AdamW needs a tensor")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        self.lr, self.betas, self.eps = lr, tuple(betas), eps
        if len(self.betas) != 2 or not all(0.0 <= b < 1.0 for b in self.betas) or not 1e-30 <= eps < float("inf"):
            raise ValueError("betas must be two numbers in [0, 1), eps at least 1e-30")
        self.state_bits, self.seed = state_bits, int(seed)
        if not 0 <= self.seed < 2 ** 64:
            raise ValueError("seed must be in [0, 2^64)")
        self.stochastic = state_bits == 8 if stochastic is None else bool(stochastic)
        decay = [float(w) for w in weight_decay] if isinstance(weight_decay, (list, tuple)) else \
            [float(weight_decay)] * len(self.params)
        if len(decay) != len(self.params):
            raise ValueError(f"weight_decay needs a value for each of the {len(self.params)} tensors")
        self.weight_decay = decay
        self.device = dev = self.params[0].device
        self._check_params()
        self.numels = [p.numel() for p in self.params]
        first, at = [], 0
        for n in self.numels:
            first.append(at)
            at += -(-n // BLOCK)
        self._first, total = first, at * BLOCK
        kind = dict(dtype=torch.uint8 if state_bits == 8 else torch.float32, device=dev)
        self.exp_avg, self.exp_avg_sq = torch.zeros(total, **kind), torch.zeros(total, **kind)
        self.scale = torch.zeros(at, 2, dtype=torch.float32, device=dev) if state_bits == 8 else None
        self.master, self._masters = None, bool(master)
        if master and any(p.dtype == torch.bfloat16 for p in self.params):
            self.master = torch.zeros(total, dtype=torch.float32, device=dev)
            self.reset_master()
        self._state = torch.zeros(4, dtype=torch.int64, device=dev)   # grpo_adamw_state
        self._build()

    # -- what is kept --------------------------------------------------------------------
    def _check_params(self):
        spans = []
        for p in self.params:
            if not p.is_cuda or p.device != self.device:
                raise ValueError(f"parameters must be CUDA tensors on one device, got {p.device}")
            if p.dtype not in rp._DTYPES:
                raise TypeError(f"parameter dtype {p.dtype} not supported (bf16 or fp32)")
            if not p.is_contiguous():
                raise ValueError("parameters must be contiguous")
            if p.numel():
                spans.append((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size()))
        spans.sort()
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("parameters must not share memory (one is listed twice?)")

    def _build(self):
        """The packed grpo_adamw_tensor array, without the gradients."""
        self._pointers = list(map(rp._ptrs_of, self.params))
        self._versioned = [p for p in self.params if not p.is_inference()]   # autograd is told of the change
        table = array("Q", bytes(8 * _WORDS * len(self.params)))
        step = 1 if self.state_bits == 8 else 4
        for i, (p, n, f, w) in enumerate(zip(self.params, self.numels, self._first, self.weight_decay)):
            has_master = self.master is not None and p.dtype == torch.bfloat16
            at = f * BLOCK
            word = struct.unpack("=Q", struct.pack("=fi", w, 0))[0]
            table[_WORDS * i:_WORDS * (i + 1)] = array("Q", [
                p.data_ptr(), 0, self.master.data_ptr() + 4 * at if has_master else 0,
                self.exp_avg.data_ptr() + step * at, self.exp_avg_sq.data_ptr() + step * at,
                self.scale.data_ptr() + 8 * f if self.scale is not None else 0, n, rp._DTYPES[p.dtype], word])
        self._table, self._counts = table, table[6::_WORDS]
        self._param_words = table[7::_WORDS]
        self._shapes, self._dtypes = [p.shape for p in self.params], list(map(rp._dtype_of, self.params))
        self._grad_dtypes = None                                  # of the last call, and their words

    def __setstate__(self, attributes):
        """Of a copy, or of one that was saved: the table's addresses are the original's."""
        self.__dict__.update(attributes)
        self.device = self.params[0].device
        self._check_params()
        self._build()

    def views(self, flat):
        """Each tensor's part of a flat buffer, in its shape."""
        return [flat[f * BLOCK:f * BLOCK + n].view(p.shape) for p, n, f in zip(self.params, self.numels, self._first)]

    def reset_master(self):
        """Take the master copies, if there are any, from the parameters (after these were loaded)."""
        if self.master is None:
            return
        for p, v in zip(self.params, self.views(self.master)):
            v.copy_(p.detach())

    def _follow_types(self):
        """A parameter that has become bf16 since the table was built takes its master copy from itself: what
        its slot holds is of the start, or of the last time that it was bf16."""
        became = [i for i, (p, was) in enumerate(zip(self.params, self._dtypes))
                  if p.dtype == torch.bfloat16 and was != torch.bfloat16]
        if not became or not self._masters:
            return
        if torch.cuda.is_current_stream_capturing():   # the copy would be repeated by each replay
            raise RuntimeError("a parameter has become bf16: make a step before the capture")
        if self.master is None:
            self.master = torch.zeros(self.exp_avg.numel(), dtype=torch.float32, device=self.device)
        views = self.views(self.master)
        for i in became:
            views[i].copy_(self.params[i].detach())

    def moments(self):
        """(exp_avg, exp_avg_sq) as fp32 in the flat layout: the states themselves with 32 bits, what
        the codes stand for with 8."""
        if self.state_bits == 32:
            return self.exp_avg, self.exp_avg_sq
        m = torch.empty(self.exp_avg.numel(), dtype=torch.float32, device=self.device)
        v = torch.empty_like(m)
        rp._call("adamw_moments", self.device, self.exp_avg.data_ptr(), self.exp_avg_sq.data_ptr(),
                 self.scale.data_ptr(), m.numel(), m.data_ptr(), v.data_ptr())
        return m, v

    def state_dict(self):
        """Copies of the states, and the step count (waits for the GPU)."""
        copy = lambda t: None if t is None else t.clone()  # noqa: E731
        return dict(step=int(self._state[0]), exp_avg=copy(self.exp_avg), exp_avg_sq=copy(self.exp_avg_sq),
                    scale=copy(self.scale), master=copy(self.master))

    def load_state_dict(self, state):
        """Take over states of the same tensors, bits and master copies (the parameters themselves
        are the caller's)."""
        mine = dict(exp_avg=self.exp_avg, exp_avg_sq=self.exp_avg_sq, scale=self.scale, master=self.master)
        for name, t in mine.items():
            other = state[name]
            if (t is None) != (other is None) or (t is not None and (t.shape != other.shape or t.dtype != other.dtype)):
                raise ValueError(f"{name} is of another layout")
        step = int(state["step"])
        if step < 0:
            raise ValueError("step must not be negative")
        for name, t in mine.items():
            if t is not None:
                t.copy_(state[name])
        words = struct.unpack("=qqqq", struct.pack("=qddq", step, *(float(b) ** step for b in self.betas), 0))
        self._state.copy_(torch.tensor(words, dtype=torch.int64))

    # -- one step ------------------------------------------------------------------------
    def step(self, grads=None, *, norm=None, max_norm=None):
        """One update from ``grads`` (default: the parameters' ``grad``; bf16 or fp32, contiguous, of
        the parameters' shapes; None leaves a tensor and its state as they are).

        ``max_norm``: gradients are scaled down to that norm where theirs is larger, and a norm that
        is not finite leaves everything as it is, the step count too.  ``norm``: theirs, if it is
        known (one fp32 element on the GPU, of other ranks' gradients too); else it is computed.
        Returns the norm (None without ``max_norm`` and ``norm``)."""
        params, dev = self.params, self.device
        grads = [p.grad for p in params] if grads is None else list(grads)
        if len(grads) != len(params):
            raise ValueError(f"{len(params)} gradients are needed, got {len(grads)}")
        # a parameter's memory was exchanged, or is seen in another type, size or order (in any of them alone:
        # another type over the same bytes is another size)
        if list(map(rp._ptrs_of, params)) != self._pointers or list(map(rp._dtype_of, params)) != self._dtypes or \
                list(map(rp._numels_of, params)) != self.numels or not all(map(rp._contiguous, params)):
            self._check_params()
            if list(map(rp._numels_of, params)) != self.numels:
                raise ValueError("a parameter has another size than at the start")
            self._follow_types()
            self._build()
        table, counts, shapes = self._table[:], self._counts, self._shapes
        missing, given = (), grads
        if rp._NONE in set(map(type, grads)):
            missing = [i for i, g in enumerate(grads) if g is None]
            given = [g for g in grads if g is not None]
            shapes = [v for v, g in zip(shapes, grads) if g is not None]
            counts = counts[:]
            for i in missing:
                counts[i] = 0
            table[6::_WORDS] = counts
        dtypes = rp.grad_dtypes(given, dev)
        if [g.shape for g in given] != shapes and \
                [g.shape for g in given] != [p.shape for p, g in zip(params, grads) if g is not None]:
            raise ValueError("gradients must have the parameters' shapes")
        pointers = array("Q", map(rp._ptrs_of, given))
        for i in missing:
            pointers.insert(i, 0)
            dtypes.insert(i, torch.float32)
        if dtypes != self._grad_dtypes:
            self._grad_words = rp.dtype_words(dtypes)
            self._words7 = array("Q", [w | d << 32 for w, d in zip(self._param_words, self._grad_words)])
            self._grad_dtypes = dtypes
        if norm is None and max_norm is not None:
            norm = rp.norm_of_table(pointers, counts, self._grad_words, dev)
        table[1::_WORDS], table[7::_WORDS] = pointers, self._words7
        lr, lr_dev = self.lr, 0
        if isinstance(lr, torch.Tensor):
            lr, lr_dev = 0.0, rp._on(lr, torch.float32, 1, "lr", dev)
        limit = float("inf") if max_norm is None else float(max_norm)
        args = _ARGS.pack(lr, *self.betas, self.eps, lr_dev, rp._on(norm, torch.float32, 1, "norm", dev), limit,
                          self.state_bits, self.stochastic, 0, self.seed)
        rp._call("adamw_step", dev, table.buffer_info()[0], len(params), args, self._state.data_ptr())
        if self._versioned:
            torch.autograd.graph.increment_version(self._versioned)
        return norm
