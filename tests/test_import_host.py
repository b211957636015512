"""Importing the package needs neither a GPU nor a CUDA build of torch."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):   # absent from a CPU build
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import rl_fine_tuning_pass_gb300 as rl
from rl_fine_tuning_pass_gb300 import autograd, binding, vocab_parallel, workloads
assert rl.distill_topk_loss is autograd.distill_topk_loss

class Stream:
    cuda_stream = 77
calls = []
torch.cuda.current_stream = lambda device=None: calls.append(device) or Stream
torch.cuda.current_device = lambda: 3
class Lib:
    def topk_log_softmax(self, *args):
        calls.append(args)
        return binding.GRPO_OK
binding._lib = Lib()
binding._call("topk_log_softmax", torch.device("cuda", 3), 1, 2)   # torch's public names stand in
assert calls == [3, (1, 2, 77)], calls
"""


def test_import_without_torchs_cuda_names():
    res = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
