"""A list length that topk_log_softmax cannot take is refused by the library before anything of its
size is allocated."""
import pytest
import torch

from logits_ops_util import DEV, randn
from rl_fine_tuning_pass_gb300 import binding as rp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


@pytest.mark.parametrize("K", [257, 1 << 36, 1 << 62, (1 << 64) + 4, 0, -1, -(1 << 64) + 4])
def test_list_lengths_refused(K):
    x = randn(64, 500, seed=1).to(DEV)
    before = torch.cuda.max_memory_allocated()
    with pytest.raises(rp.GrpoError):
        rp.topk_log_softmax(x, K)
    assert torch.cuda.max_memory_allocated() <= before + 64 * 256 * 16
