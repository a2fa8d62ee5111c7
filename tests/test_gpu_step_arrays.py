"""Step maps whose arrays lie beside one another in one buffer, without a gap, and
whose inputs share memory: nothing is refused, and nothing else is written."""
import numpy as np
import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B
from test_gpu_steps import Step

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("n,T", [(4, 16), (301, 1200)])
def test_arrays_without_a_gap(n, T, cuda_lib):
    rng = np.random.default_rng(n)
    fresh = rng.integers(0, 4, n)
    s = Step(rng.integers(0, 60, n), fresh, 16, 8, rng.permutation(5 * n), 3, T=T)
    names = [k for k, v in s.d.items() if isinstance(v, torch.Tensor) and k != "slot"]
    whole = torch.full((sum(s.d[k].numel() for k in names) + 2 * T + 9,), -99, dtype=torch.int32, device=DEV)
    s.d["slot"] = whole[4:4 + 2 * T].view(torch.int64)
    at = 4 + 2 * T
    for k in names:
        old = s.d[k]
        s.d[k] = whole[at:at + old.numel()].view(old.shape)
        s.d[k].copy_(old)
        at += old.numel()
    s.run()
    s.check()
    assert bool((whole[:4] == -99).all()) and bool((whole[at:] == -99).all())


def test_inputs_may_share_memory(cuda_lib):
    """As many tokens cached as are added, and a list that holds its head."""
    s = Step([2, 5, 1], [2, 5, 1], 4, 4, [1, 9, 8, 7], 1)
    s.d["fresh"], s.d["free_head"] = s.d["cached"], s.d["free_pages"][:1]
    s.run()
    s.check()
    assert B.device_error() == 0
