"""Step maps whose arrays lie beside one another in one buffer, without a gap, and
whose inputs share memory: nothing is refused, and nothing else is written."""
import numpy as np
import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B
from sparse_attention_prolog_gb300.pipeline import StepMaps
from test_gpu_steps import Step, reference

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


def test_a_request_ends_and_another_takes_its_pages(cuda_lib):
    """Two requests live in pages for two and a half: one ends, its pages go back in
    front of the head, and the next one in its place gets them first."""
    bs, blocks = 8, 10
    free = np.random.default_rng(4).permutation(64)[:16].astype(np.int32)
    m = StepMaps(2, 80, bs, blocks, torch.from_numpy(free).to(DEV))
    lens, head, table = np.zeros(2, dtype=np.int32), 0, np.full((2, blocks), -1, dtype=np.int32)
    for fresh, ends in (((40, 30), None), ((1, 1), None), ((1, 1), 0), ((60, 1), None), ((1, 9), 1), ((1, 40), None)):
        if ends is not None:
            k = -(-int(lens[ends]) // bs)
            m.free_pages[head - k:head] = m.block_table[ends, :k]
            m.counts[m.step][1] -= k
            m.kv_len[ends] = 0
            free[head - k:head] = table[ends, :k]
            head, lens[ends] = head - k, 0
        m.run(torch.tensor(fresh, dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        assert B.device_error() == 0
        cu, kv_len, counts, seq, pos, slot = reference(lens, fresh, free, head, table, bs, 80)
        lens, head = np.asarray(kv_len, dtype=np.int32), counts[1]
        assert m.kv_len.tolist() == kv_len and m.counts[m.step].tolist() == counts and counts[2] == 2
        assert m.slot.tolist() == slot and m.pos.tolist() == pos and m.cu_tokens.tolist() == cu
        assert np.array_equal(m.block_table.cpu().numpy(), table)
        used = [int(p) for b in range(2) for p in table[b, :-(-int(lens[b]) // bs)]]
        assert len(set(used)) == len(used)
