"""Lengths and token counts that the latent attention has to clamp: what it says, which
tokens it attends, and that it leaves everything else as it was, in front of its arrays
and behind them as well."""
import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B
from test_gpu_latent import DATA_ERROR, Case, ok

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SPARE = 3  # tokens in front of out and lse and behind them


def framed(c):
    """c's out and lse become the middle of larger ones; all of it is 7."""
    out = torch.full((c.T + 2 * SPARE, c.H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((c.T + 2 * SPARE, c.H), 7.0, device=DEV)
    c.out, c.lse = out[SPARE:SPARE + c.T], lse[SPARE:SPARE + c.T]
    return out, lse


def run(c, kv_len, cu):
    out, lse = framed(c)
    c.kv_len.copy_(torch.tensor(kv_len, dtype=torch.int32))
    c.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    c.run()
    torch.cuda.synchronize()
    error = B.device_error()
    left = ((out == 7.0).all(2).all(1) & (lse == 7.0).all(1)).tolist()
    return error, [t - SPARE for t, same in enumerate(left) if not same]


# kv_len, cu, and (token, sequence, rows that it sees) of the tokens attended: two sequences of 300
# and 128 rows, five rows of q
@pytest.mark.parametrize("kv_len,cu,seen", [
    ([300, -3], [0, 1, 3], [(0, 0, 300), (1, 1, 0), (2, 1, 0)]),
    ([300, 10 ** 6], [0, 1, 1], [(0, 0, 300)]),                   # (the sequence whose length is clamped has no token)
    ([300, 128], [0, 1, 99], [(0, 0, 300)] + [(1 + i, 1, 125 + i) for i in range(4)]),
    ([300, 128], [0, 99, 99], [(i, 0, 296 + i) for i in range(5)]),
    ([300, 128], [-4, 1, 3], [(0, 0, 300), (1, 1, 127), (2, 1, 128)]),
    ([300, 128], [2, 3, 4], [(2, 0, 300), (3, 1, 128)]),
    ([300, 128], [0, 1, -1], [(0, 0, 300)]),
    ([300, 128], [-1, -1, -1], []),
    ([300, 128], [7, 8, 9], []),
    ([300, 128], [5, 3, 1], []),
    ([-1, -2 ** 31], [0, 1, 2], [(0, 0, 0), (1, 1, 0)]),
])
def test_what_is_clamped_and_what_is_left(kv_len, cu, seen, cuda_lib):
    c = Case([1, 2], [300, 128], 128, 64, pad=2, seed=8)
    error, written = run(c, kv_len, cu)
    assert error == DATA_ERROR
    assert written == [t for t, _, _ in seen]
    for t, b, rows in seen:
        if t >= 3:  # (padding of the case: its q is NaN, and so is what the call made of it)
            assert bool(c.out[t].isnan().all())
        else:
            c._token(t, c.kv[c.rows_of[b]].double()[:rows], True)
    error, written = run(c, [300, 128], [0, 1, 3])
    assert error == 0 and written == [0, 1, 2]
    c.check()


@pytest.mark.parametrize("n,cu", [
    (6, [0, 5, 0, 5, 0, 5, 0]), (2, [5, 0, 5]), (3, [0, 4, 1, 4]), (1000, [0, 5] * 500 + [0]), (400, [0] * 399 + [5, 4]),
])
def test_counts_whose_sequences_overlap(n, cu, cuda_lib):
    """Sequences of more tokens in all than there are rows (in garbage it may be any
    multiple of them, and the call would last as much longer): none is attended.  Counts
    that decrease without that are attended as they are clamped."""
    c = Case([1] + [0] * (n - 1), [300] + [64] * (n - 1), 16, 64, pad=4, seed=8)
    tokens = [max(0, b - a) for a, b in zip(cu, cu[1:])]
    error, written = run(c, [300] + [64] * (n - 1), cu)
    assert error == DATA_ERROR
    assert written == ([] if sum(tokens) > c.T else list(range(5)))
    error, written = run(c, [300] + [64] * (n - 1), [0] + [1] * n)
    assert error == 0 and written == [0]
    c.check()
