"""Waits of the latent attention that run out at every stage of a call: the CTAs leave
once the copies that they began have landed, without waiting for copies that some of
the lanes or warps of a unit never began (each such wait would last seconds), and the
next call is right.

A limit is a time, so where a call stops is not known beforehand: some limits stop it
at its first wait, some in the middle, and some not at all (its result is then right)."""
import time

import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B
from test_gpu_latent import TIMEOUT, Case, ok

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

LIMITS = (1, 300, 700, 1000, 1300, 1700, 2100, 2600, 3200, 4000, 5000)


@pytest.mark.parametrize("n,lens,H,page", [
    ([1], [100], 128, 8),                         # a tile a stretch at most: it ends inside the rings
    ([1, 1], [200, 130], 16, 64),
    ([2], [200], 128, 16), ([3, 2], [256, 250], 128, 0),
    ([1] * 20, [300 + 17 * i for i in range(20)], 128, 8),  # 16 lanes share a unit, blocks follow one another
    ([1, 1, 1], [9000, 70, 4000], 128, 64), ([2, 5, 1], [9000, 700, 4000], 128, 16), ([4] * 30, [700] * 30, 128, 8),
])
def test_a_wait_that_runs_out_anywhere(n, lens, H, page, cuda_lib):
    c = Case(n, lens, H, page)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    ws = torch.empty(B.workspace_bytes("latent_attn", c.args()), dtype=torch.uint8, device=DEV)
    args = c.args()
    c.run(ws)
    ok()
    stopped = 0
    for limit in LIMITS * 3:
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        flush.zero_()  # (the rows come from HBM)
        torch.cuda.synchronize()
        B.set_wait_limit_ns(limit)
        try:
            since = time.monotonic()
            B.dsa_latent_attn(args, ws)
            torch.cuda.synchronize()
            took = time.monotonic() - since
            error = B.device_error()
        finally:
            B.set_wait_limit_ns(0)
        assert error in (0, TIMEOUT), (limit, error)
        assert took < 1.0, (limit, took)
        stopped += error == TIMEOUT
        if error == 0:
            c.check(tokens={0, sum(n) - 1})
    assert stopped >= 3
    ws.zero_()
    c.fresh()
    c.run(ws)
    ok()
    c.check(tokens={0, 1, sum(n) - 1})
