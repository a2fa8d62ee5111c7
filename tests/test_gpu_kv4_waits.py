"""The wait limit of the 4-bit attention is a time: a call whose waits run out ends
within a small multiple of it."""
import numpy as np
import pytest
import torch

import oracle as O
from sparse_attention_prolog_gb300 import binding as B
from sparse_attention_prolog_gb300.pipeline import DecodeBuffers, Kv4Cache, to_dev
from test_gpu_kv4 import TIMEOUT, _batch, _check_tokens, _pick, ok

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _ms(work):
    """Device time of work() in ms."""
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    work()
    end.record()
    end.synchronize()
    return start.elapsed_time(end)


def test_a_wait_that_runs_out_takes_about_the_limit(cuda_lib):
    """The call starts beside a top-k over one row of 2^27 scores (milliseconds on a
    few SMs), so its roles wait for the first row lookups until that has ended.
    Under an eighth of its time some give up; those that meet the ones that left
    give up in turn, a limit later.  A role can follow another that left through
    the two products and the epilogue: five limits, each a wait's shortest to 3.5
    times it, are below 2.2 of the top-k's time.  (Waits counted in tries of one
    length, whoever waits, took a warp 94 times the limit.)"""
    n, k = 1 << 27, 64
    scores = torch.rand(1, n, device=DEV)
    pos = torch.full((1,), n - 1, dtype=torch.int32, device=DEV)
    picked = torch.empty(1, k, dtype=torch.int32, device=DEV)
    none = torch.zeros(16, dtype=torch.int8, device=DEV)  # the indexer's inputs: not read here
    before = B.topk_args(1, 1, 1, 64, 128, k, n, none, none, none, none, none, pos, picked)
    inp = _batch(1, 1, [2048], 700, 128, 110)
    rows = O.kv4_quantise(inp.kv_cache)
    cache = Kv4Cache(rows.shape[0], DEV)
    cache.data.copy_(to_dev(rows, DEV))
    buf = DecodeBuffers(inp, DEV, kv4=cache)
    idx = _pick(np.random.default_rng(5), inp)
    buf.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))

    def both():
        B.dsa_topk_from_scores(before, scores)
        buf.run_attn()

    def check():
        out, lse = buf.out[0].float().cpu().numpy(), buf.lse[0].cpu().numpy()
        _check_tokens(inp.q_attn[0], O.kv4_values(rows[O.cache_rows(inp, 0, idx[0])]), inp.scale, out, lse)

    both()
    alone = min(_ms(lambda: B.dsa_topk_from_scores(before, scores)) for _ in range(3))
    ok()
    assert 0.5 < alone < 200
    B.set_wait_limit_ns(int(alone * 1e6 / 8))
    try:
        took = _ms(both)
        assert B.device_error() == TIMEOUT
    finally:
        B.set_wait_limit_ns(0)
    assert took < 1.1 * alone + 2.2 * alone, f"{took:.2f} ms beside {alone:.2f} ms"
    B.set_wait_limit_ns(int(alone * 1e6 * 8))
    try:
        buf.out.zero_()
        both()
        ok()
    finally:
        B.set_wait_limit_ns(0)
    check()
