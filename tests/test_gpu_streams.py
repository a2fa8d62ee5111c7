"""Calls on a stream other than the current one, whose memory is still in use by
work queued on the current stream."""
import numpy as np
import pytest
import torch

import oracle as O
from sparse_attention_prolog_gb300 import binding as B
from sparse_attention_prolog_gb300.pipeline import DecodeBuffers, Kv4Cache, to_dev
from test_gpu_kv4 import _batch, _check_tokens, _pick, ok

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _freed_block_in_use(nbytes):
    """A block freed on the current stream, whose queued work still reads it some
    50 ms from now: (its address, what that work sees of it)."""
    block = torch.full((nbytes,), 1, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    return block.data_ptr(), block.clone()


def test_the_4_bit_attention_s_own_workspace(cuda_lib):
    inp = _batch(1, 2, [500], 300, 128, 102)
    rows = O.kv4_quantise(inp.kv_cache)
    cache = Kv4Cache(rows.shape[0], DEV)
    cache.data.copy_(to_dev(rows, DEV))
    buf = DecodeBuffers(inp, DEV, kv4=cache)
    idx = _pick(np.random.default_rng(6), inp)
    buf.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
    need = B.workspace_bytes("attn_kv4", buf.aargs)
    assert need > 0
    s = torch.cuda.Stream()
    address, seen = _freed_block_in_use(need)
    ws = B.dsa_sparse_attn_kv4(buf.aargs, stream=s)
    ok()
    assert ws.data_ptr() != address and bool((seen == 1).all())
    out, lse = buf.out.float().cpu().numpy(), buf.lse.cpu().numpy()
    for t in range(inp.T):
        _check_tokens(inp.q_attn[t], O.kv4_values(rows[O.cache_rows(inp, 0, idx[t])]), inp.scale, out[t], lse[t])


def test_a_read_into_memory_of_its_own(cuda_lib):
    """The result is dropped at once, while the read may still be writing it."""
    rng = np.random.default_rng(3)
    n = 4000
    bits = rng.standard_normal((n, 576)).astype(np.float32)
    cache = Kv4Cache(n, DEV)
    cache.write(torch.from_numpy(bits).to(DEV).bfloat16(), torch.arange(n, device=DEV))
    slot = torch.arange(n, device=DEV).flip(0)
    want = cache.read(slot)
    s = torch.cuda.Stream()
    address, seen = _freed_block_in_use(n * 576 * 2)
    got = cache.read(slot, stream=s)
    assert got.data_ptr() != address
    with torch.cuda.stream(s):
        kept = got.clone()
    del got
    other = torch.full((n * 576,), 3.0, dtype=torch.bfloat16, device=DEV)  # the current stream gets no block of the read
    ok()
    assert torch.equal(kept, want) and bool((seen == 1).all()) and bool((other == 3.0).all())
