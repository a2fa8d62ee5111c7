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
