"""The 4-bit attention where a selected row does not exist, and over many tokens
with full selections (the bounds are those of the attention's other tests)."""
import numpy as np
import pytest
import torch

import oracle as O
from sparse_attention_prolog_gb300 import binding as B
from sparse_attention_prolog_gb300.pipeline import DecodeBuffers, Kv4Cache, to_dev
from test_gpu_kv4 import DATA_ERROR, _attend, _batch, _check_tokens, _pick, ok

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("n_q,topk", [(1, 100), (1, 700), (20, 200)])
def test_a_row_that_does_not_exist_reads_as_zeros(n_q, topk, sink, cuda_lib):
    """A selected row of an unmapped page, of a page past the cache, or past the end
    of a cache that stops inside a page: a logit of 0 in the sums, a value of 0.
    Tokens split into chunks (n_q = 1) and whole ones (80 of them)."""
    inp = _batch(4, n_q, [640] * 4, topk, 128, 72, block_size=64, max_L=640)
    rows = O.kv4_quantise(inp.kv_cache)
    rng = np.random.default_rng(73)
    idx = _pick(rng, inp, 0.05)
    n = rows.shape[0] - 20                        # the last page has 44 rows
    table = inp.block_table.copy()
    table[0, 3] = -1
    table[1, [2, 7]] = -1, rows.shape[0] // 64 + 5
    table[2] = -1                                 # nothing of this sequence is mapped
    inp.block_table = table
    cache = Kv4Cache(n, DEV)
    cache.data.copy_(to_dev(rows[:n], DEV))
    buf = DecodeBuffers(inp, DEV, kv4=cache)
    buf.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
    s = rng.normal(0, 2, 128).astype(np.float32) if sink else None
    if sink:
        buf.sink = to_dev(s, DEV)
        buf.aargs.sink = buf.sink.data_ptr()
    buf.out.fill_(float("nan"))
    buf.lse.fill_(float("nan"))
    buf.run_attn()
    torch.cuda.synchronize()
    assert B.device_error() == DATA_ERROR and B.device_error() == 0
    out, lse = buf.out.float().cpu().numpy(), buf.lse.cpu().numpy()
    missing = np.zeros(4, np.int64)
    for t in sorted({*range(0, inp.T, n_q), *range(n_q - 1, inp.T, n_q), *range(n_q // 2, inp.T, n_q)}):
        b = int(inp.seq_of_token[t])
        sel = idx[t][idx[t] >= 0]
        page = table[b, sel // 64].astype(np.int64)
        row = page * 64 + sel % 64
        there = (page >= 0) & (row < n)
        vals = np.zeros((len(sel), 576))
        vals[there] = O.kv4_values(rows[row[there]])
        _check_tokens(inp.q_attn[t], vals, inp.scale, out[t], lse[t], s)
        missing[b] += (~there).sum()
    assert (missing[:3] > 0).all() and not out[inp.seq_of_token == 2].any()


def test_a_cache_that_ends_inside_a_page(cuda_lib):
    """Rows up to its end are read, the one after it is not."""
    inp = _batch(1, 1, [128], 16, 128, 74, block_size=64, max_L=128)
    rows = O.kv4_quantise(inp.kv_cache)
    last = int(np.argmax(inp.block_table[0]))     # the page that holds the cache's last rows
    n = rows.shape[0] - 20
    idx = np.arange(last * 64 + 36, last * 64 + 52)[None]  # rows 36 to 51 of it: 43 is the cache's last
    cache = Kv4Cache(n, DEV)
    cache.data.copy_(to_dev(rows[:n], DEV))
    buf = DecodeBuffers(inp, DEV, kv4=cache)
    buf.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
    buf.run_attn()
    torch.cuda.synchronize()
    assert B.device_error() == DATA_ERROR
    vals = O.kv4_values(rows[O.cache_rows(inp, 0, idx[0])])
    vals[8:] = 0
    _check_tokens(inp.q_attn[0], vals, inp.scale, buf.out[0].float().cpu().numpy(), buf.lse[0].cpu().numpy())


@pytest.mark.parametrize("page", [0, 64])
def test_a_prompt_of_full_selections(page, cuda_lib):
    """128 heads, 2048 of 8192 rows for each of 400 tokens: five or six items of 16
    tiles pass through every cluster's roles."""
    paged = dict(block_size=page, max_L=8192) if page else {}
    inp = _batch(1, 400, [8192], 2048, 128, 75, **paged)
    _attend(inp, _pick(np.random.default_rng(76), inp), tokens=[*range(0, 400, 17), 399])


@pytest.mark.parametrize("fill", [0xff, 0x7f])
@pytest.mark.parametrize("sink", [False, True])
def test_chunks_that_select_nothing_and_whatever_the_workspace_holds(sink, fill, cuda_lib):
    """Short selections of a long index row: most chunks of a token write no partial
    output, and the workspace has NaN (0xff..) or 3.4e38 (0x7f..) in their place."""
    topk, picks = 2000, [0, 1, 63, 64, 65, 700]
    inp = _batch(1, len(picks), [2500], topk, 128, 77)
    idx = _pick(np.random.default_rng(78), inp)
    for t, n in enumerate(picks):
        idx[t, n:] = -1
    idx[5, 64:640] = -1                            # chunks with nothing between two that have rows
    rows = O.kv4_quantise(inp.kv_cache)
    cache = Kv4Cache(rows.shape[0], DEV)
    cache.data.copy_(to_dev(rows, DEV))
    buf = DecodeBuffers(inp, DEV, kv4=cache)
    buf.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
    s = np.random.default_rng(79).normal(0, 2, 128).astype(np.float32) if sink else None
    if sink:
        buf.sink = to_dev(s, DEV)
        buf.aargs.sink = buf.sink.data_ptr()
    assert B.workspace_bytes("attn_kv4", buf.aargs) == buf.aws.numel() > 256
    buf.aws.fill_(fill)
    buf.out.fill_(float("nan"))
    buf.lse.fill_(float("nan"))
    buf.run_attn()
    ok()
    out, lse = buf.out.float().cpu().numpy(), buf.lse.cpu().numpy()
    for t in range(inp.T):
        sel = idx[t][idx[t] >= 0]
        vals = O.kv4_values(rows[O.cache_rows(inp, 0, sel)]) if sel.size else np.zeros((0, 576))
        _check_tokens(inp.q_attn[t], vals, inp.scale, out[t], lse[t], s)


def test_a_captured_call_with_a_workspace_of_its_own(cuda_lib):
    """The workspace is the graph's: replays on new indices, with memory made and
    filled between them, give what an eager call gives."""
    inp = _batch(1, 2, [2000], 700, 128, 80)
    rows = O.kv4_quantise(inp.kv_cache)
    cache = Kv4Cache(rows.shape[0], DEV)
    cache.data.copy_(to_dev(rows, DEV))
    buf = DecodeBuffers(inp, DEV, kv4=cache)
    s = torch.cuda.Stream()
    buf.topk_idx.fill_(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        need = B.dsa_sparse_attn_kv4(buf.aargs, stream=s).numel()
    for seed in (1, 2):
        idx = _pick(np.random.default_rng(seed), inp, 0.05)
        buf.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
        other = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
        buf.out.fill_(float("nan"))
        g.replay()
        ok()
        assert bool((other == 0xff).all())
        out, lse = buf.out.float().cpu().numpy(), buf.lse.cpu().numpy()
        for t in range(inp.T):
            vals = O.kv4_values(rows[O.cache_rows(inp, 0, idx[t][idx[t] >= 0])])
            _check_tokens(inp.q_attn[t], vals, inp.scale, out[t], lse[t])
