"""Calls on a stream other than the current one, whose memory is still in use by
work queued on the current stream."""
import numpy as np
import pytest
import torch

import oracle as O
from sparse_attention_prolog_gb300 import binding as B
from sparse_attention_prolog_gb300 import workloads as W
from sparse_attention_prolog_gb300.pipeline import DecodeBuffers, DiaBuffers, Kv4Cache, to_dev
from parity_utils import check_codes
from test_gpu_chain import _close_bf16
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


@pytest.fixture(scope="module")
def step(cuda_lib):
    """The DIA step's buffers after a run on the current stream."""
    dia = W.dia_decode(B=2, n_q=2, L=4096)
    st = DiaBuffers(dia, DEV)
    st.run()
    ok()
    return dia, st


def _on_a_side_stream(run, call, kind, args, outputs):
    """The call as run() makes it, then with a workspace of its own, behind work on the current stream: a
    workspace that the current stream cleared would be cleared too late, or be a
    block still in use.  Returns the outputs of both."""
    run()
    ok()
    before = [o.clone() for o in outputs]
    for o in outputs:
        o.zero_()
    s = torch.cuda.Stream()
    need = B.workspace_bytes(kind, args)
    assert need > 0
    address, seen = _freed_block_in_use(need)
    ws = call(args, stream=s)
    ok()
    assert ws.data_ptr() != address and bool((seen == 1).all())
    return zip(before, outputs)


def test_the_mla_prolog_s_own_workspace(step):
    dia, st = step
    _on_a_side_stream(st.mla.run, B.dsa_mla_prolog, "mla", st.mla.args, [st.mla.q, st.mla.q_lora, st.mla.q_lora_scale])
    ref = O.mla_prolog(dia.mla)
    lora, scale = st.mla.q_lora.cpu().numpy(), st.mla.q_lora_scale.cpu().numpy()
    check_codes(lora, scale, ref["q_lora"], ref["q_lora_scale"], "q_lora")
    m = dia.mla
    q = O.mla_q(lora, scale, m.w_uq, m.w_uq_scale, O.bf16_bits_to_f64(m.w_uk), m.H, m.pos, m.rope_cos, m.rope_sin,
                bool(m.rope_interleaved))
    _close_bf16(st.mla.q.float().cpu().numpy(), q, "q")


def test_the_indexer_prolog_s_own_workspace(step):
    """The query codes come from integer sums: the same bits.  The head weights come
    from fp32 sums added with atomics, which the prolog's own tests hold to 1e-4 of
    the largest: two runs to twice that."""
    _, st = step
    q, w = _on_a_side_stream(st.pro.run, B.dsa_indexer_prolog, "prolog", st.pro.args, [st.pro.q_out, st.pro.w_out])
    assert torch.equal(*q)
    assert (w[0] - w[1]).abs().max() <= 2e-4 * max(1.0, float(w[0].abs().max()))


def test_the_top_k_s_own_workspace(step):
    _, st = step
    [(a, b)] = _on_a_side_stream(st.buf.run_topk, B.dsa_indexer_topk, "topk", st.buf.targs, [st.buf.topk_idx])
    assert torch.equal(a.sort(dim=1).values, b.sort(dim=1).values)


def test_the_attention_s_own_workspace(step):
    _, st = step
    for a, b in _on_a_side_stream(st.buf.run_attn, B.dsa_sparse_attn, "attn", st.buf.aargs, [st.buf.out, st.buf.lse]):
        assert torch.equal(a, b)
