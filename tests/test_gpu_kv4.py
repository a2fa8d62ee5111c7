"""The 4-bit latent cache on the GPU: written and read rows bit for bit against
the oracle, the sparse attention over the cache against a float64 form with
error bounds worked out from its roundings, and the refusals that need a GPU.

Attention bounds, per output element, with A = sum_j p_j |v_j| (p_j the softmax
weights): the probabilities are rounded to bf16 (at most 2^-8 of each:
2^-8 A) and the result is (2^-8 |out|).  A logit is a sum of
576 exact products held in fp32, off by at most 576 * 2^-23 of the largest
sum of their magnitudes, delta (a step of 2^-23 allows truncation as well as
rounding); an error of delta in a logit changes a weight by delta and the
normalisation by delta again: 2 delta A.  exp2 and the scaled logit add
2^-22 * (1 + the logit's distance from the maximum), below 2^-16 for any weight
that counts.  lse moves by delta, by the fp32 sum of at most topk + 64 terms and
by 2^-22 of itself."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle as O
from sparse_attention_prolog_gb300 import binding as B
from sparse_attention_prolog_gb300 import workloads as W
from sparse_attention_prolog_gb300.pipeline import DecodeBuffers, DiaBuffers, Kv4Cache, to_dev
from test_gpu_chain import _bits, _close_bf16

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DATA_ERROR = 6
TIMEOUT = 5


def ok():
    torch.cuda.synchronize()
    assert B.device_error() == 0


# ------------------------------------------------------------ write and read
def _rows(n, seed):
    """Latent rows that meet every path of the quantiser: normal rows of very
    different sizes, random bit patterns (NaN, infinities, subnormals), zeros,
    ties."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, 576)) * np.exp(rng.uniform(-12, 12, (n, 1)))
    bits = W.f32_to_bf16_bits(x.astype(np.float32))
    for i in range(n):
        if i % 5 == 1:
            bits[i] = rng.integers(0, 65536, 576)
        elif i % 5 == 2:
            bits[i, rng.integers(0, 2, 576) == 0] &= 0x83ff     # many values of very small magnitude
        elif i % 5 == 3:
            half = rng.integers(-14, 15, 576) / 2.0             # ties of scale 1
            half[::16] = 7.0
            bits[i] = W.f32_to_bf16_bits((half * 2.0 ** float(rng.integers(-17, 20))).astype(np.float32))
        elif i % 5 == 4:
            bits[i, :256] = 0
    return bits


@pytest.mark.parametrize("n,pad,skip", [(1, 0, 0), (1, 24, 0), (2, 8, 0), (8, 0, 0), (33, 64, 3), (1000, 8, 5),
                                        (4099, 0, 0)])
def test_write_and_read_bit_for_bit(n, pad, skip, cuda_lib):
    rng = np.random.default_rng(n + pad)
    rows = n + 37
    bits = _rows(n, n)
    slot = rng.permutation(rows)[:n].astype(np.int64)
    if skip:
        slot[::skip] = -1 - np.arange(len(slot[::skip]))  # any negative slot: not written, read as zeros
    before = rng.integers(0, 256, (rows, 416)).astype(np.uint8)
    kv4 = to_dev(before, DEV)
    wide = torch.full((n, 576 + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :576] = to_dev(bits, DEV)
    B.dsa_kv4_write(wide[:, :576], kv4, to_dev(slot, DEV))
    out = torch.full((n, 576 + pad), 3.0, dtype=torch.bfloat16, device=DEV)
    B.dsa_kv4_read(kv4, to_dev(slot, DEV), out[:, :576])
    ok()
    want = before.copy()
    want[slot[slot >= 0]] = O.kv4_quantise(bits)[slot >= 0]
    assert np.array_equal(kv4.cpu().numpy(), want)
    ref = np.zeros((n, 576))
    ref[slot >= 0] = O.kv4_values(want[slot[slot >= 0]])
    got = out[:, :576].float().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    np.testing.assert_array_equal(got[~np.isnan(got)], ref[~np.isnan(ref)])
    assert (out[:, 576:] == 3.0).all()


def test_read_of_every_byte_value(cuda_lib):
    """Every scale byte with every code (-8, which is never written, too)."""
    rows = np.zeros((32, 416), np.uint8)
    rows[:, :256] = np.arange(256)
    rows[:, 256:288] = (np.arange(32)[:, None] * 8 + np.arange(32)[None, :] // 4) % 256
    slot = np.concatenate([np.arange(32), np.arange(32)[::-1]]).astype(np.int64)  # slots may repeat
    got = Kv4Cache(32, DEV)
    got.data.copy_(to_dev(rows, DEV))
    out = got.read(to_dev(slot, DEV))
    ok()
    np.testing.assert_array_equal(out.float().cpu().numpy(), O.kv4_values(rows[slot]).astype(np.float32))


def test_every_scale_with_every_value(cuda_lib):
    """Each of the 255 scales with every bf16 of either sign up to 7 of it (halfway
    points among them), then each finite bf16 as the largest of a group."""
    groups = []
    for u in range(255):
        s = float(O.kv4_scale(u))
        top = int(W.f32_to_bf16_bits(np.array([7.0 * s], np.float32))[0])  # (at most 7 significant bits)
        low = int(W.f32_to_bf16_bits(np.array([s / 8.0], np.float32))[0])
        v = np.arange(low, top, dtype=np.int64)
        v = np.concatenate([v, v | 0x8000])
        v = np.concatenate([v, np.zeros(-len(v) % 15, np.int64)]).reshape(-1, 15)
        groups.append(np.concatenate([np.full((len(v), 1), top), v], axis=1))
    rng = np.random.default_rng(5)
    top = np.arange(0x7f80)[:, None]
    groups.append(np.concatenate([top, np.maximum(top - rng.integers(0, 600, (0x7f80, 15)), 0)], axis=1))
    g = rng.permuted(np.concatenate(groups), axis=1)
    g = np.concatenate([g, np.zeros((-len(g) % 32, 16), np.int64)]).reshape(-1, 512)
    bits = np.concatenate([g, np.zeros((len(g), 64), np.int64)], axis=1).astype(np.uint16)
    cache = Kv4Cache(len(bits), DEV)
    cache.write(to_dev(bits, DEV), torch.arange(len(bits), device=DEV))
    ok()
    assert np.array_equal(cache.data.cpu().numpy(), O.kv4_quantise(bits))


def test_slots_past_the_cache_are_reported(cuda_lib):
    bits = _rows(6, 3)
    cache = Kv4Cache(5, DEV)
    slot = to_dev(np.array([4, 5, 0, 2 ** 40, -1, 2], np.int64), DEV)
    cache.write(to_dev(bits, DEV), slot)
    torch.cuda.synchronize()
    assert B.device_error() == DATA_ERROR and B.device_error() == 0
    want = np.zeros((5, 416), np.uint8)
    want[[4, 0, 2]] = O.kv4_quantise(bits)[[0, 2, 5]]
    assert np.array_equal(cache.data.cpu().numpy(), want)
    out = cache.read(slot)
    torch.cuda.synchronize()
    assert B.device_error() == DATA_ERROR
    assert not out[[1, 3, 4]].any()


def test_wrappers_refuse_what_the_library_would_misread(cuda_lib):
    x = torch.zeros(4, 576, dtype=torch.bfloat16, device=DEV)
    kv4 = torch.zeros(8, 416, dtype=torch.uint8, device=DEV)
    slot = torch.arange(4, device=DEV)
    bad = [
        (x.half(), kv4, slot), (x[:, :512], kv4, slot), (x, kv4[:, :400], slot), (x, kv4[::2], slot),
        (x, kv4, slot.int()), (x[:3], kv4, slot), (x, kv4.cpu(), slot), (x, kv4, slot.repeat(2)[::2]),
        (torch.zeros(576, 4, dtype=torch.bfloat16, device=DEV).t(), kv4, slot),
        (torch.zeros(4, 577, dtype=torch.bfloat16, device=DEV)[:, :576], kv4, slot),   # row stride 577
        (torch.zeros(4, 584, dtype=torch.bfloat16, device=DEV)[:, 4:580], kv4, slot),  # 8-byte aligned rows
        (x[:1].expand(4, 576), kv4, slot),                                             # one row for all
    ]
    for a in bad:
        with pytest.raises(B.DSAError):
            B.dsa_kv4_write(*a)
        with pytest.raises(B.DSAError):
            B.dsa_kv4_read(a[1], a[2], a[0])
    B.dsa_kv4_write(x[:0], kv4, slot[:0])
    B.dsa_kv4_read(kv4, slot[:0], x[:0])
    ok()


# ----------------------------------------------------------------- attention
def _check_tokens(q_bits, values, scale, out, lse, sink=None):
    """out [H, 512], lse [H] of one token against the float64 form over the
    selected rows' values [n, 576], within the bounds of the module docstring."""
    q = O.bf16_bits_to_f64(q_bits)
    ref_o, ref_l = O.sparse_attention_token(q, values, scale, 512, sink)
    n = values.shape[0]
    out, lse = out.astype(np.float64), lse.astype(np.float64)
    if n == 0:
        assert not out.any()
        assert np.array_equal(lse, ref_l) if sink is None else np.allclose(lse, ref_l, rtol=2.0 ** -21, atol=0)
        return
    S = scale * (q @ values.T)
    p = np.exp(S - ref_l[:, None])
    A = p @ np.abs(values[:, :512])
    delta = 576 * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(values).T).max(axis=1, keepdims=True) + 2.0 ** -16
    bound = 2.0 ** -8 * (A + np.abs(ref_o)) * (1 + 2.0 ** -7) + 2 * delta * A + 1e-30
    worst = (np.abs(out - ref_o) / bound).max()
    assert worst <= 1, f"out: {worst:.2f} of the bound"
    finite = np.isfinite(ref_l)
    lb = delta[:, 0] + (n + 64) * 2.0 ** -23 + 2.0 ** -21 * np.abs(ref_l)
    assert np.array_equal(lse[~finite], ref_l[~finite])
    worst = (np.abs(lse - ref_l)[finite] / lb[finite]).max()
    assert worst <= 1, f"lse: {worst:.2f} of the bound"


def _cache_bits(inp, seed):
    """Quantised rows of the batch's own latent rows (uint8 [rows, 416])."""
    return O.kv4_quantise(inp.kv_cache)


def _attend(inp, idx, rows=None, sink=None, seq_map=False, tokens=None, lse=True, stream=None):
    """Runs the attention over the quantised cache and checks the tokens."""
    rows = _cache_bits(inp, 0) if rows is None else rows
    cache = Kv4Cache(rows.shape[0], DEV)
    cache.data.copy_(to_dev(rows, DEV))
    buf = DecodeBuffers(inp, DEV, kv4=cache, seq_map=seq_map)
    buf.topk_idx.copy_(torch.from_numpy(np.asarray(idx).astype(np.int32)))
    if sink is not None:
        buf.sink = to_dev(np.asarray(sink, np.float32), DEV)
        buf.aargs.sink = buf.sink.data_ptr()
    if not lse:
        buf.aargs.lse = None
    buf.out.fill_(float("nan"))
    buf.lse.fill_(float("nan"))
    buf.run_attn(stream)
    ok()
    out, got_lse = buf.out.float().cpu().numpy(), buf.lse.cpu().numpy()
    for t in range(inp.T) if tokens is None else tokens:
        sel = np.asarray(idx[t], np.int64)
        sel = sel[(sel >= 0) & (sel < inp.max_L)]
        vals = O.kv4_values(rows[O.cache_rows(inp, int(inp.seq_of_token[t]), sel)]) if sel.size else np.zeros((0, 576))
        _check_tokens(inp.q_attn[t], vals, inp.scale, out[t], got_lse[t] if lse else _lse(inp, t, vals, sink), sink)
    if not lse:
        assert np.isnan(got_lse).all()
    return buf


def _lse(inp, t, vals, sink):
    return O.sparse_attention_token(O.bf16_bits_to_f64(inp.q_attn[t]), vals, inp.scale, 512, sink)[1]


def _pick(rng, inp, invalid=0.0):
    idx = np.empty((inp.T, inp.topk), np.int64)
    for t in range(inp.T):
        n = int(inp.pos[t]) + 1
        idx[t] = rng.choice(n, size=inp.topk, replace=n < inp.topk)
        if invalid:
            idx[t, rng.random(inp.topk) < invalid] = -1
    return idx


def _batch(B_, n_q, lens, topk, H, seed, **more):
    return W.make_decode_inputs(B=B_, n_q=n_q, seq_lens=lens, H_I=4, d_I=64, topk=topk, H=H, seed=seed, **more)


@pytest.mark.parametrize("topk", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 191, 200, 257, 1000, 2048])
def test_selection_sizes(topk, cuda_lib):
    """Every remainder of the tiles that a selection can end in, one token and
    128 heads (the most chunks a token is split into)."""
    inp = _batch(1, 1, [2500], topk, 128, 100 + topk)
    _attend(inp, _pick(np.random.default_rng(topk), inp))


@pytest.mark.parametrize("topk", [33, 200, 1000])
@pytest.mark.parametrize("T", [4, 40, 200])
def test_token_counts(T, topk, cuda_lib):
    """More tokens, fewer chunks of each: down to one chunk per token."""
    inp = _batch(2, T // 2, [1500, 1300], topk, 32, T + topk)
    _attend(inp, _pick(np.random.default_rng(T), inp, 0.1), tokens=list(range(0, T, max(1, T // 8))))


@pytest.mark.parametrize("H", [1, 3, 16, 64, 100, 128, 129, 160, 256])
def test_head_counts(H, cuda_lib):
    inp = _batch(2, 2, [900, 700], 300, H, 200 + H)
    sink = np.random.default_rng(H).normal(0, 2, H)
    sink[0] = -np.inf
    if H > 1:
        sink[H - 1] = 40.0
    _attend(inp, _pick(np.random.default_rng(H), inp, 0.05), sink=sink)


@pytest.mark.parametrize("topk", [96, 1000])
@pytest.mark.parametrize("sink", [False, True])
def test_masks(topk, sink, cuda_lib):
    """Nothing selected, one row, one row many times, masked heads and tails
    of tiles, indices past max_L."""
    inp = _batch(1, 9, [1200], topk, 128, 31)
    rng = np.random.default_rng(32)
    idx = np.full((9, topk), -1, np.int64)
    idx[1, topk - 1] = 5
    idx[2] = 7
    idx[3] = rng.integers(0, 1190, topk)
    idx[4, ::64] = 11
    idx[5, :40] = rng.integers(0, 1190, 40)
    idx[6, 50:] = rng.integers(0, 1190, topk - 50)
    idx[7] = rng.integers(0, 1190, topk)
    idx[7, rng.random(topk) < 0.5] = -7
    idx[8] = rng.integers(0, 1190, topk)
    idx[8, ::3] = 1200 + rng.integers(0, 2 ** 30, len(idx[8, ::3]))
    inp.max_L = 1200
    _attend(inp, idx, sink=rng.normal(0, 2, 128) if sink else None)


@pytest.mark.parametrize("topk", [100, 600])
def test_logits_far_apart(topk, cuda_lib):
    """Logits of hundreds, later rows far above the earlier ones (the running
    maximum is raised and the sums rescaled), and heads whose logits are all
    far below zero."""
    inp = _batch(1, 3, [2048], topk, 128, 23)
    q = O.bf16_bits_to_f64(inp.q_attn) * 20.0
    q[:, 64:] *= -1.0
    inp.q_attn = W.f32_to_bf16_bits(q.astype(np.float32))
    kv = O.bf16_bits_to_f64(inp.kv_cache)
    kv[1200:, 512:] = np.abs(kv[1200:, 512:]) * 8.0
    inp.kv_cache = W.f32_to_bf16_bits(kv.astype(np.float32))
    start = 1200 - topk // 2
    _attend(inp, np.tile(np.arange(start, start + topk), (3, 1)))


@pytest.mark.parametrize("page", [1, 3, 16, 64, 256])
def test_pages(page, cuda_lib):
    max_L = -(-2048 // page) * page
    inp = _batch(3, 1, [700, 2000, 1500], 300, 128, 60 + page, block_size=page, max_L=max_L)
    _attend(inp, _pick(np.random.default_rng(page), inp, 0.05))


@pytest.mark.parametrize("topk", [64, 700])
def test_sequence_map_and_no_lse(topk, cuda_lib):
    """Tokens of different sequences in any order; lse left out."""
    inp = _batch(3, [1, 4, 2], [300, 900, 500], topk, 64, 44)
    order = np.random.default_rng(4).permutation(inp.T)
    inp.seq_of_token, inp.pos, inp.q_attn = inp.seq_of_token[order], inp.pos[order], inp.q_attn[order]
    _attend(inp, _pick(np.random.default_rng(5), inp), seq_map=True, lse=False)


def test_bad_pages_and_sequences_are_reported(cuda_lib):
    """A selected row in an unmapped page or past the cache, and a token of no
    sequence, are recorded; the other tokens keep their results."""
    inp = _batch(4, 1, [640] * 4, 100, 128, 71, block_size=64, max_L=640)
    rows = O.kv4_quantise(inp.kv_cache)
    idx = _pick(np.random.default_rng(6), inp)
    table = inp.block_table.copy()
    inp.block_table[1, int(idx[1, 3]) // 64] = -1
    inp.block_table[2, int(idx[2, 3]) // 64] = rows.shape[0] // 64
    cache = Kv4Cache(rows.shape[0], DEV)
    cache.data.copy_(to_dev(rows, DEV))
    for seq, first in ((None, 0), (np.array([0, 1, 2, 4], np.int32), 0), (np.array([0, 0, 0, -1], np.int32), 3)):
        buf = DecodeBuffers(inp, DEV, kv4=cache, seq_map=True)
        if seq is not None:
            buf.seq.copy_(torch.from_numpy(seq))
        if first == 3:
            buf.block_table.copy_(torch.from_numpy(table))
        buf.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
        buf.run_attn()
        torch.cuda.synchronize()
        assert B.device_error() == DATA_ERROR
        out, lse = buf.out.float().cpu().numpy(), buf.lse.cpu().numpy()
        assert np.isfinite(out).all()
        good = [0, 3] if seq is None else [0]
        for t in good:
            keep = dataclasses.replace(inp, block_table=table)
            _check_tokens(inp.q_attn[t], O.kv4_values(rows[O.cache_rows(keep, t, idx[t])]), inp.scale, out[t], lse[t])
        if seq is not None:
            assert not out[3].any() and np.isneginf(lse[3]).all()


def test_nan_rows_count_only_where_selected(cuda_lib):
    inp = _batch(1, 2, [400], 130, 128, 81)
    inp.kv_cache[300:] = 0x7fc0
    rows = O.kv4_quantise(inp.kv_cache)
    idx = np.stack([np.random.default_rng(7).integers(0, 300, 130)] * 2)
    _attend(inp, idx, rows=rows)
    idx[1, 128] = 350
    buf = _attend(inp, idx, rows=rows, tokens=[0])
    assert torch.isnan(buf.out[1]).all() and torch.isnan(buf.lse[1]).all()


@pytest.mark.parametrize("topk", [8, 17, 70, 130])
def test_nothing_is_left_behind_by_other_rows(topk, cuda_lib):
    """Rows of NaN and infinity fill the shared memory of every SM, in an earlier call
    and in earlier tokens; tokens that select a few clean rows after them are unhurt."""
    n_q = 160
    inp = _batch(1, n_q, [900], topk, 128, 97)
    inp.kv_cache[400:650] = 0x7fc0
    inp.kv_cache[650:] = 0x7f80
    rows = O.kv4_quantise(inp.kv_cache)
    rng = np.random.default_rng(topk)
    bad = rng.integers(400, 900, (n_q, topk))
    _attend(inp, bad, rows=rows, tokens=[])
    clean = rng.integers(0, 400, (n_q, topk))
    _attend(inp, clean, rows=rows, tokens=range(0, n_q, 9))
    for odd in (0, 1):
        mixed = np.where((np.arange(n_q) // 76 % 2 == odd)[:, None], bad, clean)
        _attend(inp, mixed, rows=rows, tokens=[t for t in range(n_q) if t // 76 % 2 != odd][::9])


def test_rows_past_four_gigabytes(cuda_lib):
    """A cache of 4.6 GB: the byte offsets of its last rows need 33 bits."""
    n = 11_000_000
    cache = Kv4Cache(n, DEV)
    inp = _batch(1, 2, [600], 64, 16, 91)
    far = np.int64(n - 600)
    cache.write(to_dev(inp.kv_cache, DEV), torch.arange(n - 600, n, device=DEV))
    rows = O.kv4_quantise(inp.kv_cache)
    assert np.array_equal(cache.data[n - 600:].cpu().numpy(), rows) and not cache.data[:n - 600].any()
    got = cache.read(torch.arange(n - 600, n, device=DEV))
    np.testing.assert_array_equal(got.float().cpu().numpy(), O.kv4_values(rows).astype(np.float32))
    idx = np.random.default_rng(8).integers(0, 599, (2, 64))
    out = torch.empty(2, 16, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(2, 16, device=DEV)
    q, ix = to_dev(inp.q_attn, DEV), torch.from_numpy((idx + far).astype(np.int32)).to(DEV)
    B.dsa_sparse_attn_kv4(B.attn_kv4_args(2, 1, 2, 16, 64, n, inp.scale, q, cache.data, ix, out, lse))
    ok()
    for t in range(2):
        _check_tokens(inp.q_attn[t], O.kv4_values(rows[idx[t]]), inp.scale, out[t].float().cpu().numpy(),
                      lse[t].cpu().numpy())


def test_attention_wrapper_refusals(cuda_lib):
    def args(**ch):
        d = dict(T=2, B=1, n_q=2, H=4, topk=8, max_L=16, scale=0.1,
                 q=torch.zeros(2, 4, 576, dtype=torch.bfloat16, device=DEV),
                 kv4=torch.zeros(16, 416, dtype=torch.uint8, device=DEV),
                 topk_idx=torch.zeros(2, 8, dtype=torch.int32, device=DEV),
                 out=torch.zeros(2, 4, 512, dtype=torch.bfloat16, device=DEV))
        d.update(ch)
        return B.attn_kv4_args(**d)
    f32 = dict(dtype=torch.float32, device=DEV)
    for ch in (dict(q=torch.zeros(2, 4, 576, **f32)), dict(q=torch.zeros(2, 4, 640, dtype=torch.bfloat16, device=DEV)[:, :, :576]),
               dict(out=torch.zeros(2, 4, 576, dtype=torch.bfloat16, device=DEV)), dict(topk_idx=torch.zeros(2, 8, dtype=torch.int64, device=DEV)),
               dict(topk_idx=torch.zeros(2, 9, dtype=torch.int32, device=DEV)), dict(lse=torch.zeros(2, 5, **f32)),
               dict(sink=torch.zeros(3, **f32)), dict(seq_of_token=torch.zeros(2, dtype=torch.int64, device=DEV)),
               dict(block_table=torch.zeros(2, 4, dtype=torch.int32, device=DEV)), dict(kv4=torch.zeros(16, 208, dtype=torch.int16, device=DEV))):
        with pytest.raises(B.DSAError):
            args(**ch)
    with pytest.raises(B.DSAError, match="invalid argument"):
        B.dsa_sparse_attn_kv4(args(max_L=17))
    a = args()
    if B.workspace_bytes("attn_kv4", a):
        with pytest.raises(B.DSAError, match="workspace"):
            B.dsa_sparse_attn_kv4(a, torch.zeros(0, dtype=torch.uint8, device=DEV))
    a = args(T=1, n_q=1, topk=700, max_L=16, q=torch.zeros(1, 4, 576, dtype=torch.bfloat16, device=DEV),
             topk_idx=torch.zeros(1, 700, dtype=torch.int32, device=DEV),
             out=torch.zeros(1, 4, 512, dtype=torch.bfloat16, device=DEV))
    n = B.workspace_bytes("attn_kv4", a)
    assert n > 0
    for bad in (torch.zeros(n, dtype=torch.uint8), torch.zeros(2 * n, dtype=torch.uint8, device=DEV)[::2],
                torch.zeros(1, dtype=torch.uint8, device=DEV).expand(n)):
        with pytest.raises(B.DSAError, match="workspace"):
            B.dsa_sparse_attn_kv4(a, bad)
    ok()


def test_a_workspace_of_the_call_s_own_on_a_side_stream(cuda_lib):
    """Without a workspace each call makes one, which outlives its kernels."""
    inp = _batch(1, 2, [500], 300, 128, 101)
    rows = O.kv4_quantise(inp.kv_cache)
    cache = Kv4Cache(rows.shape[0], DEV)
    cache.data.copy_(to_dev(rows, DEV))
    buf = DecodeBuffers(inp, DEV, kv4=cache)
    idx = _pick(np.random.default_rng(6), inp)
    buf.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        B.dsa_sparse_attn_kv4(buf.aargs, stream=s)
        torch.full((1 << 20,), float("nan"), device=DEV)  # takes freed memory on the current stream
    ok()
    out, lse = buf.out.float().cpu().numpy(), buf.lse.cpu().numpy()
    for t in range(inp.T):
        vals = O.kv4_values(rows[O.cache_rows(inp, 0, idx[t])])
        _check_tokens(inp.q_attn[t], vals, inp.scale, out[t], lse[t])


# ------------------------------------------------------- streams, graphs, chain
def test_side_stream_and_graph_replay(cuda_lib):
    """Write, read and attention captured into one graph on a side stream and
    replayed on new inputs in the same buffers; twice the same inputs give the
    same bits."""
    inp = _batch(2, 2, [500, 600], 200, 128, 95)
    cache = Kv4Cache(inp.kv_cache.shape[0], DEV)
    buf = DecodeBuffers(inp, DEV, kv4=cache)
    idx = _pick(np.random.default_rng(9), inp)
    buf.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
    x, slot = to_dev(inp.kv_cache, DEV), torch.arange(inp.kv_cache.shape[0], device=DEV)
    back = torch.empty_like(x)
    s = torch.cuda.Stream()

    def step():
        cache.write(x, slot)
        cache.read(slot, back)
        buf.run_attn()

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    seen = []
    for seed in (1, 2, 1):
        bits = W.f32_to_bf16_bits(np.random.default_rng(seed).standard_normal(inp.kv_cache.shape).astype(np.float32))
        x.copy_(to_dev(bits, DEV))
        buf.out.zero_()
        g.replay()
        ok()
        rows = O.kv4_quantise(bits)
        assert np.array_equal(cache.data.cpu().numpy(), rows)
        np.testing.assert_array_equal(back.float().cpu().numpy(), O.kv4_values(rows).astype(np.float32))
        out, lse = buf.out.float().cpu().numpy(), buf.lse.cpu().numpy()
        for t in range(inp.T):
            vals = O.kv4_values(rows[O.cache_rows(inp, int(inp.seq_of_token[t]), idx[t])])
            _check_tokens(inp.q_attn[t], vals, inp.scale, out[t], lse[t])
        seen.append((out, lse))
    assert np.array_equal(seen[0][0], seen[2][0]) and np.array_equal(seen[0][1], seen[2][1])


def test_two_streams_at_once(cuda_lib):
    """Two calls with workspaces of their own on two streams."""
    inp = _batch(2, 2, [500, 600], 300, 128, 96)
    rows = O.kv4_quantise(inp.kv_cache)
    cache = Kv4Cache(rows.shape[0], DEV)
    cache.data.copy_(to_dev(rows, DEV))
    idx = [_pick(np.random.default_rng(s), inp) for s in (1, 2)]
    bufs = [DecodeBuffers(inp, DEV, kv4=cache) for _ in idx]
    for b, i in zip(bufs, idx):
        b.topk_idx.copy_(torch.from_numpy(i.astype(np.int32)))
    streams = [torch.cuda.Stream() for _ in idx]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, s in zip(bufs, streams):
            b.run_attn(s)
    ok()
    for b, i in zip(bufs, idx):
        out, lse = b.out.float().cpu().numpy(), b.lse.cpu().numpy()
        for t in range(inp.T):
            vals = O.kv4_values(rows[O.cache_rows(inp, int(inp.seq_of_token[t]), i[t])])
            _check_tokens(inp.q_attn[t], vals, inp.scale, out[t], lse[t])


@pytest.mark.parametrize("H", [16, 128])
def test_many_tokens_with_selections_of_all_lengths(H, cuda_lib):
    """More tokens than clusters, each with its own number of selected rows (none,
    one, up to all, and holes anywhere): the clusters' roles pass from item to item."""
    inp = _batch(2, 130, [700, 900], 420, H, 98)
    rng = np.random.default_rng(H)
    idx = _pick(rng, inp)
    for t in range(inp.T):
        n = int(rng.choice([0, 0, 1, 15, 16, 63, 64, 65, 128, 129, 256, 300, 420]))
        idx[t, n:] = -1
        if t % 3 == 0:
            idx[t, rng.random(420) < 0.4] = -1
    idx[:3] = idx[-3:] = -1
    sink = rng.standard_normal(H) if H == 16 else None
    _attend(inp, idx, sink=sink, tokens=sorted({0, 1, 2, 3, *range(0, inp.T, 11), *range(inp.T - 5, inp.T)}))


def test_each_call_reads_what_the_one_before_wrote(cuda_lib):
    """Write, then the queries out of the cache by a read, then the attention with
    them, enqueued back to back."""
    inp = _batch(1, 150, [2048], 200, 128, 99)
    T, H = inp.T, inp.H
    rows = O.kv4_quantise(inp.kv_cache)
    cache = Kv4Cache(rows.shape[0], DEV)
    buf = DecodeBuffers(inp, DEV, kv4=cache)
    idx = _pick(np.random.default_rng(3), inp)
    buf.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
    rng = np.random.default_rng(4)
    x, n = to_dev(inp.kv_cache, DEV), rows.shape[0]
    for rep in range(4):
        take = rng.integers(0, n, T * H)
        slot, order = to_dev(take.astype(np.int64), DEV), rng.permutation(n)
        where = to_dev(order.astype(np.int64), DEV)
        buf.q_attn.zero_()
        torch.cuda.synchronize()
        cache.write(x, where)
        cache.read(slot, buf.q_attn.view(T * H, 576))
        buf.run_attn()
        ok()
        held = np.empty_like(rows)
        held[order] = rows
        q = W.f32_to_bf16_bits(O.kv4_values(held[take]).astype(np.float32)).reshape(T, H, 576)
        out, lse = buf.out.float().cpu().numpy(), buf.lse.cpu().numpy()
        for t in range(rep, T, 25):
            vals = O.kv4_values(held[O.cache_rows(inp, 0, idx[t])])
            _check_tokens(q[t], vals, inp.scale, out[t], lse[t])


@pytest.mark.parametrize("T,H,topk,rows", [(65535, 1, 3, 5000), (1, 1024, 100, 3000), (2, 130, 3, 1),
                                           (1, 4, 65536, 70001)])
def test_largest_and_smallest_sizes(T, H, topk, rows, cuda_lib):
    """The bounds of the header, one at a time, with lengths of a single row."""
    rng = np.random.default_rng(T + H)
    bits = W.f32_to_bf16_bits(rng.standard_normal((rows, 576)).astype(np.float32))
    held = O.kv4_quantise(bits)
    q = W.f32_to_bf16_bits(rng.standard_normal((T, H, 576)).astype(np.float32))
    idx = rng.integers(0, rows, (T, topk)).astype(np.int32)
    idx[T // 2, 1:] = -1
    scale = 576 ** -0.5
    dq, dkv, didx = to_dev(q, DEV).view(torch.bfloat16), to_dev(held, DEV), to_dev(idx, DEV)
    out = torch.full((T, H, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, H), float("nan"), dtype=torch.float32, device=DEV)
    B.dsa_sparse_attn_kv4(B.attn_kv4_args(T, 1, T, H, topk, rows, scale, dq, dkv, didx, out, lse))
    ok()
    assert bool(torch.isfinite(lse).all()) and bool(torch.isfinite(out).all())
    for t in sorted({0, T // 2, T - 1, *rng.integers(0, T, 8).tolist()}):
        sel = idx[t][idx[t] >= 0]
        _check_tokens(q[t], O.kv4_values(held[sel]), scale, out[t].float().cpu().numpy(), lse[t].cpu().numpy())


@pytest.mark.parametrize("n_q,topk", [(2, 700), (160, 300)])
def test_wait_limit_runs_out_then_the_next_call_passes(n_q, topk, cuda_lib):
    """With a 1 ns limit after an L2 flush waits give up, in one item and in the
    midst of several; the call reports it and the next one is right."""
    inp = _batch(1, n_q, [2048], topk, 128, 100)
    rows = O.kv4_quantise(inp.kv_cache)
    cache = Kv4Cache(rows.shape[0], DEV)
    cache.data.copy_(to_dev(rows, DEV))
    buf = DecodeBuffers(inp, DEV, kv4=cache)
    idx = _pick(np.random.default_rng(5), inp)
    buf.topk_idx.copy_(torch.from_numpy(idx.astype(np.int32)))
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    ok()
    B.set_wait_limit_ns(1)
    try:
        flush.zero_()
        buf.run_attn()
        torch.cuda.synchronize()
        assert B.device_error() == TIMEOUT
    finally:
        B.set_wait_limit_ns(0)
    buf.run_attn()
    ok()
    out, lse = buf.out.float().cpu().numpy(), buf.lse.cpu().numpy()
    for t in range(0, inp.T, 1 + inp.T // 10):
        vals = O.kv4_values(rows[O.cache_rows(inp, 0, idx[t])])
        _check_tokens(inp.q_attn[t], vals, inp.scale, out[t], lse[t])


def test_dia_step_on_a_4_bit_cache(cuda_lib):
    """The whole DIA step with its latent cache in 4 bits: the MLA Prolog's rows
    are what the cache holds after quantisation, every other row is as it was,
    and the attention reads them with the MLA Prolog's query.  (Those rows are
    held to the oracle's, not to another run's: the MLA Prolog adds its partial
    sums with atomics, in any order.)"""
    dia = W.dia_decode(B=2, n_q=2, L=4096)
    inp = dia.decode
    st = DiaBuffers(dia, DEV, kv4=True)
    st.run()
    ok()
    _close_bf16(st.kv.float().cpu().numpy(), O.mla_prolog(dia.mla)["kv"], "latent rows")
    rows = O.kv4_quantise(inp.kv_cache)
    rows[dia.mla.slot] = O.kv4_quantise(_bits(st.kv))
    assert np.array_equal(st.kv4.data.cpu().numpy(), rows)
    idx = st.buf.topk_idx.cpu().numpy()
    q, out, lse = _bits(st.mla.q), st.buf.out.float().cpu().numpy(), st.buf.lse.cpu().numpy()
    for t in range(inp.T):
        vals = O.kv4_values(rows[O.cache_rows(inp, int(inp.seq_of_token[t]), idx[t][idx[t] >= 0])])
        _check_tokens(q[t], vals, inp.scale, out[t], lse[t])
