"""The latent attention, the residual norm and the step maps at their limits: a wait
that runs out, sequences of no tokens in a padded batch of wide blocks, page sizes
past a tile, the longest rows and offsets past 2^31 elements, the most requests."""
import numpy as np
import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B
from sparse_attention_prolog_gb300.pipeline import StepMaps
from test_gpu_latent import TIMEOUT, Case, ok

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("n,lens", [([1, 1, 1], [9000, 70, 4000]), ([2, 5, 1], [9000, 700, 4000])])
def test_a_wait_that_runs_out_then_the_next_call_passes(n, lens, cuda_lib):
    """With a 1 ns limit the first wait for a copy from HBM gives up; the CTAs let
    their copies and products finish and leave.  (Blocks of 128 and of 256 rows.)"""
    c = Case(n, lens, 128, page=64)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    ws = torch.empty(B.workspace_bytes("latent_attn", c.args()), dtype=torch.uint8, device=DEV)
    ok()
    B.set_wait_limit_ns(1)
    try:
        flush.zero_()
        c.run(ws)
        torch.cuda.synchronize()
        assert B.device_error() == TIMEOUT
    finally:
        B.set_wait_limit_ns(0)
    ws.zero_()
    c.fresh()
    c.run(ws)
    ok()
    c.check()


@pytest.mark.parametrize("n,lens,H,page,pad", [
    ([0, 3, 0, 0, 7, 0], [500, 300, 0, 64, 1, 128], 128, 16, 5),  # wide blocks, idle sequences, fewer rows than tokens
    ([0, 0, 0], [100, 0, 1], 16, 64, 3),                          # nothing but padding
    ([40, 0, 3], [4000, 20, 3], 16, 32, 1),
    ([1, 300], [20000, 300], 16, 512, 2),                         # a first block of nothing but a prompt's beginning
    ([2], [1], 1024, 8, 0),                                       # the most heads; a token before the sequence
    ([3, 3], [65536, 200], 64, 65536, 0)])                        # one page a sequence
def test_batches_with_idle_sequences_and_large_pages(n, lens, H, page, pad, cuda_lib):
    c = Case(n, lens, H, page=page, pad=pad, sink=True)
    c.run()
    ok()
    c.check()


def test_two_calls_at_once_share_nothing(cuda_lib):
    """Both kinds of blocks on two streams, with workspaces of their own, many times."""
    cases = [Case([2, 3, 2], [3000, 500, 7000], 128, page=64, seed=1), Case([1] * 9, [900 * i for i in range(1, 10)], 64, seed=2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    ok()
    for c in cases:
        c.check()


@pytest.mark.parametrize("D,off", [(32768, 0), (32768, 1), (32767, 0), (20001, 3), (9001, 0)])
@pytest.mark.parametrize("x,res", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)])
def test_long_rows_of_any_alignment(D, off, x, res, cuda_lib):
    """y within a rounding (2^-8) and fp32's (2^-18: a sum of up to 2^15 squares, of
    which a thread adds 32 and the rest are joined in 10 steps, a root, two products)."""
    g = torch.Generator(device=DEV).manual_seed(D + off)
    a = torch.randn(3 * D + off, device=DEV, generator=g).to(x)[off:].view(3, D)
    r = torch.randn(3 * D + off, device=DEV, generator=g).to(res)[off:].view(3, D)
    gamma = torch.randn(D, device=DEV, generator=g)
    out, y = torch.empty_like(r), torch.empty(3, D, dtype=torch.bfloat16, device=DEV)
    codes, scale = torch.empty(3, D, dtype=torch.int8, device=DEV), torch.empty(3, device=DEV)
    B.dsa_add_rmsnorm(a, gamma, 1e-5, r, out, y, codes, scale)
    ok()
    h = (a.float() + r.float()).to(res)
    assert torch.equal(out, h)
    z = h.double()
    z = z / (z.square().mean(1, keepdim=True) + 1e-5).sqrt() * gamma.double()
    assert bool(((y.double() - z).abs() <= z.abs() * (2.0 ** -8 + 2.0 ** -18) + 2.0 ** -133).all())
    top = z.abs().amax(1)
    assert bool(((scale.double() * 127 - top).abs() <= top * 2.0 ** -18).all())
    assert bool(((codes.double() * scale.double()[:, None] - z).abs() <= scale.double()[:, None] * (0.5 + 2.0 ** -9)).all())


@pytest.mark.parametrize("D", [1, 7, 8, 9, 23, 24, 40, 41, 264, 517])
@pytest.mark.parametrize("x_kind,r_kind", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                           (torch.bfloat16, None)])
def test_every_alignment_of_every_array(D, x_kind, r_kind, cuda_lib):
    """Rows of x, the residuals, gamma, y and the codes at offsets of their own, and what
    lies before, between and behind the rows as it was.  Bounds as above; with the codes'
    scale as the kernel gave it, a code is within half of one and 2^-9 (127 of the
    value's 2^-18 and of the quotient's own roundings)."""
    T = 5
    rng = np.random.default_rng(D)
    g = torch.Generator(device=DEV).manual_seed(D)

    def rows(kind, off, stride, fill=None):
        whole = torch.full((off + T * stride + 16,), 77, dtype=kind, device=DEV)
        view = torch.as_strided(whole, (T, D), (stride, 1), off)
        if fill is None:
            view.copy_(torch.randn(T, D, device=DEV, generator=g))
        return whole, view

    def untouched(whole, off, stride):
        mask = torch.ones_like(whole, dtype=torch.bool)
        torch.as_strided(mask, (T, D), (stride, 1), off).zero_()
        return bool((whole[mask] == 77).all())

    for _ in range(24):
        off = [int(v) for v in rng.integers(0, 17, 6)]
        gap = [int(v) for v in rng.integers(0, 10, 3)]
        _, x = rows(x_kind, off[0], D + gap[0])
        gamma = torch.randn(D + off[5], device=DEV, generator=g)[off[5]:]
        y_all, y = rows(torch.bfloat16, off[3], D, 0)
        c_all, codes = rows(torch.int8, off[4], D, 0)
        scale = torch.zeros(T, device=DEV)
        res = out = None
        h = x
        if r_kind is not None:
            r_all, res = rows(r_kind, off[1], D + gap[1])
            in_place = rng.random() < 0.3
            o_all, out = (r_all, res) if in_place else rows(r_kind, off[2], D + gap[2], 0)
            h = (x.float() + res.float()).to(r_kind)
        with_y, with_codes = rng.choice([True, True, False]), rng.choice([True, True, False])
        if not with_y and not with_codes:
            with_y = True
        B.dsa_add_rmsnorm(x, gamma, 1e-5, res, out, y if with_y else None, codes if with_codes else None,
                          scale if with_codes else None)
        ok()
        if r_kind is not None:
            assert torch.equal(out, h)
            assert untouched(o_all, *((off[1], D + gap[1]) if in_place else (off[2], D + gap[2])))
        z = h.double()
        z = z / (z.square().mean(1, keepdim=True) + 1e-5).sqrt() * gamma.double()
        assert untouched(y_all, off[3], D) and untouched(c_all, off[4], D)
        if with_y:
            assert bool(((y.double() - z).abs() <= z.abs() * (2.0 ** -8 + 2.0 ** -18) + 2.0 ** -133).all())
        if with_codes:
            s = scale.double()[:, None]
            assert bool(((scale.double() * 127 - z.abs().amax(1)).abs() <= z.abs().amax(1) * 2.0 ** -18).all())
            assert bool(((codes.double() * s - z).abs() <= s * (0.5 + 2.0 ** -9)).all())


def test_rows_past_4_gb(cuda_lib):
    """T * D past 2^31: the last rows' offsets need 64 bits."""
    T, D = 300_001, 7168
    x = torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
    x.fill_(3.0)
    x[-1] = torch.arange(D, device=DEV).bfloat16()
    y, codes, scale = torch.empty_like(x), torch.empty(T, D, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    res = torch.zeros_like(x)
    B.dsa_add_rmsnorm(x, torch.ones(D, device=DEV), 0.0, res, res, y, codes, scale)
    ok()
    assert torch.equal(res[-3:], x[-3:]) and bool((y[:-1:1000] == 1.0).all()) and bool((codes[:-1:1000] == 127).all())
    assert bool((y[-2] == 1.0).all()) and bool((codes[-2] == 127).all())
    z = x[-1].double()
    z = z / z.square().mean().sqrt()
    assert bool(((y[-1].double() - z).abs() <= z * (2.0 ** -8 + 2.0 ** -18)).all())
    assert abs(float(scale[-1]) * 127 - float(z.max())) <= float(z.max()) * 2.0 ** -18


def test_the_most_requests(cuda_lib):
    """8192 requests, three steps with idle ones; pages of the longest tables."""
    rng = np.random.default_rng(0)
    n, bs, blocks = 8192, 64, 40
    free = rng.permutation(n * 8).astype(np.int32)
    m = StepMaps(n, 3 * n, bs, blocks, torch.from_numpy(free).to(DEV))
    table, lens, head = np.full((n, blocks), -1), np.zeros(n, dtype=int), 0
    for _ in range(3):
        fresh = rng.integers(0, 3, n)
        fresh[rng.integers(0, n, 5)] = 120
        m.run(torch.from_numpy(fresh.astype(np.int32)).to(DEV))
        ok()
        want = []
        for b in range(n):
            for pos in range(lens[b], lens[b] + fresh[b]):
                if pos % bs == 0:
                    table[b, pos // bs] = free[head]
                    head += 1
                want.append((b, pos, table[b, pos // bs] * bs + pos % bs))
        lens += fresh
        want = np.array(want)
        k = len(want)
        assert m.counts[m.step].tolist() == [k, head, n]
        assert np.array_equal(m.kv_len.cpu().numpy(), lens) and np.array_equal(m.block_table.cpu().numpy(), table)
        got = np.stack([m.seq_of_token.cpu().numpy(), m.pos.cpu().numpy(), m.slot.cpu().numpy()], 1)
        assert np.array_equal(got[:k], want)
        assert bool((m.slot[k:] == -1).all()) and bool((m.pos[k:] == 0).all())


def test_numbers_that_no_argument_block_holds(cuda_lib):
    x, y = torch.zeros(2, 8, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 8, dtype=torch.bfloat16, device=DEV)
    for eps in ("1e-6", None, -1.0, float("nan"), 1e300):
        with pytest.raises(B.DSAError):
            B.dsa_add_rmsnorm(x, torch.ones(8, device=DEV), eps, y=y)
    i = torch.zeros(1, dtype=torch.int32, device=DEV)
    for size in (2 ** 31, 0, -1, 2.5):
        with pytest.raises(B.DSAError):
            B.dsa_step_maps(i, i, i, i.view(1, 1), size, i.new_zeros(2), i.clone(), i.new_zeros(3), i.clone(), i.clone(),
                            torch.zeros(1, dtype=torch.int64, device=DEV))
