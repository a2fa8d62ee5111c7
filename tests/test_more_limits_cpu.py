"""The ends of the ranges of the step maps and the latent attention, without a GPU:
sizes whose index arithmetic would leave 32 bits, and arrays over one another, are
refused before anything is launched."""
import pytest

from sparse_attention_prolog_gb300 import binding as B
from test_abi_cpu import lib  # noqa: F401
from test_more_operators_cpu import BASE, INVALID, UNSUPPORTED, _with

FAR = 1 << 40  # apart from all else by more than the largest array here


@pytest.mark.parametrize("name", ["T", "n_free"])
def test_step_maps_leave_room_for_a_stride(lib, name):  # noqa: F811
    a = B.StepMapsArgs(4, 16, 64, 32, 100, *[BASE + i * FAR for i in range(11)])
    for n in (2 ** 31 - 2 ** 20 + 1, 2 ** 31 - 1):
        assert lib.dsa_step_maps(_with(a, **{name: n}), None) == UNSUPPORTED, n
    # (the largest is only looked at: something else is wrong with the call)
    assert lib.dsa_step_maps(_with(a, slot=a.slot + 4, **{name: 2 ** 31 - 2 ** 20}), None) == INVALID


def test_latent_attn_leaves_room_behind_the_last_row(lib):  # noqa: F811
    p = [BASE + i * FAR for i in range(8)]
    a = B.LatentAttnArgs(8, 4, 2, 128, 64, 0.1, p[0], p[1], 4096, p[4], 64, 1, None, p[2], p[3], None, None)
    for blocks, size in ((2 ** 25 - 1, 64), (2 ** 25 - 15, 64), (2 ** 27 - 63, 16)):
        kw = {"max_blocks": blocks, "block_size": size, "max_L": blocks * size}
        assert lib.dsa_latent_attn(_with(a, **kw), None, 0, None) == UNSUPPORTED, kw
        assert lib.dsa_latent_attn_workspace(_with(a, **kw)) == 0
    kw = {"max_blocks": 2 ** 25 - 16, "block_size": 64, "max_L": 2 ** 31 - 1024}
    assert lib.dsa_latent_attn_workspace(_with(a, **kw)) > 0
    # contiguous, where a sequence's rows are the cache's
    kw = {"block_table": 0, "T": 1, "B": 1, "n_q": 1, "max_L": 2 ** 31 - 1023, "cache_rows": 2 ** 31 - 1}
    assert lib.dsa_latent_attn(_with(a, **kw), None, 0, None) == UNSUPPORTED


def test_latent_attn_refuses_a_scale_that_overflows_in_base_2(lib):  # noqa: F811
    p = [BASE + i * FAR for i in range(8)]
    a = B.LatentAttnArgs(8, 4, 2, 128, 4096, 0.1, p[0], p[1], 4 * 4096, None, 0, 0, None, p[2], p[3], None, None)
    for scale in (2.4e38, 3.4e38):  # times log2(e) past fp32's largest, 3.4028e38
        assert lib.dsa_latent_attn(_with(a, scale=scale), None, 0, None) == INVALID
        assert lib.dsa_latent_attn_workspace(_with(a, scale=scale)) == 0
    assert lib.dsa_latent_attn_workspace(_with(a, scale=2.3e38)) > 0


def test_step_maps_refuse_arrays_over_one_another(lib):  # noqa: F811
    """Every CTA reads the lengths and the list while the first ones write, so nothing
    that is written may lie over what is read, or over what else is written."""
    sizes = {"cached": 16, "fresh": 16, "free_pages": 400, "free_head": 4, "block_table": 4 * 4 * 32, "cu_tokens": 20,
             "kv_len": 16, "counts": 12, "seq_of_token": 64, "pos": 64, "slot": 128}
    written = list(sizes)[4:]
    base = {f: BASE + i * FAR for i, f in enumerate(sizes)}
    a = B.StepMapsArgs(4, 16, 64, 32, 100, *base.values())
    call = lambda **kw: lib.dsa_step_maps(_with(a, **kw), None)  # noqa: E731
    for out in written:
        step = 8 if out == "slot" else 4
        for other, n in sizes.items():
            if other == out:
                continue
            for at in {0, -(-n // step) * step - step, -sizes[out] + step}:  # whole, its end, its beginning
                assert call(**{out: base[other] + at}) == INVALID, (out, other, at)
