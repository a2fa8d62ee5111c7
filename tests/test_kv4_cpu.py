"""The 4-bit latent cache without a GPU: the oracle's quantiser and row layout
against hand-worked cases and properties, the C structs, and every host-side
refusal of the three entry points and of their Python wrappers."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def bf16_bits(x) -> np.ndarray:
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


# ------------------------------------------------------------------ oracle
def test_scale_bytes_are_monotonic_with_four_significant_bits():
    s = O.kv4_scale(np.arange(255))
    assert s[0] == 2.0 ** -15 and s[120] == 1.0 and s[121] == 1.125 and s[254] == 1.75 * 2.0 ** 16
    assert (np.diff(s) > 0).all() and np.isnan(O.kv4_scale(255))
    m, _ = np.frexp(s)
    assert np.array_equal(m * 16, np.rint(m * 16))


def test_every_value_is_exact_in_bf16():
    v = np.arange(-8, 8)[:, None] * O.kv4_scale(np.arange(255))[None, :]
    assert np.array_equal(O.bf16_bits_to_f64(bf16_bits(v)), v)


def test_a_row_of_zero_bytes_is_zero():
    assert not O.kv4_values(np.zeros((2, 416), np.uint8)).any()


def test_layout_by_hand():
    """Group 0 holds 0..7 and -7..0 (largest 7, scale 1); dims 0..7 sit in the
    first word as nibbles 0 2 4 6 1 3 5 7, dims 8..15 (-7..0, two's
    complement 9 a b c d e f 0) in the second."""
    x = np.zeros((1, 576), np.float32)
    x[0, :16] = [0, 1, 2, 3, 4, 5, 6, 7, -7, -6, -5, -4, -3, -2, -1, 0]
    x[0, 512:] = np.arange(64)
    row = O.kv4_quantise(bf16_bits(x))[0]
    assert row[:8].tolist() == [0x20, 0x64, 0x31, 0x75, 0xb9, 0xfd, 0xca, 0x0e]
    assert row[256] == 120 and (row[257:288] == 0).all()
    assert np.array_equal(row[288:].view(np.uint16), bf16_bits(x)[0, 512:])
    assert np.array_equal(O.kv4_values(row[None])[0], x[0])


def test_half_a_scale_and_the_clamps():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 576)).astype(np.float32) * np.exp(rng.uniform(-6, 6, (64, 1))).astype(np.float32)
    bits = bf16_bits(x)
    rows = O.kv4_quantise(bits)
    s = O.kv4_scale(rows[:, 256:288]).repeat(16, 1)
    d = np.abs(O.kv4_values(rows) - O.bf16_bits_to_f64(bits))
    assert (d[:, :512] <= s / 2).all() and not d[:, 512:].any()
    amax = np.abs(O.bf16_bits_to_f64(bits)[:, :512]).reshape(64, 32, 16).max(-1)
    assert (np.abs(O.kv4_scale(rows[:, 256:288]) - amax / 7) <= amax / 7 / 16).all()  # half a step of 4 bits
    x[:] = 0
    x[0, 0], x[0, 16], x[0, 17] = 1e30, 2.0 ** -17, 2.0 ** -15 * 1.5
    v = O.kv4_values(O.kv4_quantise(bf16_bits(x)))[0]
    assert v[0] == 7 * 1.75 * 2.0 ** 16          # the largest scale
    assert v[16] == 0 and v[17] == 2.0 ** -14    # the smallest scale: 1.5 steps round to the even 2


def test_ties_go_to_even():
    x = np.zeros((1, 576), np.float32)
    x[0, :6] = [7, 0.5, 1.5, 2.5, -0.5, -1.5]    # scale 1
    x[0, 16] = 7 * 1.0625                        # scale halfway between 1 and 1.125: the even significand 1
    x[0, 32] = 7 * 1.1875                        # halfway between 1.125 and 1.25: 1.25
    rows = O.kv4_quantise(bf16_bits(x))
    assert O.kv4_values(rows)[0, :6].tolist() == [7, 0, 2, 2, 0, -2]
    assert rows[0, 256:259].tolist() == [120, 120, 122]


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_group_with_a_nonfinite_value_reads_as_nan(bad):
    x = np.ones((1, 576), np.float32)
    x[0, 37] = bad
    rows = O.kv4_quantise(bf16_bits(x))
    v = O.kv4_values(rows)[0]
    assert rows[0, 258] == 255 and not rows[0, 16:24].any()
    assert np.isnan(v[32:48]).all() and np.isfinite(np.delete(v, np.arange(32, 48))).all()


# --------------------------------------------------------------------- ABI
@pytest.fixture(scope="module")
def lib():
    import glob
    from sparse_attention_prolog_gb300 import binding, build
    srcs = glob.glob(os.path.join(build.CSRC, "*")) + [os.path.join(ROOT, "include", "dsa.h")]
    if not os.path.exists(binding.LIB_PATH) or \
            os.path.getmtime(binding.LIB_PATH) < max(os.path.getmtime(s) for s in srcs):
        build.build()
    return binding.load()


def test_struct_layouts_match_the_header(lib, tmp_path):
    from sparse_attention_prolog_gb300 import binding as B
    structs = (("dsa_kv4_write_args", B.Kv4WriteArgs), ("dsa_kv4_read_args", B.Kv4ReadArgs),
               ("dsa_attn_kv4_args", B.AttnKv4Args))
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "dsa.h"', "int main(void) {",
             'printf("row %d\\n", DSA_KV4_ROW_BYTES);']
    for cname, py in structs:
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                                 text=True).stdout.splitlines())
    assert int(got["row"]) == B.KV4_ROW_BYTES == O.KV4_ROW
    for cname, py in structs:
        assert int(got[cname]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(py, f).offset, f"{cname}.{f}"


OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4
BASE = 1 << 20  # fake, aligned device addresses: checked on the host, never read


def test_write_and_read_refusals(lib):
    from sparse_attention_prolog_gb300 import binding as B
    null = ctypes.c_void_p(0)
    for struct, fn, stride, buf in ((B.Kv4WriteArgs, lib.dsa_kv4_write, "x_stride", "x"),
                                    (B.Kv4ReadArgs, lib.dsa_kv4_read, "out_stride", "out")):
        assert fn(None, null) == INVALID

        def call(**change):
            a = struct()
            a.n, a.cache_rows = 4, 64
            setattr(a, stride, 576)
            for i, f in enumerate((buf, "kv4", "slot")):
                setattr(a, f, BASE * (i + 1))
            for k, v in change.items():
                setattr(a, k, v)
            return fn(ctypes.byref(a), null)

        assert call(n=-1) == INVALID
        assert call(**{stride: 575}) == INVALID and call(**{stride: 580}) == INVALID
        assert call(**{stride: -576}) == INVALID
        assert call(cache_rows=-1) == INVALID and call(cache_rows=2 ** 31) == UNSUPPORTED
        for f, off in ((buf, 8), ("kv4", 8), ("slot", 4)):
            assert call(**{f: None}) == INVALID and call(**{f: BASE + off}) == INVALID
        assert call(n=0, **{buf: None}) == OK


def test_attention_refusals(lib):
    from sparse_attention_prolog_gb300 import binding as B
    null = ctypes.c_void_p(0)
    assert lib.dsa_sparse_attn_kv4(None, null, 0, null) == INVALID
    assert lib.dsa_sparse_attn_kv4_workspace(None) == 0

    def call(**change):
        a = B.AttnKv4Args()
        a.T, a.B, a.n_q, a.H, a.topk, a.max_L, a.scale, a.cache_rows = 8, 4, 2, 128, 2048, 4096, 0.07, 4 * 4096
        for i, f in enumerate(("q", "kv4", "topk_idx", "out")):
            setattr(a, f, BASE * (i + 1))
        for k, v in change.items():
            setattr(a, k, v)
        return lib.dsa_sparse_attn_kv4(ctypes.byref(a), null, 0, null)

    assert call() in (OK, WORKSPACE, CUDA)  # past the argument checks: the rest needs a GPU
    assert call(T=7) == INVALID                                   # T != B * n_q
    assert call(T=7, seq_of_token=BASE) in (OK, WORKSPACE, CUDA)  # a map lifts that
    assert call(seq_of_token=BASE + 2) == INVALID
    assert call(T=65536, B=65536, n_q=1, max_L=1, cache_rows=65536) == UNSUPPORTED
    for f in ("H", "topk", "max_L", "cache_rows"):
        assert call(**{f: 0}) == INVALID and call(**{f: -3}) == INVALID
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == INVALID
    assert call(H=1025) == UNSUPPORTED and call(topk=65537) == UNSUPPORTED
    assert call(cache_rows=2 ** 31) == UNSUPPORTED
    assert call(cache_rows=4 * 4096 - 1) == INVALID               # a contiguous cache that ends early
    for f, off in (("q", 8), ("kv4", 8), ("topk_idx", 2), ("out", 8)):
        assert call(**{f: None}) == INVALID and call(**{f: BASE + off}) == INVALID
    assert call(lse=BASE + 2) == INVALID and call(sink=BASE + 2) == INVALID
    paged = dict(block_table=BASE * 9, block_size=64, max_blocks=64)
    assert call(**paged) in (OK, WORKSPACE, CUDA)
    assert call(**{**paged, "block_table": BASE + 2}) == INVALID
    assert call(**{**paged, "block_size": 0}) == INVALID and call(**{**paged, "max_blocks": 63}) == INVALID
    assert call(T=0, q=None) == OK                                # no tokens: nothing to do


def test_wrappers_refuse_cpu_tensors():
    from sparse_attention_prolog_gb300 import binding as B
    x, slot = torch.zeros(2, 576, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    kv4 = torch.zeros(4, 416, dtype=torch.uint8)
    for call in (lambda: B.dsa_kv4_write(x, kv4, slot), lambda: B.dsa_kv4_read(kv4, slot, x),
                 lambda: B.attn_kv4_args(2, 1, 2, 1, 4, 4, 1.0, x[:, None], kv4, slot[:, None].int(), x[:, None])):
        with pytest.raises(B.DSAError, match="not a CUDA tensor"):
            call()


def _cpu_attention_args(monkeypatch, **change):
    """An argument block over CPU tensors (the checks of the tensors left out)."""
    from sparse_attention_prolog_gb300 import binding as B
    monkeypatch.setattr(B, "_device", lambda name, t: 0)
    monkeypatch.setattr(B, "_tensor", lambda *a, **k: None)
    d = dict(T=2, B=1, n_q=2, H=4, topk=8, max_L=16, scale=0.1, q=torch.zeros(2, 4, 576, dtype=torch.bfloat16),
             kv4=torch.zeros(16, 416, dtype=torch.uint8), topk_idx=torch.zeros(2, 8, dtype=torch.int32),
             out=torch.zeros(2, 4, 512, dtype=torch.bfloat16))
    d.update(change)
    return B.attn_kv4_args(**d)


@pytest.mark.parametrize("name", ["T", "B", "n_q", "H", "topk", "max_L", "block_size"])
def test_sizes_past_32_bits_are_refused(name, monkeypatch):
    """(A C int would take their lower 32 bits: another, valid size.)"""
    from sparse_attention_prolog_gb300 import binding as B
    _cpu_attention_args(monkeypatch)
    for value in (2 ** 31, 2 ** 32 + 2, -2 ** 31 - 1):
        with pytest.raises(B.DSAError, match=name):
            _cpu_attention_args(monkeypatch, **{name: value})
    assert getattr(_cpu_attention_args(monkeypatch, **{name: 2 ** 31 - 1}), name) == 2 ** 31 - 1
