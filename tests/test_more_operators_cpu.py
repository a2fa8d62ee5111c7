"""The step maps, the latent attention and the residual norm without a GPU: the ctypes
structs match the header, the C entry points refuse what they cannot take before
anything is launched, argument blocks keep their tensors, and the wrappers make
memory in the pool of the call's stream."""
import ctypes
import gc
import os
import subprocess
import weakref

import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B
from test_abi_cpu import ROOT, lib  # noqa: F401
from test_streams_cpu import SIDE, Memory, made  # noqa: F401

BASE = 1 << 20  # fake, aligned device addresses: only validated, never read
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def test_struct_layout_matches_header(lib, tmp_path):  # noqa: F811
    structs = (("dsa_step_maps_args", B.StepMapsArgs), ("dsa_latent_attn_args", B.LatentAttnArgs),
               ("dsa_add_rmsnorm_args", B.AddRmsnormArgs))
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "dsa.h"', "int main(void) {"]
    for cname, py in structs:
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    got = dict(line.split() for line in out if line)
    for cname, py in structs:
        assert int(got[cname]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(py, f).offset, f"{cname}.{f}"


def test_packed_blocks_are_the_structs(lib):  # noqa: F811
    a = B.StepMapsArgs(*range(1, 6), *[BASE + i * 64 for i in range(11)])
    assert B._STEP_MAPS.pack(*[getattr(a, f) or 0 for f, _ in a._fields_]) == bytes(a)
    a = B.AddRmsnormArgs(1, 2, 3.5, 1, 0, 1, 7, 8, 2 ** 40, *[BASE + i * 64 for i in range(7)])
    assert B._ADD_RMSNORM.pack(*[getattr(a, f) or 0 for f, _ in a._fields_]) == bytes(a)
    assert lib.step_maps_packed(B._STEP_MAPS.pack(-1, *[0] * 15), None) == INVALID
    assert lib.step_maps_packed(B._STEP_MAPS.pack(*[0] * 16), None) == OK


def _with(args, **kw):
    c = type(args).from_buffer_copy(args)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def test_step_maps_refuse(lib):  # noqa: F811
    a = B.StepMapsArgs(4, 16, 64, 32, 100, *[BASE + i * 65536 for i in range(11)])
    call = lambda **kw: lib.dsa_step_maps(_with(a, **kw), None)  # noqa: E731
    assert lib.dsa_step_maps(None, None) == INVALID
    assert call(B=0) == OK
    for kw in ({"B": -1}, {"T": -1}, {"n_free": -1}, {"block_size": 0}, {"max_blocks": 0}, {"cached": 0}, {"fresh": 0},
               {"free_pages": 0}, {"block_table": 0}, {"cu_tokens": 0}, {"kv_len": 0}, {"counts": 0}, {"seq_of_token": 0},
               {"pos": 0}, {"slot": 0}, {"cached": BASE + 2}, {"slot": BASE + 4}, {"free_head": BASE + 1}):
        assert call(**kw) == INVALID, kw
    for kw in ({"B": 8193}, {"block_size": 1 << 30, "max_blocks": 2}, {"max_blocks": 1 << 26}):
        assert call(**kw) == UNSUPPORTED, kw
    # outputs over inputs that are read meanwhile, whole or in part
    for kw in ({"kv_len": a.cached}, {"kv_len": a.fresh}, {"kv_len": a.cached + 12}, {"cu_tokens": a.fresh - 16},
               {"counts": a.free_head}, {"counts": a.free_head - 8}, {"cu_tokens": a.free_head}, {"counts": a.cached}):
        assert call(**kw) == INVALID, kw


def test_latent_attn_refuses(lib):  # noqa: F811
    p = [BASE + i * 65536 for i in range(8)]
    a = B.LatentAttnArgs(8, 4, 2, 128, 4096, 0.1, p[0], p[1], 4 * 4096, None, 0, 0, None, p[2], p[3], None, None)
    call = lambda **kw: lib.dsa_latent_attn(_with(a, **kw), None, 0, None)  # noqa: E731
    size = lambda **kw: lib.dsa_latent_attn_workspace(_with(a, **kw))  # noqa: E731
    paged = {"block_table": p[4], "block_size": 64, "max_blocks": 64}
    assert lib.dsa_latent_attn(None, None, 0, None) == INVALID and lib.dsa_latent_attn_workspace(None) == 0
    assert call(T=0) == OK and call(T=0, q=0, kv=0) == OK and size(T=0) == 0
    assert size() > 0 and call() == WORKSPACE and size(**paged) > 0 and size(cu_tokens=p[5], T=5) > 0
    for kw in ({"T": -1}, {"B": 0}, {"H": 0}, {"max_L": 0}, {"cache_rows": 0}, {"scale": 0.0}, {"scale": -1.0},
               {"scale": float("nan")}, {"scale": float("inf")}, {"n_q": 3}, {"n_q": 0}, {"T": 7}, {"cache_rows": 4 * 4096 - 1},
               {"q": 0}, {"kv": 0}, {"out": 0}, {"kv_len": 0}, {"q": BASE + 8}, {"kv": BASE + 8}, {"out": BASE + 16},
               {"kv_len": BASE + 2}, {"lse": BASE + 2}, {"sink": BASE + 2}, {"cu_tokens": BASE + 2},
               {**paged, "max_blocks": 63}, {**paged, "block_size": 0}, {**paged, "block_table": p[4] + 2}):
        assert call(**kw) == INVALID and size(**kw) == 0, kw
    for kw in ({"H": 1025}, {"B": 65536, "cu_tokens": p[5], "cache_rows": 2 ** 31 - 1, "max_L": 1}, {"cache_rows": 2 ** 31},
               {"T": 2 ** 24, "cu_tokens": p[5]}, {**paged, "block_size": 4, "max_blocks": 1024},
               {**paged, "block_size": 96, "max_blocks": 1, "max_L": 96}):
        assert call(**kw) == UNSUPPORTED and size(**kw) == 0, kw


def test_add_rmsnorm_refuses(lib):  # noqa: F811
    p = [BASE + i * 65536 for i in range(7)]
    a = B.AddRmsnormArgs(4, 64, 1e-6, 0, 0, 0, 64, 64, 64, *p)
    call = lambda **kw: lib.dsa_add_rmsnorm(_with(a, **kw), None)  # noqa: E731
    assert lib.dsa_add_rmsnorm(None, None) == INVALID
    assert call(T=0) == OK and call(T=0, x=0) == OK
    for kw in ({"T": -1}, {"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}, {"x": 0}, {"gamma": 0},
               {"residual": 0}, {"residual_out": 0}, {"codes": 0}, {"code_scale": 0}, {"y": 0, "codes": 0, "code_scale": 0},
               {"x_stride": 63}, {"residual_stride": 0}, {"residual_out_stride": -64}, {"x": BASE + 1}, {"gamma": BASE + 2},
               {"residual_fp32": 1, "residual": p[1] + 2}, {"residual_out": p[1], "residual_out_stride": 72}, {"y": p[4] + 1},
               {"code_scale": p[6] + 2}, {"x_fp16": 2}, {"residual_fp32": -1}):
        assert call(**kw) == INVALID, kw
    assert call(D=0) == UNSUPPORTED and call(D=32769) == UNSUPPORTED


def test_an_argument_block_keeps_its_tensors(monkeypatch):
    monkeypatch.setattr(B, "_device", lambda name, t: 0)
    monkeypatch.setattr(B, "_tensor", lambda *a, **k: None)
    tensors = {n: torch.zeros(2, 4) for n in "q kv kv_len out lse cu_tokens block_table sink".split()}
    args = B.latent_attn_args(T=2, B=1, H=1, max_L=16, scale=1.0, block_size=4, **tensors)
    held = {n: (weakref.ref(t), t.data_ptr()) for n, t in tensors.items()}
    del tensors
    gc.collect()
    for name, (ref, address) in held.items():
        assert ref() is not None and any(getattr(args, f) == address for f, _ in args._fields_), name
    del args
    gc.collect()
    assert all(ref() is None for ref, _ in held.values())


def test_a_workspace_comes_from_the_call_s_stream(made, monkeypatch):  # noqa: F811
    class Library:
        def dsa_latent_attn_workspace(self, args):
            return 4096

        def dsa_latent_attn(self, args, ws, n, stream):
            self.seen = (n, stream)
            return 0

    library = Library()
    monkeypatch.setattr(B, "load", lambda: library)
    args = B.LatentAttnArgs()
    args.device = torch.device("cuda", 0)
    B.dsa_latent_attn(args, stream=SIDE)
    assert made == [SIDE] and library.seen == (4096, 7)
    B.dsa_latent_attn(args)
    assert made == [SIDE, None] and library.seen == (4096, 3)


@pytest.mark.parametrize("call", [
    lambda t: B.dsa_add_rmsnorm(t, t, 1e-6, y=t), lambda t: B.latent_attn_args(1, 1, 1, 1, 1.0, t, t, t, t),
    lambda t: B.dsa_step_maps(t, t, t, t, 64, t, t, t, t, t, t)])
def test_tensors_that_are_not_on_a_gpu(call):
    with pytest.raises(B.DSAError, match="not a CUDA tensor"):
        call(torch.zeros(4, dtype=torch.int32))
