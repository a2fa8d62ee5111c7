"""Buffers that take tensors of other kernels refuse those whose rows, type or layout
the kernels would misread (no GPU: nothing is launched)."""
import numpy as np
import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B
from sparse_attention_prolog_gb300 import workloads as W
from sparse_attention_prolog_gb300.pipeline import DenseBuffers, MlaBuffers, StepMaps

T, D = 6, 512


@pytest.fixture()
def mla(monkeypatch):
    monkeypatch.setattr(B, "workspace_bytes", lambda kind, args: 256)
    return W.make_mla_inputs(T, np.zeros(T), np.zeros(T), 1, H=2, K_q=256, D_x=D, max_pos=64)


def tensors():
    return {"x": torch.zeros(T, D, dtype=torch.bfloat16), "pos": torch.zeros(T, dtype=torch.int32),
            "slot": torch.zeros(T, dtype=torch.int64)}


def test_the_mla_prolog_takes_rows_of_its_batch(mla):
    given = tensors()
    buf = MlaBuffers(mla, "cpu", 64, **given)
    assert buf.x is given["x"] and buf.pos is given["pos"] and buf.slot is given["slot"]
    MlaBuffers(mla, "cpu", 64)


@pytest.mark.parametrize("name,wrong", [
    ("x", lambda t: t[:-1]), ("x", lambda t: t.float()), ("x", lambda t: t.half()), ("x", lambda t: t[:, :-64]),
    ("x", lambda t: torch.zeros(T, 2 * D, dtype=t.dtype)[:, ::2]), ("x", lambda t: t.to("meta")),
    ("pos", lambda t: t[:-1]), ("pos", lambda t: torch.zeros(T + 1, dtype=t.dtype)), ("pos", lambda t: t.long()),
    ("pos", lambda t: torch.zeros(2 * T, dtype=t.dtype)[::2]),
    ("slot", lambda t: t[:-1]), ("slot", lambda t: t.int()), ("slot", lambda t: t.view(T, 1)),
])
def test_the_mla_prolog_refuses(mla, name, wrong):
    given = tensors()
    given[name] = wrong(given[name])
    with pytest.raises(B.DSAError, match=name):
        MlaBuffers(mla, "cpu", 64, **given)


@pytest.mark.parametrize("rows", [T - 1, T + 1])
def test_a_dense_step_refuses_maps_of_another_batch(mla, rows):
    maps = StepMaps(2, rows, 16, 4, torch.arange(8, dtype=torch.int32))
    with pytest.raises(B.DSAError, match="pos"):
        DenseBuffers(mla, maps, torch.zeros(128, 576, dtype=torch.bfloat16), torch.ones(D), 0.1)
