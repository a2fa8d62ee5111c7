"""An argument block keeps the tensors whose addresses it holds: one that was built
for it alone (a cast, a contiguous copy) would be freed before the call, and its
memory given to the workspace."""
import gc
import weakref

import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B


def _tensors(names, shape):
    return {n: torch.zeros(shape) for n in names}


def _prolog():
    t = _tensors("q_lora q_lora_scale w_qb w_qb_scale x w_k ln_gamma ln_beta w_proj pos rope_cos rope_sin q_out "
                 "q_scale_out k_cache k_scale_cache slot w_out".split(), (2, 4))
    return t, B.prolog_args(T=2, H_I=1, d_I=4, d_rope=2, ln_eps=1e-6, w_scale=1.0, rope_interleaved=0, **t)


def _topk():
    t = _tensors("q q_scale w k_cache k_scale pos topk_idx block_table scores_out seq_of_token".split(), (2, 4))
    return t, B.topk_args(T=2, B=1, n_q=2, H_I=1, d_I=4, topk=4, max_L=16, block_size=4, **t)


def _attn():
    t = _tensors("q kv topk_idx out lse block_table sink seq_of_token".split(), (2, 4))
    return t, B.attn_args(T=2, B=1, n_q=2, H=1, topk=4, max_L=16, scale=1.0, block_size=4, **t)


def _mla():
    t = _tensors("x w_dq gamma_q w_dkv gamma_kv w_uq w_uq_scale w_uk pos rope_cos rope_sin q_lora q_lora_scale q "
                 "kv_cache slot".split(), (2, 4))
    return t, B.mla_args(rms_eps=1e-6, rope_interleaved=0, **t)


def _attn_kv4():
    t = _tensors("q kv4 topk_idx out lse block_table sink seq_of_token".split(), (2, 4))
    return t, B.attn_kv4_args(T=2, B=1, n_q=2, H=1, topk=4, max_L=16, scale=1.0, block_size=4, **t)


@pytest.mark.parametrize("make", [_prolog, _topk, _attn, _mla, _attn_kv4])
def test_an_argument_block_keeps_its_tensors(make, monkeypatch):
    monkeypatch.setattr(B, "_device", lambda name, t: 0)
    monkeypatch.setattr(B, "_tensor", lambda *a, **k: None)
    tensors, args = make()
    held = {n: (weakref.ref(t), t.data_ptr()) for n, t in tensors.items()}
    del tensors
    gc.collect()
    for name, (ref, address) in held.items():
        assert ref() is not None, name
        assert any(getattr(args, f) == address for f, _ in args._fields_), name
    del args
    gc.collect()
    assert all(ref() is None for ref, _ in held.values())
