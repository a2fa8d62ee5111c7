"""Two host threads that call one kernel for different amounts of shared memory: the
calls go to the library one behind another, and none may be refused.  (Results of
such calls are the other tests' business; these check one pass of each.)"""
import ctypes

import numpy as np
import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B
from sparse_attention_prolog_gb300 import workloads as W
from sparse_attention_prolog_gb300.pipeline import DecodeBuffers, MlaBuffers, PrologBuffers
from test_gpu_threads import at_once

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def prolog(lib, K_q, D_x):
    p = W.make_prolog_inputs(T=2, pos=np.array([3, 4]), slot=np.array([0, 1]), seed=3, H_I=4, d_I=64, K_q=K_q, D_x=D_x,
                             max_pos=256)
    buf = PrologBuffers(p, DEV)
    return buf, lib.dsa_indexer_prolog, buf.args, buf.ws, lambda: buf.q_out


def scores(lib, T, H_I):
    inp = W.make_decode_inputs(B=T, n_q=1, seq_lens=[200] * T, H_I=H_I, d_I=64, topk=16, H=4, seed=1, max_L=256)
    buf = DecodeBuffers(inp, DEV, with_attention=False, seq_map=True, keep_scores=True)
    return buf, lib.dsa_indexer_topk, buf.targs, buf.tws, lambda: buf.scores[:, :200]


def mla(lib, K_q, D_x):
    p = W.make_mla_inputs(2, np.zeros(2), np.arange(2), 3, H=2, K_q=K_q, D_x=D_x, max_pos=64)
    buf = MlaBuffers(p, DEV, 16)
    return buf, lib.dsa_mla_prolog, buf.args, buf.ws, lambda: buf.q


def quant(lib, N, _):
    x = torch.randn(1, N, device=DEV).bfloat16()
    y, s = torch.zeros(1, N, dtype=torch.int8, device=DEV), torch.zeros(1, device=DEV)
    args = B.ActQuantArgs(1, N, B._p(x), B._p(y), B._p(s), 0)
    return (x, y, s), lambda a, ws, n, stream: lib.dsa_act_quant(a, stream), args, None, lambda: y


@pytest.mark.parametrize("make,sizes", [(prolog, [(2048, 4096), (128, 512)]), (scores, [(300, 8), (2, 8)]),
                                        (mla, [(2048, 512), (128, 512)]), (quant, [(32768, 0), (25000, 0)])])
def test_no_call_is_refused(make, sizes, cuda_lib):
    calls = [make(cuda_lib, *size) for size in sizes]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for (_, fn, args, ws, _), s in zip(calls, streams):
        assert fn(ctypes.byref(args), B._p(ws), 0 if ws is None else ws.numel(), s.cuda_stream) == 0
    torch.cuda.synchronize()
    first = [out().clone() for *_, out in calls]
    refused = [0] * len(calls)

    def loop(i):
        _, fn, args, ws, _ = calls[i]
        call = ctypes.byref(args), B._p(ws), 0 if ws is None else ws.numel(), streams[i].cuda_stream

        def go():
            for _ in range(4000):
                refused[i] += fn(*call) != 0
        return go

    assert not at_once(*[loop(i) for i in range(len(calls))])
    torch.cuda.synchronize()
    assert refused == [0] * len(calls)
    assert B.device_error() == 0
    for (*_, out), want in zip(calls, first):
        assert torch.equal(out(), want)
