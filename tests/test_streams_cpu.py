"""Memory that a call makes for itself comes from the pool of the stream that its
kernels run on: a block that another stream freed may still be read or written
by work queued there.  (CPU: the library, the stream and the allocator are
stand-ins that note which stream is current when memory is asked for.)"""
import contextlib
import types

import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B
from sparse_attention_prolog_gb300 import pipeline

SIDE = types.SimpleNamespace(cuda_stream=7)


class Memory:
    """Stand-in for a device tensor."""

    shape, device = (4, 576), "cuda:0"

    def __init__(self, n):
        self.n = n

    def numel(self):
        return self.n

    def element_size(self):
        return 1

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, stream):
        pass


@pytest.fixture
def made(monkeypatch):
    """The streams that were current when memory was made, in order."""
    current, seen = [None], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s if s is not None else current[-1])
        yield
        current.pop()

    def empty(*size, **kw):
        seen.append(current[-1])
        return Memory(size[0] if isinstance(size[0], int) else size[0][0])

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 3, raising=False)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "zeros", empty)
    return seen


def _library(monkeypatch, **calls):
    monkeypatch.setattr(B, "load", lambda: types.SimpleNamespace(**calls))


@pytest.mark.parametrize("stream", [None, SIDE])
def test_workspace_of_the_4_bit_attention(stream, made, monkeypatch):
    _library(monkeypatch, dsa_sparse_attn_kv4_workspace=lambda a: 4096, dsa_sparse_attn_kv4=lambda *a: 0)
    args = B.AttnKv4Args()
    args.device = torch.device("cuda", 0)
    B.dsa_sparse_attn_kv4(args, stream=stream)
    assert made == [stream]


@pytest.mark.parametrize("stream", [None, SIDE])
def test_result_of_a_read(stream, made, monkeypatch):
    monkeypatch.setattr(B, "dsa_kv4_read", lambda *a: None)
    cache = pipeline.Kv4Cache(8, "cuda:0")
    made.clear()
    cache.read(Memory(4), stream=stream)
    assert made == [stream]
    cache.read(Memory(4), out=Memory(4), stream=stream)
    assert made == [stream]


@pytest.mark.parametrize("stream", [None, SIDE])
@pytest.mark.parametrize("name", ["dsa_indexer_prolog", "dsa_indexer_topk", "dsa_sparse_attn", "dsa_mla_prolog"])
def test_workspaces_that_have_to_be_clear(name, stream, made, monkeypatch):
    """(Made and cleared on the call's stream: the kernels come after the fill.)"""
    _library(monkeypatch, **{name + "_workspace": lambda a: 4096, name: lambda *a: 0})
    args = {"dsa_indexer_prolog": B.PrologArgs, "dsa_indexer_topk": B.TopkArgs, "dsa_sparse_attn": B.AttnArgs,
            "dsa_mla_prolog": B.MlaArgs}[name]()
    getattr(B, name)(args, stream=stream)
    assert made == [stream]
