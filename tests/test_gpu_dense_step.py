"""Decode steps of a layer without an indexer, stage by stage against the oracle and
plain loops: step maps -> residual and RMS norm -> MLA Prolog -> attention over the
whole latent cache, over steps in which requests begin, idle and grow past pages,
eagerly and from a graph.

Each stage is fed the CUDA path's own inputs; the bounds are those of the stages'
own tests (the norm's y within 2^-8 + 2^-18 of itself, the MLA Prolog's query and
rows within 8e-3 |ref| + 2e-3, the attention as in test_gpu_latent)."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle as O
from parity_utils import check_codes
from sparse_attention_prolog_gb300 import binding as B
from sparse_attention_prolog_gb300 import workloads as W
from sparse_attention_prolog_gb300.pipeline import DenseBuffers, StepMaps
from test_gpu_latent import Case
from test_gpu_mla import _bf16, _close

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 192.0 ** -0.5


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Steps:
    """Requests of a small model; what the host expects of the maps."""

    def __init__(self, n_req, T, H, bs, blocks, seed):
        rng = np.random.default_rng(seed)
        self.rng, self.n, self.T, self.H, self.bs, self.blocks = rng, n_req, T, H, bs, blocks
        self.p = W.make_mla_inputs(T, np.zeros(T), np.zeros(T), seed, H=H, K_q=256, D_x=512, max_pos=bs * blocks)
        pages = n_req * blocks
        self.free = rng.permutation(pages).astype(np.int32)
        self.maps = StepMaps(n_req, T, bs, blocks, torch.from_numpy(self.free).to(DEV))
        self.cache = torch.full((pages * bs, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.gamma = torch.from_numpy((1 + 0.1 * rng.standard_normal(512)).astype(np.float32)).to(DEV)
        self.buf = DenseBuffers(self.p, self.maps, self.cache, self.gamma, SCALE)
        self.lens, self.head = np.zeros(n_req, dtype=int), 0
        self.table = np.full((n_req, blocks), -1)

    def inputs(self):
        self.x = torch.from_numpy(self.rng.standard_normal((self.T, 512)).astype(np.float32)).to(DEV).bfloat16()
        self.res = torch.from_numpy(self.rng.standard_normal((self.T, 512)).astype(np.float32) * 2).to(DEV).bfloat16()
        self.buf.x.copy_(self.x)
        self.buf.residual.copy_(self.res)
        self.buf.out.fill_(7.0)
        self.buf.lse.fill_(7.0)

    def advance(self, fresh):
        """The host's view of a step: (sequence, position, row) of each token."""
        tokens = []
        for b, f in enumerate(fresh):
            for pos in range(self.lens[b], self.lens[b] + f):
                if pos % self.bs == 0:
                    self.table[b, pos // self.bs] = self.free[self.head]
                    self.head += 1
                tokens.append((b, pos, self.table[b, pos // self.bs] * self.bs + pos % self.bs))
            self.lens[b] += f
        return tokens

    def check(self, fresh, tokens):
        torch.cuda.synchronize()
        assert B.device_error() == 0
        m, buf, n = self.maps, self.buf, len(tokens)
        assert m.kv_len.tolist() == self.lens.tolist() and np.array_equal(m.block_table.cpu().numpy(), self.table)
        got = zip(m.seq_of_token.tolist(), m.pos.tolist(), m.slot.tolist())
        assert [tuple(t) for t in got][:n] == tokens and m.slot.tolist()[n:] == [-1] * (self.T - n)
        h = (self.x.float() + self.res.float()).bfloat16()
        assert torch.equal(buf.residual, h)
        z = h.double()
        z = z / (z.square().mean(1, keepdim=True) + 1e-6).sqrt() * self.gamma.double()
        assert bool(((buf.mla.x.double() - z).abs() <= z.abs() * (2.0 ** -8 + 2.0 ** -18) + 2.0 ** -133).all())
        pos, slot = m.pos.cpu().numpy(), m.slot.cpu().numpy()
        p = dataclasses.replace(self.p, x=_bits(buf.mla.x), pos=pos, slot=slot)
        ref = O.mla_prolog(p)
        lora, scale = buf.mla.q_lora.cpu().numpy(), buf.mla.q_lora_scale.cpu().numpy()
        check_codes(lora, scale, ref["q_lora"], ref["q_lora_scale"], "q_lora")
        _close(_bf16(buf.mla.q), O.mla_q(lora, scale, p.w_uq, p.w_uq_scale, O.bf16_bits_to_f64(p.w_uk), p.H, p.pos,
                                        p.rope_cos, p.rope_sin, bool(p.rope_interleaved)), "q")
        kv = _bf16(self.cache)
        for t, (_, _, row) in enumerate(tokens):
            _close(kv[row], ref["kv"][t], f"row of token {t}")
        c = Case(fresh, self.lens.tolist(), self.H, self.bs, pad=self.T - n)  # holds the check; its data are replaced
        c.q, c.kv, c.out, c.lse, c.sink = buf.mla.q, self.cache, buf.out, buf.lse, None
        c.rows_of = [torch.tensor([self.table[b, s // self.bs] * self.bs + s % self.bs for s in range(k)],
                                  dtype=torch.long, device=DEV) for b, k in enumerate(self.lens)]
        c.check()


@pytest.mark.parametrize("n_req,T,H,bs,blocks,seed", [(3, 8, 4, 64, 5, 1), (5, 32, 128, 16, 12, 2), (1, 1, 16, 8, 40, 3)])
def test_steps_in_a_row(n_req, T, H, bs, blocks, seed, cuda_lib):
    s = Steps(n_req, T, H, bs, blocks, seed)
    for step in range(6):
        left = np.minimum(s.bs * s.blocks - s.lens, T)
        fresh = s.rng.integers(0, np.minimum(left, T // n_req) + 1)
        if step == 0:
            fresh[0] = min(T // n_req, left[0])
        s.inputs()
        s.buf.run(torch.from_numpy(fresh.astype(np.int32)).to(DEV))
        s.check(fresh.tolist(), s.advance(fresh))


def test_two_steps_a_graph(cuda_lib):
    s = Steps(4, 12, 16, 16, 30, 4)
    fresh = [torch.zeros(4, dtype=torch.int32, device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for f in fresh:
            s.buf.run(f)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for f in fresh:
            s.buf.run(f)
    for _ in range(5):
        first, second = s.rng.integers(0, 4, 4), s.rng.integers(0, 4, 4)
        fresh[0].copy_(torch.from_numpy(first.astype(np.int32)))
        fresh[1].copy_(torch.from_numpy(second.astype(np.int32)))
        s.inputs()
        g.replay()
        # the second step adds x to the residual that the first left
        s.advance(first)
        s.res = (s.x.float() + s.res.float()).bfloat16()
        torch.cuda.synchronize()
        tokens = s.advance(second)
        n = len(tokens)
        # rows of out past this step's tokens are the first step's, or as they were
        s.buf.out[n:] = 7.0
        s.buf.lse[n:] = 7.0
        s.check(second.tolist(), tokens)
