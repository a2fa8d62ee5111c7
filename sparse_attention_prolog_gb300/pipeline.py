"""Device-side buffers and the decode step chain (prolog -> indexer/top-k ->
sparse attention) over the C ABI.  PyTorch provides device memory and
streams only; the computation is the library's."""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

from . import binding as B

INT16_VIEW = {"fp16": torch.float16, "bf16": torch.bfloat16}


def to_dev(a: np.ndarray, device, kind: str = None) -> torch.Tensor:
    """Uploads a numpy array; uint16 arrays holding fp16/bf16 bits become
    fp16/bf16 tensors with the same bits."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        t = torch.from_numpy(a.view(np.int16)).to(device)
        return t.view(INT16_VIEW[kind or "bf16"])
    if a.dtype == np.float16:
        return torch.from_numpy(a).to(device)
    return torch.from_numpy(a).to(device)


class PrologBuffers:
    """Device copies of a workloads.PrologInputs plus its outputs.  q_lora,
    q_lora_scale and x may be given as device tensors (another kernel's
    outputs or inputs, e.g. the MLA Prolog's)."""

    def __init__(self, p, device, k_cache: torch.Tensor = None, k_scale_cache: torch.Tensor = None,
                 q_lora: torch.Tensor = None, q_lora_scale: torch.Tensor = None, x: torch.Tensor = None):
        self.p = p
        d = device
        self.q_lora = to_dev(p.q_lora, d) if q_lora is None else q_lora
        self.q_lora_scale = to_dev(p.q_lora_scale, d) if q_lora_scale is None else q_lora_scale
        self.w_qb = to_dev(p.w_qb, d)
        self.w_qb_scale = to_dev(p.w_qb_scale, d)
        self.x = to_dev(p.x, d, "bf16") if x is None else x
        self.w_k = to_dev(p.w_k, d, "bf16")
        self.ln_gamma = to_dev(p.ln_gamma, d)
        self.ln_beta = to_dev(p.ln_beta, d)
        self.w_proj = None if p.w_proj is None else to_dev(p.w_proj, d, "bf16")
        self.pos = to_dev(p.pos, d)
        self.rope_cos = to_dev(p.rope_cos, d)
        self.rope_sin = to_dev(p.rope_sin, d)
        self.slot = to_dev(p.slot, d)
        T, H, D = p.T, p.H_I, p.d_I
        self.q_out = torch.zeros(T, H, D, dtype=torch.int8, device=d)
        self.q_scale_out = torch.zeros(T, H, dtype=torch.float16, device=d)
        rows = int(max(p.slot.max() + 1, 1)) if k_cache is None else k_cache.shape[0]
        self.k_cache = k_cache if k_cache is not None else torch.zeros(rows, D, dtype=torch.int8, device=d)
        self.k_scale_cache = (k_scale_cache if k_scale_cache is not None
                              else torch.zeros(rows, dtype=torch.float16, device=d))
        self.w_out = None if p.w_proj is None else torch.zeros(T, H, dtype=torch.float32, device=d)
        self.args = B.prolog_args(T, H, D, p.d_rope, self.q_lora, self.q_lora_scale, self.w_qb, self.w_qb_scale,
                                  self.x, self.w_k, self.ln_gamma, self.ln_beta, p.ln_eps, self.w_proj, p.w_scale,
                                  self.pos, self.rope_cos, self.rope_sin, p.rope_interleaved, self.q_out,
                                  self.q_scale_out, self.k_cache, self.k_scale_cache, self.slot, self.w_out)
        self.ws = torch.zeros(max(B.workspace_bytes("prolog", self.args), 256), dtype=torch.uint8, device=d)

    def run(self, stream=None):
        B.dsa_indexer_prolog(self.args, self.ws, stream)


class MlaBuffers:
    """Device copies of a workloads.MlaInputs plus the MLA Prolog's outputs
    (q_lora, q_lora_scale, q) and a latent cache of ``cache_rows`` rows.  x, pos
    and slot may be given as device tensors (another kernel's outputs): bf16 [T,
    D_x], int32 [T] and int64 [T]."""

    def __init__(self, p, device, cache_rows: int, kv_fill: float = 0.0, kv_cache: torch.Tensor = None,
                 x: torch.Tensor = None, pos: torch.Tensor = None, slot: torch.Tensor = None):
        self.p = p
        d = device
        self.w_dq = to_dev(p.w_dq, d, "bf16")
        for name, t, dtype, shape in (("x", x, torch.bfloat16, (p.T, p.D_x)), ("pos", pos, torch.int32, (p.T,)),
                                      ("slot", slot, torch.int64, (p.T,))):
            if t is not None and not (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                                      and t.device == self.w_dq.device):
                raise B.DSAError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}; expected "
                                 f"contiguous {dtype} {shape} on {self.w_dq.device}")
        self.x = to_dev(p.x, d, "bf16") if x is None else x
        self.gamma_q = to_dev(p.gamma_q, d)
        self.w_dkv = to_dev(p.w_dkv, d, "bf16")
        self.gamma_kv = to_dev(p.gamma_kv, d)
        self.w_uq = to_dev(p.w_uq, d)
        self.w_uq_scale = to_dev(p.w_uq_scale, d)
        self.w_uk = to_dev(p.w_uk, d, "bf16")
        self.pos = to_dev(p.pos, d) if pos is None else pos
        self.rope_cos = to_dev(p.rope_cos, d)
        self.rope_sin = to_dev(p.rope_sin, d)
        self.slot = to_dev(p.slot, d) if slot is None else slot
        self.q_lora = torch.zeros(p.T, p.K_q, dtype=torch.int8, device=d)
        self.q_lora_scale = torch.zeros(p.T, dtype=torch.float16, device=d)
        self.q = torch.zeros(p.T, p.H, 576, dtype=torch.bfloat16, device=d)
        self.kv_cache = (torch.full((cache_rows, 576), kv_fill, dtype=torch.bfloat16, device=d) if kv_cache is None
                         else kv_cache)
        self.args = B.mla_args(self.x, self.w_dq, self.gamma_q, self.w_dkv, self.gamma_kv, p.rms_eps, self.w_uq,
                               self.w_uq_scale, self.w_uk, self.pos, self.rope_cos, self.rope_sin,
                               p.rope_interleaved, self.q_lora, self.q_lora_scale, self.q, self.kv_cache, self.slot)
        self.ws = torch.zeros(max(B.workspace_bytes("mla", self.args), 256), dtype=torch.uint8, device=d)

    def run(self, stream=None):
        B.dsa_mla_prolog(self.args, self.ws, stream)


def is_uniform(inp) -> bool:
    """True if token t of the batch belongs to sequence t // n_q, n_q = T / B."""
    if inp.T % inp.B:
        return False
    return bool(np.array_equal(inp.seq_of_token, np.repeat(np.arange(inp.B, dtype=np.int32), inp.T // inp.B)))


class Kv4Cache:
    """A latent cache of ``rows`` rows held in 4 bits (416 bytes a row; all
    zeros at first) and the calls that write and read its rows by slot."""

    def __init__(self, rows: int, device):
        self.data = torch.zeros(rows, B.KV4_ROW_BYTES, dtype=torch.uint8, device=device)

    def write(self, x: torch.Tensor, slot: torch.Tensor, stream=None):
        """Quantises x bf16 [n, 576] into the rows slot int64 [n] (-1: skipped)."""
        B.dsa_kv4_write(x, self.data, slot, stream)

    def read(self, slot: torch.Tensor, out: torch.Tensor = None, stream=None) -> torch.Tensor:
        """The rows slot int64 [n] as bf16 [n, 576] (-1: zeros).  A new ``out`` is
        memory of ``stream``: another stream that uses it waits for this one, and
        records itself on it (``record_stream``) if it may be dropped before."""
        if out is None:
            with B.pool_of(stream):
                out = torch.empty(slot.shape[0], 576, dtype=torch.bfloat16, device=self.data.device)
        B.dsa_kv4_read(self.data, slot, out, stream)
        return out


class DecodeBuffers:
    """Device copies of a workloads.DecodeInputs and the indexer/attention
    outputs.  ``q_idx``/``q_idx_scale``/``w_idx`` may be replaced by the
    prolog's outputs (then pass them in).  The calls get the token map
    (seq_of_token) when the batch is not uniform, or when ``seq_map``.  With
    ``kv4`` (a Kv4Cache) the attention reads that 4-bit cache in place of
    ``kv``."""

    def __init__(self, inp, device, q_idx=None, q_idx_scale=None, w_idx=None, k_cache=None, k_scale=None,
                 with_attention=True, keep_scores=False, seq_map=False, q_attn=None, kv=None, kv4=None):
        self.inp = inp
        d = device
        self.q_idx = q_idx if q_idx is not None else to_dev(inp.q_idx, d)
        self.q_idx_scale = q_idx_scale if q_idx_scale is not None else to_dev(inp.q_idx_scale, d)
        self.w_idx = w_idx if w_idx is not None else to_dev(inp.w_idx, d)
        self.k_cache = k_cache if k_cache is not None else to_dev(inp.k_cache, d)
        self.k_scale = k_scale if k_scale is not None else to_dev(inp.k_scale, d)
        self.block_table = None if inp.block_table is None else to_dev(inp.block_table, d)
        self.pos = to_dev(inp.pos, d)
        T = inp.T
        self.seq = to_dev(inp.seq_of_token.astype(np.int32), d) if (seq_map or not is_uniform(inp)) else None
        n_q = max(T // inp.B, 1)
        self.topk_idx = torch.full((T, inp.topk), -7, dtype=torch.int32, device=d)
        self.scores = torch.empty(T, inp.max_L, dtype=torch.float32, device=d) if keep_scores else None
        self.targs = B.topk_args(T, inp.B, n_q, inp.H_I, inp.d_I, inp.topk, inp.max_L, self.q_idx,
                                 self.q_idx_scale, self.w_idx, self.k_cache, self.k_scale, self.pos, self.topk_idx,
                                 self.block_table, inp.block_size, self.scores, seq_of_token=self.seq)
        self.tws = torch.zeros(max(B.workspace_bytes("topk", self.targs), 256), dtype=torch.uint8, device=d)
        self.with_attention = with_attention
        if with_attention:
            self.q_attn = to_dev(inp.q_attn, d, "bf16") if q_attn is None else q_attn
            self.kv4 = kv4
            self.kv = None if kv4 is not None else to_dev(inp.kv_cache, d, "bf16") if kv is None else kv
            self.out = torch.zeros(T, inp.H, inp.d_v, dtype=torch.bfloat16, device=d)
            self.lse = torch.zeros(T, inp.H, dtype=torch.float32, device=d)
            if kv4 is not None:
                self.aargs = B.attn_kv4_args(T, inp.B, n_q, inp.H, inp.topk, inp.max_L, inp.scale, self.q_attn,
                                             kv4.data, self.topk_idx, self.out, self.lse, self.block_table,
                                             inp.block_size, seq_of_token=self.seq)
            else:
                self.aargs = B.attn_args(T, inp.B, n_q, inp.H, inp.topk, inp.max_L, inp.scale, self.q_attn,
                                         self.kv, self.topk_idx, self.out, self.lse, self.block_table,
                                         inp.block_size, seq_of_token=self.seq)
            need = B.workspace_bytes("attn" if kv4 is None else "attn_kv4", self.aargs)
            self.aws = torch.zeros(max(need, 256), dtype=torch.uint8, device=d)

    def run_topk(self, stream=None):
        B.dsa_indexer_topk(self.targs, self.tws, stream)

    def run_attn(self, stream=None):
        if self.kv4 is not None:
            B.dsa_sparse_attn_kv4(self.aargs, self.aws, stream)
        else:
            B.dsa_sparse_attn(self.aargs, self.aws, stream)

    def run(self, stream=None):
        self.run_topk(stream)
        if self.with_attention:
            self.run_attn(stream)


class DiaBuffers:
    """One decode step of DeepSeek Indexer Attention on the device: the MLA
    Prolog (query latent q_lora, attention query q, latent KV rows into the
    latent cache) -> the Indexer Prolog (fed the MLA Prolog's q_lora and the
    same hidden states x; new keys into the key cache) -> Lightning Indexer
    + top-k -> sparse attention (the MLA Prolog's q over the latent cache).
    `dia` is a workloads.DiaInputs.

    With ``kv4`` the latent cache is held in 4 bits (416 instead of 1152 bytes
    a row): the prior rows are quantised once here, the MLA Prolog leaves the
    step's rows in a [T, 576] buffer, dsa_kv4_write puts them into the cache and
    the attention is dsa_sparse_attn_kv4."""

    def __init__(self, dia, device, keep_scores=False, kv4=False):
        d = device
        inp = dia.decode
        self.dia = dia
        self.k_cache = to_dev(inp.k_cache, d)
        self.k_scale = to_dev(inp.k_scale, d)
        self.kv = to_dev(inp.kv_cache, d, "bf16")
        self.kv4 = None
        if kv4:
            self.kv4 = Kv4Cache(self.kv.shape[0], d)
            self.kv4.write(self.kv, torch.arange(self.kv.shape[0], dtype=torch.int64, device=d))
            self.slot = to_dev(dia.mla.slot, d)
            self.kv = torch.zeros(inp.T, 576, dtype=torch.bfloat16, device=d)
            mla = dataclasses.replace(dia.mla, slot=np.arange(inp.T, dtype=np.int64))
        else:
            mla = dia.mla
        self.mla = MlaBuffers(mla, d, self.kv.shape[0], kv_cache=self.kv)
        self.pro = PrologBuffers(dia.prolog, d, self.k_cache, self.k_scale, q_lora=self.mla.q_lora,
                                 q_lora_scale=self.mla.q_lora_scale, x=self.mla.x)
        self.buf = DecodeBuffers(inp, d, q_idx=self.pro.q_out, q_idx_scale=self.pro.q_scale_out, w_idx=self.pro.w_out,
                                 k_cache=self.k_cache, k_scale=self.k_scale, keep_scores=keep_scores,
                                 q_attn=self.mla.q, kv=self.kv, kv4=self.kv4)

    def run(self, stream=None):
        self.mla.run(stream)
        if self.kv4 is not None:
            self.kv4.write(self.kv, self.slot, stream)
        self.pro.run(stream)
        self.buf.run(stream)


class StepMaps:
    """The tables of the steps of ``B`` requests over a paged cache, kept on the
    device: a block table, a list of free pages and the lengths.  Each run()
    adds fresh int32 [B] tokens to the requests and leaves what the step's calls
    take: block_table, cu_tokens, kv_len, seq_of_token, pos and slot (T rows; see
    dsa_step_maps), counts (tokens, free pages taken so far, requests served).
    A step reads one set of lengths and writes the other, and sets its free head
    from its counts, so a captured run() has to be of an even number of steps.
    Steps only take pages.  Between two steps a caller ends a request b of k pages
    by writing them back in front of the head (h = counts[step][1]: free_pages[h -
    k:h] = block_table[b, :k], then h - k into its place) and 0 into kv_len[b]."""

    def __init__(self, B_: int, T: int, block_size: int, max_blocks: int, free_pages: torch.Tensor):
        d = free_pages.device
        i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device=d)  # noqa: E731
        self.block_size = block_size
        self.free_pages = free_pages
        self.block_table = torch.full((B_, max_blocks), -1, dtype=torch.int32, device=d)
        self.lens = [i32(B_), i32(B_)]
        self.counts = [i32(3), i32(3)]
        self.cu_tokens, self.seq_of_token, self.pos = i32(B_ + 1), i32(T), i32(T)
        self.slot = torch.zeros(T, dtype=torch.int64, device=d)
        self.step = 0  # which set the next run reads

    @property
    def kv_len(self) -> torch.Tensor:
        """The lengths after the latest step (a view that the next step keeps)."""
        return self.lens[self.step]

    def run(self, fresh: torch.Tensor, stream=None):
        now, then = self.step, 1 - self.step
        B.dsa_step_maps(self.lens[now], fresh, self.free_pages, self.block_table, self.block_size, self.cu_tokens,
                        self.lens[then], self.counts[then], self.seq_of_token, self.pos, self.slot,
                        free_head=self.counts[now][1:2], stream=stream)
        self.step = then


class DenseBuffers:
    """One decode step of a layer without an indexer: the residual addition and
    RMS norm of the hidden states (their output is the MLA Prolog's x) -> the MLA
    Prolog (positions and cache rows from the step maps) -> attention over the
    whole latent cache of each request.  ``p`` is a workloads.MlaInputs whose x,
    pos and slot are not used; T = p.T rows, of which a step may fill fewer (the
    maps' padding).  ``x`` and ``residual`` bf16 [T, D_x] are the step's inputs,
    ``residual`` is updated in place."""

    def __init__(self, p, maps: StepMaps, kv_cache: torch.Tensor, gamma: torch.Tensor, scale: float, eps: float = 1e-6):
        d = kv_cache.device
        self.maps, self.gamma, self.eps, self.scale, self.kv_cache = maps, gamma, eps, scale, kv_cache
        self.x = torch.zeros(p.T, p.D_x, dtype=torch.bfloat16, device=d)
        self.residual = torch.zeros_like(self.x)
        self.mla = MlaBuffers(p, d, kv_cache.shape[0], kv_cache=kv_cache, x=torch.zeros_like(self.x), pos=maps.pos,
                              slot=maps.slot)
        self.out = torch.zeros(p.T, p.H, 512, dtype=torch.bfloat16, device=d)
        self.lse = torch.zeros(p.T, p.H, dtype=torch.float32, device=d)
        B_, blocks = maps.block_table.shape
        self.aargs = [B.latent_attn_args(p.T, B_, p.H, blocks * maps.block_size, scale, self.mla.q, kv_cache, lens,
                                         self.out, self.lse, cu_tokens=maps.cu_tokens, block_table=maps.block_table,
                                         block_size=maps.block_size) for lens in maps.lens]
        self.aws = torch.empty(B.workspace_bytes("latent_attn", self.aargs[0]), dtype=torch.uint8, device=d)

    def run(self, fresh: torch.Tensor, stream=None):
        """fresh int32 [B]: the tokens that each request adds, in x's row order."""
        self.maps.run(fresh, stream)
        B.dsa_add_rmsnorm(self.x, self.gamma, self.eps, self.residual, self.residual, self.mla.x, stream=stream)
        self.mla.run(stream)
        B.dsa_latent_attn(self.aargs[self.maps.step], self.aws, stream)
