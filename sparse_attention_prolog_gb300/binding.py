"""ctypes binding of libdsa.so: argument marshalling only.

Each wrapper takes torch CUDA tensors, fills the C argument struct with their
device pointers and calls the entry point of the same name; every step of
the computation runs in the library's kernels.  Loading fails loudly when the
library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsa.so")

c_int = ctypes.c_int32
c_ptr = ctypes.c_void_p


class PrologArgs(ctypes.Structure):
    _fields_ = [
        ("T", c_int), ("H_I", c_int), ("d_I", c_int), ("d_rope", c_int), ("K_q", c_int), ("D_x", c_int),
        ("q_lora", c_ptr), ("q_lora_scale", c_ptr), ("w_qb", c_ptr), ("w_qb_scale", c_ptr),
        ("x", c_ptr), ("w_k", c_ptr), ("ln_gamma", c_ptr), ("ln_beta", c_ptr), ("ln_eps", ctypes.c_float),
        ("w_proj", c_ptr), ("w_scale", ctypes.c_float), ("pos", c_ptr), ("rope_cos", c_ptr), ("rope_sin", c_ptr),
        ("rope_max_pos", c_int), ("rope_interleaved", c_int), ("q_out", c_ptr), ("q_scale_out", c_ptr),
        ("k_cache", c_ptr), ("k_scale_cache", c_ptr), ("slot", c_ptr), ("cache_rows", ctypes.c_int64),
        ("w_out", c_ptr),
    ]


class TopkArgs(ctypes.Structure):
    _fields_ = [
        ("T", c_int), ("B", c_int), ("n_q", c_int), ("H_I", c_int), ("d_I", c_int), ("topk", c_int), ("max_L", c_int),
        ("q", c_ptr), ("q_scale", c_ptr), ("w", c_ptr), ("k_cache", c_ptr), ("k_scale", c_ptr),
        ("block_table", c_ptr), ("block_size", c_int), ("max_blocks", c_int), ("pos", c_ptr),
        ("topk_idx", c_ptr), ("scores_out", c_ptr), ("seq_of_token", c_ptr),
    ]


class AttnArgs(ctypes.Structure):
    _fields_ = [
        ("T", c_int), ("B", c_int), ("n_q", c_int), ("H", c_int), ("d_qk", c_int), ("d_v", c_int), ("topk", c_int),
        ("max_L", c_int), ("scale", ctypes.c_float), ("q", c_ptr), ("kv", c_ptr), ("block_table", c_ptr),
        ("block_size", c_int), ("max_blocks", c_int), ("topk_idx", c_ptr), ("out", c_ptr), ("lse", c_ptr),
        ("sink", c_ptr), ("seq_of_token", c_ptr),
    ]


class ActQuantArgs(ctypes.Structure):
    _fields_ = [("M", c_int), ("N", c_int), ("x", c_ptr), ("y", c_ptr), ("scale", c_ptr), ("round_scale", c_int)]


class Int8GemmArgs(ctypes.Structure):
    _fields_ = [("M", c_int), ("N", c_int), ("K", c_int), ("a", c_ptr), ("a_scale", c_ptr), ("b", c_ptr),
                ("b_scale", c_ptr), ("c", c_ptr)]


class MhcArgs(ctypes.Structure):
    _fields_ = [("n", c_int), ("hc", c_int), ("iters", c_int), ("eps", ctypes.c_float), ("mixes", c_ptr),
                ("hc_scale", c_ptr), ("hc_base", c_ptr), ("pre", c_ptr), ("post", c_ptr), ("comb", c_ptr)]


class MlaArgs(ctypes.Structure):
    _fields_ = [("T", c_int), ("H", c_int), ("K_q", c_int), ("D_x", c_int), ("rms_eps", ctypes.c_float),
                ("rope_max_pos", c_int), ("rope_interleaved", c_int), ("x", c_ptr), ("w_dq", c_ptr),
                ("gamma_q", c_ptr), ("w_dkv", c_ptr), ("gamma_kv", c_ptr), ("w_uq", c_ptr), ("w_uq_scale", c_ptr),
                ("w_uk", c_ptr), ("pos", c_ptr), ("rope_cos", c_ptr), ("rope_sin", c_ptr), ("q_lora", c_ptr),
                ("q_lora_scale", c_ptr), ("q", c_ptr), ("kv_cache", c_ptr), ("slot", c_ptr),
                ("cache_rows", ctypes.c_int64)]


class Kv4WriteArgs(ctypes.Structure):
    _fields_ = [("n", c_int), ("x_stride", ctypes.c_int64), ("x", c_ptr), ("kv4", c_ptr), ("slot", c_ptr),
                ("cache_rows", ctypes.c_int64)]


class Kv4ReadArgs(ctypes.Structure):
    _fields_ = [("n", c_int), ("out_stride", ctypes.c_int64), ("kv4", c_ptr), ("slot", c_ptr),
                ("cache_rows", ctypes.c_int64), ("out", c_ptr)]


class AttnKv4Args(ctypes.Structure):
    _fields_ = [
        ("T", c_int), ("B", c_int), ("n_q", c_int), ("H", c_int), ("topk", c_int), ("max_L", c_int),
        ("scale", ctypes.c_float), ("q", c_ptr), ("kv4", c_ptr), ("cache_rows", ctypes.c_int64),
        ("block_table", c_ptr), ("block_size", c_int), ("max_blocks", c_int), ("topk_idx", c_ptr), ("out", c_ptr),
        ("lse", c_ptr), ("sink", c_ptr), ("seq_of_token", c_ptr),
    ]


class StepMapsArgs(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int), ("block_size", c_int), ("max_blocks", c_int), ("n_free", c_int),
                ("cached", c_ptr), ("fresh", c_ptr), ("free_pages", c_ptr), ("free_head", c_ptr),
                ("block_table", c_ptr), ("cu_tokens", c_ptr), ("kv_len", c_ptr), ("counts", c_ptr),
                ("seq_of_token", c_ptr), ("pos", c_ptr), ("slot", c_ptr)]


class LatentAttnArgs(ctypes.Structure):
    _fields_ = [("T", c_int), ("B", c_int), ("n_q", c_int), ("H", c_int), ("max_L", c_int), ("scale", ctypes.c_float),
                ("q", c_ptr), ("kv", c_ptr), ("cache_rows", ctypes.c_int64), ("block_table", c_ptr),
                ("block_size", c_int), ("max_blocks", c_int), ("cu_tokens", c_ptr), ("kv_len", c_ptr), ("out", c_ptr),
                ("lse", c_ptr), ("sink", c_ptr)]


class AddRmsnormArgs(ctypes.Structure):
    _fields_ = [("T", c_int), ("D", c_int), ("eps", ctypes.c_float), ("x_fp16", c_int), ("residual_fp32", c_int),
                ("round_scale", c_int), ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64),
                ("residual_out_stride", ctypes.c_int64), ("x", c_ptr), ("residual", c_ptr), ("residual_out", c_ptr),
                ("gamma", c_ptr), ("y", c_ptr), ("codes", c_ptr), ("code_scale", c_ptr)]


EXPORTS = [
    "dsa_status_string", "dsa_abi_version", "dsa_get_device_error", "dsa_set_wait_limit_ns",
    "dsa_indexer_prolog_workspace", "dsa_indexer_prolog",
    "dsa_indexer_topk_workspace", "dsa_indexer_topk", "dsa_indexer_dots_debug",
    "dsa_indexer_scores", "dsa_topk_from_scores",
    "dsa_sparse_attn_workspace", "dsa_sparse_attn", "dsa_indexer_prolog_noalloc", "dsa_act_quant",
    "dsa_int8_gemm", "dsa_mhc", "dsa_mla_prolog_workspace", "dsa_mla_prolog",
    "dsa_kv4_write", "dsa_kv4_read", "dsa_sparse_attn_kv4_workspace", "dsa_sparse_attn_kv4",
    "dsa_step_maps", "dsa_latent_attn_workspace", "dsa_latent_attn", "dsa_add_rmsnorm",
]

KV4_ROW_BYTES = 416  # one row of the 4-bit latent cache

_lib = None


class DSAError(RuntimeError):
    pass


def load(path: str = LIB_PATH):
    """Loads libdsa.so once; raises if it is missing (no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise DSAError(f"{path} is missing: build it with sparse_attention_prolog_gb300.build.build()")
    lib = ctypes.CDLL(path)
    lib.dsa_status_string.restype = ctypes.c_char_p
    lib.dsa_status_string.argtypes = [c_int]
    lib.dsa_abi_version.restype = c_int
    lib.dsa_get_device_error.argtypes = [c_ptr]
    lib.dsa_get_device_error.restype = c_int
    lib.dsa_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.dsa_set_wait_limit_ns.restype = c_int
    for name, st in (("prolog", PrologArgs), ("topk", TopkArgs), ("attn", AttnArgs)):
        ws = {"prolog": "dsa_indexer_prolog_workspace", "topk": "dsa_indexer_topk_workspace",
              "attn": "dsa_sparse_attn_workspace"}[name]
        run = {"prolog": "dsa_indexer_prolog", "topk": "dsa_indexer_topk", "attn": "dsa_sparse_attn"}[name]
        getattr(lib, ws).argtypes = [ctypes.POINTER(st)]
        getattr(lib, ws).restype = ctypes.c_size_t
        getattr(lib, run).argtypes = [ctypes.POINTER(st), c_ptr, ctypes.c_size_t, c_ptr]
        getattr(lib, run).restype = c_int
    lib.dsa_indexer_prolog_noalloc.argtypes = [ctypes.POINTER(PrologArgs), c_ptr]
    lib.dsa_indexer_prolog_noalloc.restype = c_int
    lib.dsa_indexer_dots_debug.argtypes = [ctypes.POINTER(TopkArgs), c_ptr, c_ptr]
    lib.dsa_indexer_dots_debug.restype = c_int
    lib.dsa_indexer_scores.argtypes = [ctypes.POINTER(TopkArgs), c_ptr, c_ptr]
    lib.dsa_indexer_scores.restype = c_int
    lib.dsa_topk_from_scores.argtypes = [ctypes.POINTER(TopkArgs), c_ptr, ctypes.c_int64, c_ptr]
    lib.dsa_topk_from_scores.restype = c_int
    lib.dsa_act_quant.argtypes = [ctypes.POINTER(ActQuantArgs), c_ptr]
    lib.dsa_act_quant.restype = c_int
    lib.dsa_int8_gemm.argtypes = [ctypes.POINTER(Int8GemmArgs), c_ptr]
    lib.dsa_int8_gemm.restype = c_int
    lib.dsa_mhc.argtypes = [ctypes.POINTER(MhcArgs), c_ptr]
    lib.dsa_mhc.restype = c_int
    lib.dsa_mla_prolog_workspace.argtypes = [ctypes.POINTER(MlaArgs)]
    lib.dsa_mla_prolog_workspace.restype = ctypes.c_size_t
    lib.dsa_mla_prolog.argtypes = [ctypes.POINTER(MlaArgs), c_ptr, ctypes.c_size_t, c_ptr]
    lib.dsa_mla_prolog.restype = c_int
    lib.dsa_kv4_write.argtypes = [ctypes.POINTER(Kv4WriteArgs), c_ptr]
    lib.dsa_kv4_write.restype = c_int
    lib.dsa_kv4_read.argtypes = [ctypes.POINTER(Kv4ReadArgs), c_ptr]
    lib.dsa_kv4_read.restype = c_int
    lib.dsa_sparse_attn_kv4_workspace.argtypes = [ctypes.POINTER(AttnKv4Args)]
    lib.dsa_sparse_attn_kv4_workspace.restype = ctypes.c_size_t
    lib.dsa_sparse_attn_kv4.argtypes = [ctypes.POINTER(AttnKv4Args), c_ptr, ctypes.c_size_t, c_ptr]
    lib.dsa_sparse_attn_kv4.restype = c_int
    lib.dsa_step_maps.argtypes = [ctypes.POINTER(StepMapsArgs), c_ptr]
    lib.dsa_step_maps.restype = c_int
    lib.dsa_latent_attn_workspace.argtypes = [ctypes.POINTER(LatentAttnArgs)]
    lib.dsa_latent_attn_workspace.restype = ctypes.c_size_t
    lib.dsa_latent_attn.argtypes = [ctypes.POINTER(LatentAttnArgs), c_ptr, ctypes.c_size_t, c_ptr]
    lib.dsa_latent_attn.restype = c_int
    lib.dsa_add_rmsnorm.argtypes = [ctypes.POINTER(AddRmsnormArgs), c_ptr]
    lib.dsa_add_rmsnorm.restype = c_int
    # the same entries for packed argument blocks
    for name in ("step_maps", "add_rmsnorm"):
        entry = lib["dsa_" + name]
        entry.restype, entry.argtypes = c_int, [c_ptr, c_ptr]
        setattr(lib, name + "_packed", entry)
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().dsa_status_string(code).decode()


def _check(code: int, what: str):
    if code != 0:
        raise DSAError(f"{what}: {status_string(code)} ({code})")


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _keep(args, *tensors):
    """args, holding on to the tensors whose addresses it has (a block may be built
    from temporaries)."""
    args.tensors = tensors
    return args


def _stream(stream=None):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    # (the Stream object of current_stream() costs 2.7 us a call, its handle 0.2)
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


_HERE = contextlib.nullcontext()


def pool_of(stream):
    """Context in which memory is made for a call on `stream` (None: the current
    one): of that stream's own pool, and filled on it.  A block that another stream
    freed may still be in use there, and its fill might come after the call."""
    return _HERE if stream is None else torch.cuda.stream(stream)  # (2.3 us even for None)


def _ws(nbytes: int, device, ws: Optional[torch.Tensor], stream):
    """A workspace for a call on `stream` and its size."""
    if nbytes == 0:
        return None, 0
    if ws is not None:
        assert ws.numel() * ws.element_size() >= nbytes
        return ws, ws.numel() * ws.element_size()
    with pool_of(stream):
        return torch.zeros(nbytes, dtype=torch.uint8, device=device), nbytes


# ---------------------------------------------------------------- prolog
def prolog_args(T, H_I, d_I, d_rope, q_lora, q_lora_scale, w_qb, w_qb_scale, x, w_k, ln_gamma, ln_beta,
                ln_eps, w_proj, w_scale, pos, rope_cos, rope_sin, rope_interleaved, q_out, q_scale_out,
                k_cache, k_scale_cache, slot, w_out) -> PrologArgs:
    return _keep(PrologArgs(
        T, H_I, d_I, d_rope, q_lora.shape[1] if T else 0, x.shape[1] if T else 0,
        _p(q_lora), _p(q_lora_scale), _p(w_qb), _p(w_qb_scale), _p(x), _p(w_k), _p(ln_gamma), _p(ln_beta),
        float(ln_eps), _p(w_proj), float(w_scale), _p(pos), _p(rope_cos), _p(rope_sin), rope_cos.shape[0],
        int(rope_interleaved), _p(q_out), _p(q_scale_out), _p(k_cache), _p(k_scale_cache), _p(slot),
        k_cache.shape[0], _p(w_out)), q_lora, q_lora_scale, w_qb, w_qb_scale, x, w_k, ln_gamma, ln_beta, w_proj, pos,
        rope_cos, rope_sin, q_out, q_scale_out, k_cache, k_scale_cache, slot, w_out)


def dsa_indexer_prolog(args: PrologArgs, workspace: Optional[torch.Tensor] = None, stream=None,
                       device=None):
    lib = load()
    need = lib.dsa_indexer_prolog_workspace(ctypes.byref(args))
    ws, n = _ws(need, device or "cuda", workspace, stream)
    _check(lib.dsa_indexer_prolog(ctypes.byref(args), _p(ws), n, _stream(stream)), "dsa_indexer_prolog")
    return ws


def dsa_indexer_prolog_noalloc(args: PrologArgs, stream=None):
    """The prolog without a workspace: its scratch is a fixed array inside the
    library, for callers that cannot allocate device memory."""
    _check(load().dsa_indexer_prolog_noalloc(ctypes.byref(args), _stream(stream)), "dsa_indexer_prolog_noalloc")


# ----------------------------------------------------------------- top-k
def topk_args(T, B, n_q, H_I, d_I, topk, max_L, q, q_scale, w, k_cache, k_scale, pos, topk_idx,
              block_table=None, block_size=0, scores_out=None, seq_of_token=None) -> TopkArgs:
    """seq_of_token: int32 [T] sequence of each token (then n_q is ignored), or
    None for the uniform batch T = B * n_q."""
    max_blocks = 0 if block_table is None else block_table.shape[1]
    return _keep(TopkArgs(T, B, n_q, H_I, d_I, topk, max_L, _p(q), _p(q_scale), _p(w), _p(k_cache), _p(k_scale),
                          _p(block_table), block_size, max_blocks, _p(pos), _p(topk_idx), _p(scores_out),
                          _p(seq_of_token)),
                 q, q_scale, w, k_cache, k_scale, block_table, pos, topk_idx, scores_out, seq_of_token)


def dsa_indexer_topk(args: TopkArgs, workspace: Optional[torch.Tensor] = None, stream=None, device=None):
    lib = load()
    need = lib.dsa_indexer_topk_workspace(ctypes.byref(args))
    ws, n = _ws(need, device or "cuda", workspace, stream)
    _check(lib.dsa_indexer_topk(ctypes.byref(args), _p(ws), n, _stream(stream)), "dsa_indexer_topk")
    return ws


def dsa_indexer_dots_debug(args: TopkArgs, dots: torch.Tensor, stream=None):
    _check(load().dsa_indexer_dots_debug(ctypes.byref(args), _p(dots), _stream(stream)), "dsa_indexer_dots_debug")


def dsa_indexer_scores(args: TopkArgs, scores: torch.Tensor, stream=None):
    _check(load().dsa_indexer_scores(ctypes.byref(args), _p(scores), _stream(stream)), "dsa_indexer_scores")


def dsa_topk_from_scores(args: TopkArgs, scores: torch.Tensor, stream=None):
    _check(load().dsa_topk_from_scores(ctypes.byref(args), _p(scores), scores.stride(0), _stream(stream)),
           "dsa_topk_from_scores")


# -------------------------------------------------------------- attention
def attn_args(T, B, n_q, H, topk, max_L, scale, q, kv, topk_idx, out, lse=None, block_table=None,
              block_size=0, d_qk=576, d_v=512, sink=None, seq_of_token=None) -> AttnArgs:
    max_blocks = 0 if block_table is None else block_table.shape[1]
    return _keep(AttnArgs(T, B, n_q, H, d_qk, d_v, topk, max_L, float(scale), _p(q), _p(kv), _p(block_table),
                          block_size, max_blocks, _p(topk_idx), _p(out), _p(lse), _p(sink), _p(seq_of_token)),
                 q, kv, block_table, topk_idx, out, lse, sink, seq_of_token)


def dsa_sparse_attn(args: AttnArgs, workspace: Optional[torch.Tensor] = None, stream=None, device=None):
    lib = load()
    need = lib.dsa_sparse_attn_workspace(ctypes.byref(args))
    ws, n = _ws(need, device or "cuda", workspace, stream)
    _check(lib.dsa_sparse_attn(ctypes.byref(args), _p(ws), n, _stream(stream)), "dsa_sparse_attn")
    return ws


def workspace_bytes(kind: str, args) -> int:
    lib = load()
    fn = {"prolog": lib.dsa_indexer_prolog_workspace, "topk": lib.dsa_indexer_topk_workspace,
          "attn": lib.dsa_sparse_attn_workspace, "mla": lib.dsa_mla_prolog_workspace,
          "attn_kv4": lib.dsa_sparse_attn_kv4_workspace, "latent_attn": lib.dsa_latent_attn_workspace}[kind]
    return int(fn(ctypes.byref(args)))


def device_error(stream=None) -> int:
    return int(load().dsa_get_device_error(_stream(stream)))


def set_wait_limit_ns(ns: int):
    """Time limit of the library's bounded device waits on the current device
    (0 restores the default)."""
    _check(load().dsa_set_wait_limit_ns(int(ns)), "dsa_set_wait_limit_ns")


def dsa_act_quant(x: torch.Tensor, y: torch.Tensor, scale: torch.Tensor, round_scale: bool = False, stream=None):
    """x bf16 [M, N] -> y int8 [M, N], scale fp32 [M] (see dsa.h)."""
    M, N = x.shape
    args = ActQuantArgs(M, N, _p(x), _p(y), _p(scale), int(bool(round_scale)))
    _check(load().dsa_act_quant(ctypes.byref(args), _stream(stream)), "dsa_act_quant")


def dsa_int8_gemm(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                  c: torch.Tensor, stream=None):
    """a int8 [M, K], b int8 [N, K], fp32 scales -> c fp16 [M, N] (see dsa.h)."""
    M, K = a.shape
    N = b.shape[0]
    args = Int8GemmArgs(M, N, K, _p(a), _p(a_scale), _p(b), _p(b_scale), _p(c))
    _check(load().dsa_int8_gemm(ctypes.byref(args), _stream(stream)), "dsa_int8_gemm")


def dsa_mhc(mixes: torch.Tensor, hc_scale: torch.Tensor, hc_base: torch.Tensor, hc: int, iters: int, eps: float,
            pre: torch.Tensor, post: torch.Tensor, comb: torch.Tensor, stream=None):
    """mixes fp32 [n, hc (2 + hc)] -> pre [n, hc], post [n, hc], comb [n, hc, hc] (see dsa.h)."""
    args = MhcArgs(mixes.shape[0], hc, iters, float(eps), _p(mixes), _p(hc_scale), _p(hc_base), _p(pre), _p(post),
                   _p(comb))
    _check(load().dsa_mhc(ctypes.byref(args), _stream(stream)), "dsa_mhc")


# ------------------------------------------------------------ MLA Prolog
def mla_args(x, w_dq, gamma_q, w_dkv, gamma_kv, rms_eps, w_uq, w_uq_scale, w_uk, pos, rope_cos, rope_sin,
             rope_interleaved, q_lora, q_lora_scale, q, kv_cache, slot) -> MlaArgs:
    """x bf16 [T, D_x], w_dq bf16 [K_q, D_x], w_dkv bf16 [576, D_x], w_uq int8 [H*192, K_q], w_uk bf16
    [H, 128, 512]; outputs q_lora int8 [T, K_q], q_lora_scale fp16 [T], q bf16 [T, H, 576] and the
    kv_cache bf16 [rows, 576] rows at slot (see dsa.h)."""
    T, D_x = x.shape
    return _keep(MlaArgs(T, w_uk.shape[0], w_dq.shape[0], D_x, float(rms_eps), rope_cos.shape[0],
                         int(rope_interleaved), _p(x), _p(w_dq), _p(gamma_q), _p(w_dkv), _p(gamma_kv), _p(w_uq),
                         _p(w_uq_scale), _p(w_uk), _p(pos), _p(rope_cos), _p(rope_sin), _p(q_lora), _p(q_lora_scale),
                         _p(q), _p(kv_cache), _p(slot), kv_cache.shape[0]),
                 x, w_dq, gamma_q, w_dkv, gamma_kv, w_uq, w_uq_scale, w_uk, pos, rope_cos, rope_sin, q_lora,
                 q_lora_scale, q, kv_cache, slot)


def dsa_mla_prolog(args: MlaArgs, workspace: Optional[torch.Tensor] = None, stream=None, device=None):
    """Runs the MLA Prolog; a new workspace is zero-filled, a given one must
    have been zero-filled before its first use.  Returns the workspace."""
    lib = load()
    need = lib.dsa_mla_prolog_workspace(ctypes.byref(args))
    ws, n = _ws(need, device or "cuda", workspace, stream)
    _check(lib.dsa_mla_prolog(ctypes.byref(args), _p(ws), n, _stream(stream)), "dsa_mla_prolog")
    return ws


# ----------------------------------------------------- 4-bit latent cache
def _device(name: str, t: torch.Tensor) -> int:
    """The current device, which has to be the one of t."""
    device = t.get_device()
    if device < 0:
        raise DSAError(f"{name}: not a CUDA tensor")
    if device != torch.cuda.current_device():
        raise DSAError(f"{name}: on {t.device}, which is not the current device")
    return device


def _tensor(name: str, t: torch.Tensor, dtype, shape, device: int, last_dense=False):
    """Refuses a tensor whose device, type, shape or layout the library would
    misread (None in a shape matches any size)."""
    if t.get_device() != device:  # (-1 for one that is not a CUDA tensor)
        raise DSAError(f"{name}: on {t.device}, which is not the current device")
    if t.dtype is not dtype:
        raise DSAError(f"{name}: {t.dtype}, expected {dtype}")
    if t.shape != shape and (t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape))):
        raise DSAError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous() and not (last_dense and (t.stride(-1) == 1 or t.shape[-1] <= 1)):
        raise DSAError(f"{name}: strides {t.stride()} are not supported")


def _kv4_rows(name: str, t: torch.Tensor, kv4: torch.Tensor, slot: torch.Tensor):
    """Checks rows t bf16 [n, 576], the cache and the slots: (device, n, row
    stride of t, rows of the cache).  (One condition for the calls that pass, as a
    check of each tensor costs as much as a launch.)"""
    device = _device("slot", slot)
    shape, cache = t.shape, kv4.shape
    if not (t.dtype is torch.bfloat16 and kv4.dtype is torch.uint8 and slot.dtype is torch.int64
            and len(shape) == 2 and shape[1] == 576 and slot.shape == shape[:1]
            and len(cache) == 2 and cache[1] == KV4_ROW_BYTES
            and t.get_device() == device and kv4.get_device() == device
            and t.stride(1) == 1 and kv4.is_contiguous() and slot.is_contiguous()):
        _tensor("slot", slot, torch.int64, (None,), device)
        _tensor(name, t, torch.bfloat16, (slot.shape[0], 576), device, last_dense=True)
        _tensor("kv4", kv4, torch.uint8, (None, KV4_ROW_BYTES), device)
    n = shape[0]
    # (a single row has no stride of its own)
    return device, n, t.stride(0) if n > 1 else max(576, t.stride(0) // 8 * 8), cache[0]


def _stream_of(device: int, stream):
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def dsa_kv4_write(x: torch.Tensor, kv4: torch.Tensor, slot: torch.Tensor, stream=None):
    """Quantises latent rows x bf16 [n, 576] (rows 16-byte aligned, a multiple of 8
    elements apart) into rows `slot` int64 [n] of the 4-bit cache kv4 uint8
    [rows, 416] (see dsa.h)."""
    device, n, stride, rows = _kv4_rows("x", x, kv4, slot)
    args = Kv4WriteArgs(n, stride, x.data_ptr(), kv4.data_ptr(), slot.data_ptr(), rows)
    _check(load().dsa_kv4_write(ctypes.byref(args), _stream_of(device, stream)), "dsa_kv4_write")


def dsa_kv4_read(kv4: torch.Tensor, slot: torch.Tensor, out: torch.Tensor, stream=None):
    """Rows `slot` int64 [n] of the 4-bit cache kv4 uint8 [rows, 416] -> out
    bf16 [n, 576] (rows 16-byte aligned, a multiple of 8 elements apart; see dsa.h)."""
    device, n, stride, rows = _kv4_rows("out", out, kv4, slot)
    args = Kv4ReadArgs(n, stride, kv4.data_ptr(), slot.data_ptr(), rows, out.data_ptr())
    _check(load().dsa_kv4_read(ctypes.byref(args), _stream_of(device, stream)), "dsa_kv4_read")


def attn_kv4_args(T, B, n_q, H, topk, max_L, scale, q, kv4, topk_idx, out, lse=None, block_table=None, block_size=0,
                  sink=None, seq_of_token=None) -> AttnKv4Args:
    """Arguments of dsa_sparse_attn_kv4: q bf16 [T, H, 576], kv4 uint8 [rows, 416], topk_idx int32 [T, topk], out
    bf16 [T, H, 512], lse fp32 [T, H]; block_table int32 [B, max_blocks] for a paged cache; sink fp32 [H];
    seq_of_token int32 [T] (then n_q is ignored)."""
    for name, v in (("T", T), ("B", B), ("n_q", n_q), ("H", H), ("topk", topk), ("max_L", max_L),
                    ("block_size", block_size)):
        if not -2 ** 31 <= v < 2 ** 31:  # (the C int would take its lower 32 bits)
            raise DSAError(f"{name}: {v} does not fit 32 bits")
    device = _device("q", q)
    _tensor("q", q, torch.bfloat16, (T, H, 576), device)
    _tensor("kv4", kv4, torch.uint8, (None, KV4_ROW_BYTES), device)
    _tensor("topk_idx", topk_idx, torch.int32, (T, topk), device)
    _tensor("out", out, torch.bfloat16, (T, H, 512), device)
    max_blocks = 0
    if block_table is not None:
        _tensor("block_table", block_table, torch.int32, (B, None), device)
        max_blocks = block_table.shape[1]
    if lse is not None:
        _tensor("lse", lse, torch.float32, (T, H), device)
    if sink is not None:
        _tensor("sink", sink, torch.float32, (H,), device)
    if seq_of_token is not None:
        _tensor("seq_of_token", seq_of_token, torch.int32, (T,), device)
    args = AttnKv4Args(T, B, n_q, H, topk, max_L, float(scale), _p(q), _p(kv4), kv4.shape[0], _p(block_table),
                       block_size, max_blocks, _p(topk_idx), _p(out), _p(lse), _p(sink), _p(seq_of_token))
    args.device = q.device
    return _keep(args, q, kv4, block_table, topk_idx, out, lse, sink, seq_of_token)


def _run_on(args, fn, size, what: str, workspace, stream):
    """Calls fn with args, the workspace (one of the stream's own is made when none
    is given and the shape needs one) and the stream.  Returns the workspace."""
    if torch.cuda.current_device() != args.device.index:
        raise DSAError(f"{what}: tensors on {args.device}, which is not the current device")
    if workspace is None:
        n = size(ctypes.byref(args))
        if n:
            with pool_of(stream):
                workspace = torch.empty(n, dtype=torch.uint8, device=args.device)
    else:
        n = workspace.numel() * workspace.element_size()
        if workspace.get_device() != args.device.index or not workspace.is_contiguous():
            raise DSAError(f"{what}: the workspace is not contiguous on the tensors' device")
    _check(fn(ctypes.byref(args), _p(workspace), n, _stream_of(args.device.index, stream)), what)
    return workspace


def dsa_sparse_attn_kv4(args: AttnKv4Args, workspace: Optional[torch.Tensor] = None, stream=None):
    """Runs the sparse attention over a 4-bit cache.  Returns the workspace
    (one of the stream's own is made when none is given and the shape needs
    one)."""
    lib = load()
    return _run_on(args, lib.dsa_sparse_attn_kv4, lib.dsa_sparse_attn_kv4_workspace, "dsa_sparse_attn_kv4", workspace,
                   stream)


# ------------------------------------------------------- latent attention
def _fits_32(**sizes):
    for name, v in sizes.items():
        if not -2 ** 31 <= v < 2 ** 31:  # (the C int would take its lower 32 bits)
            raise DSAError(f"{name}: {v} does not fit 32 bits")


def latent_attn_args(T, B, H, max_L, scale, q, kv, kv_len, out, lse=None, cu_tokens=None, n_q=0, block_table=None,
                     block_size=0, sink=None) -> LatentAttnArgs:
    """Arguments of dsa_latent_attn: q bf16 [T, H, 576], kv bf16 [rows, 576], kv_len int32 [B], out bf16 [T, H, 512],
    lse fp32 [T, H]; cu_tokens int32 [B + 1], or None for n_q tokens of each sequence; block_table int32
    [B, max_blocks] for a paged cache (max_L = max_blocks * block_size); sink fp32 [H] (see dsa.h)."""
    _fits_32(T=T, B=B, H=H, max_L=max_L, n_q=n_q, block_size=block_size)
    device = _device("q", q)
    _tensor("q", q, torch.bfloat16, (T, H, 576), device)
    _tensor("kv", kv, torch.bfloat16, (None, 576), device)
    _tensor("kv_len", kv_len, torch.int32, (B,), device)
    _tensor("out", out, torch.bfloat16, (T, H, 512), device)
    max_blocks = 0
    if block_table is not None:
        _tensor("block_table", block_table, torch.int32, (B, None), device)
        max_blocks = block_table.shape[1]
    if lse is not None:
        _tensor("lse", lse, torch.float32, (T, H), device)
    if sink is not None:
        _tensor("sink", sink, torch.float32, (H,), device)
    if cu_tokens is not None:
        _tensor("cu_tokens", cu_tokens, torch.int32, (B + 1,), device)
    args = LatentAttnArgs(T, B, n_q, H, max_L, float(scale), _p(q), _p(kv), kv.shape[0], _p(block_table), block_size,
                          max_blocks, _p(cu_tokens), _p(kv_len), _p(out), _p(lse), _p(sink))
    args.device = q.device
    return _keep(args, q, kv, kv_len, out, lse, cu_tokens, block_table, sink)


def dsa_latent_attn(args: LatentAttnArgs, workspace: Optional[torch.Tensor] = None, stream=None):
    """Runs the attention over the whole latent cache.  Returns the workspace
    (one of the stream's own is made when none is given)."""
    lib = load()
    return _run_on(args, lib.dsa_latent_attn, lib.dsa_latent_attn_workspace, "dsa_latent_attn", workspace, stream)


# --------------------------------------------------------------- step maps
# The argument blocks of calls that are made as often as launches, packed (a ctypes struct costs 0.4 us more).
_STEP_MAPS = struct.Struct("5i4x11P")       # StepMapsArgs
_ADD_RMSNORM = struct.Struct("2if3i3q7P")   # AddRmsnormArgs


def _unpackable(e) -> DSAError:
    return DSAError(f"arguments: {e}")  # a size past 32 bits, a number that is none


def dsa_step_maps(cached: torch.Tensor, fresh: torch.Tensor, free_pages: torch.Tensor, block_table: torch.Tensor,
                  block_size: int, cu_tokens: torch.Tensor, kv_len: torch.Tensor, counts: torch.Tensor,
                  seq_of_token: torch.Tensor, pos: torch.Tensor, slot: torch.Tensor,
                  free_head: Optional[torch.Tensor] = None, stream=None):
    """The tables of a step from its requests' lengths: cached, fresh int32 [B], free_pages int32 [n], free_head int32
    [1] -> block_table int32 [B, max_blocks] (new pages entered), cu_tokens int32 [B + 1], kv_len int32 [B], counts
    int32 [3] (tokens, head after the step, requests served), seq_of_token and pos int32 [T], slot int64 [T] (see
    dsa.h)."""
    device, n, tokens, table = cached.get_device(), cached.shape, slot.shape, block_table.shape
    i32 = torch.int32
    # (one condition for the calls that pass, written out: a function's call for each tensor costs as much as a launch)
    if not (device >= 0 and device == torch._C._cuda_getDevice() and len(n) == len(tokens) == 1
            and cached.dtype is i32 and cached.is_contiguous()
            and fresh.shape == n and fresh.dtype is i32 and fresh.get_device() == device and fresh.is_contiguous()
            and free_pages.dim() == 1 and free_pages.dtype is i32 and free_pages.get_device() == device
            and free_pages.is_contiguous()
            and len(table) == 2 and table[0] == n[0] and block_table.dtype is i32
            and block_table.get_device() == device and block_table.is_contiguous()
            and cu_tokens.shape == (n[0] + 1,) and cu_tokens.dtype is i32 and cu_tokens.get_device() == device
            and cu_tokens.is_contiguous()
            and kv_len.shape == n and kv_len.dtype is i32 and kv_len.get_device() == device and kv_len.is_contiguous()
            and counts.shape == (3,) and counts.dtype is i32 and counts.get_device() == device and counts.is_contiguous()
            and seq_of_token.shape == tokens and seq_of_token.dtype is i32 and seq_of_token.get_device() == device
            and seq_of_token.is_contiguous()
            and pos.shape == tokens and pos.dtype is i32 and pos.get_device() == device and pos.is_contiguous()
            and slot.dtype is torch.int64 and slot.get_device() == device and slot.is_contiguous()
            and -2 ** 31 <= block_size < 2 ** 31
            and (free_head is None or free_head.shape == (1,) and free_head.dtype is i32
                 and free_head.get_device() == device)):
        device = _device("cached", cached)
        _fits_32(block_size=block_size)
        _tensor("cached", cached, i32, (None,), device)
        _tensor("slot", slot, torch.int64, (None,), device)
        for name, t, shape in (("fresh", fresh, n), ("free_pages", free_pages, (None,)),
                               ("block_table", block_table, (n[0], None)), ("cu_tokens", cu_tokens, (n[0] + 1,)),
                               ("kv_len", kv_len, n), ("counts", counts, (3,)), ("seq_of_token", seq_of_token, tokens),
                               ("pos", pos, tokens), ("free_head", free_head, (1,))):
            if t is not None:
                _tensor(name, t, i32, shape, device)
    try:
        args = _STEP_MAPS.pack(
            n[0], tokens[0], block_size, table[1], free_pages.shape[0], cached.data_ptr(), fresh.data_ptr(),
            free_pages.data_ptr(), 0 if free_head is None else free_head.data_ptr(), block_table.data_ptr(),
            cu_tokens.data_ptr(), kv_len.data_ptr(), counts.data_ptr(), seq_of_token.data_ptr(), pos.data_ptr(),
            slot.data_ptr())
    except (struct.error, OverflowError) as e:
        raise _unpackable(e) from None
    code = load().step_maps_packed(args, _stream_of(device, stream))
    if code:
        _check(code, "dsa_step_maps")


# --------------------------------------------------- residual and RMS norm
def _rows(name: str, t: torch.Tensor, dtype, shape, device: int) -> int:
    """Checks a [T, D] tensor whose rows may lie apart: its row stride."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == device and t.stride(1) == 1):
        _tensor(name, t, dtype, tuple(shape), device, last_dense=True)
    # (a single row has no stride of its own)
    return t.stride(0) if shape[0] > 1 else max(shape[1], t.stride(0))


def dsa_add_rmsnorm(x: torch.Tensor, gamma: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                    residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                    codes: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                    round_scale: bool = False, stream=None):
    """x bf16 or fp16 [T, D], gamma fp32 [D], residual and residual_out bf16 or fp32 [T, D] (residual_out may be
    residual) -> residual_out = x + residual, and its RMS norm times gamma as y bf16 [T, D], as codes int8 [T, D] with
    scale fp32 [T], or both (see dsa.h).  x and the residuals may be rows of wider tensors."""
    device, shape, kind, bf16 = x.get_device(), x.shape, x.dtype, torch.bfloat16
    if device < 0 or device != torch._C._cuda_getDevice():
        _device("x", x)
    if len(shape) != 2 or kind is not bf16 and kind is not torch.float16:
        raise DSAError(f"x: {kind} {tuple(shape)}, expected bf16 or fp16 [T, D]")
    if (residual is None) != (residual_out is None) or (codes is None) != (scale is None):
        raise DSAError("dsa_add_rmsnorm: residual goes with residual_out, codes go with scale")
    T, D = shape
    x_stride, inner = x.stride()
    if inner != 1:
        _tensor("x", x, kind, tuple(shape), device, last_dense=True)
    if T == 1:  # (a single row has no stride of its own)
        x_stride = max(D, x_stride)
    r_kind, r_stride, out_stride = bf16, 0, 0
    if residual is not None:
        r_kind = residual.dtype
        if r_kind is not bf16 and r_kind is not torch.float32:
            raise DSAError(f"residual: {r_kind}, expected bf16 or fp32")
        r_stride = _rows("residual", residual, r_kind, shape, device)
        out_stride = r_stride if residual_out is residual else _rows("residual_out", residual_out, r_kind, shape, device)
    if not (gamma.shape == (D,) and gamma.dtype is torch.float32 and gamma.get_device() == device
            and gamma.is_contiguous()):
        _tensor("gamma", gamma, torch.float32, (D,), device)
    if y is not None and not (y.dtype is bf16 and y.shape == shape and y.get_device() == device and y.is_contiguous()):
        _tensor("y", y, bf16, shape, device)
    if codes is not None and not (codes.dtype is torch.int8 and codes.shape == shape and codes.get_device() == device
                                  and codes.is_contiguous() and scale.dtype is torch.float32 and scale.shape == (T,)
                                  and scale.get_device() == device and scale.is_contiguous()):
        _tensor("codes", codes, torch.int8, shape, device)
        _tensor("scale", scale, torch.float32, (T,), device)
    try:
        args = _ADD_RMSNORM.pack(
            T, D, eps, kind is not bf16, r_kind is not bf16, bool(round_scale), x_stride, r_stride, out_stride, x.data_ptr(),
            0 if residual is None else residual.data_ptr(), 0 if residual is None else residual_out.data_ptr(),
            gamma.data_ptr(), 0 if y is None else y.data_ptr(), 0 if codes is None else codes.data_ptr(),
            0 if codes is None else scale.data_ptr())
    except (struct.error, OverflowError) as e:
        raise _unpackable(e) from None
    code = load().add_rmsnorm_packed(args, _stream_of(device, stream))
    if code:
        _check(code, "dsa_add_rmsnorm")
