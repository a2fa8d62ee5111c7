"""The operators of a decode step around the latent cache: what is measured, on
which inputs, and what each computes in plain torch.

  maps: the tables of a step from its requests' lengths.  Request b has
        cached[b] tokens in a paged cache and adds fresh[b]; its new pages come
        from a list of free ones, in the requests' order.  Gives the block
        table, the running token counts, the new lengths, and for each token
        its sequence, position and cache row.  From the first request that
        does not fit on (list, table or token capacity) none is served.
        Rows past the last token: the last token's sequence, position 0, no row.
  attn: softmax attention of each sequence's newest tokens over all rows of
        its latent cache (576 wide, the value is the first 512), causal, with
        an optional sink in each head's denominator; bf16 output, fp32
        log-sum-exp; rows past the last token stay as they are.
  norm: residual addition and RMS norm.  h = x + residual, rounded to the
        residual's type; z = h / sqrt(mean(h^2) + eps) gamma; z in bf16, or in
        8 bits with a scale per row (max |z| / 127, or the power of two at or
        above it), or both.  8-bit codes come back as code x scale, in bf16.
"""
import math

import torch

own = False

D, DV = 576, 512
SCALE = 192.0 ** -0.5
EPS = 1e-6
DEV = "cuda"


def listed():
    return [
        # the first tokens of a short sequence with 4 heads: the smallest call
        {"name": "attn_tiny", "op": "attn", "B": 1, "n_lo": 2, "n_hi": 2, "H": 4, "L": 256, "lo": 256, "page": 0,
         "pad": 0, "empty": False, "sink": False},
        # one token of one user over a 128K context: the latency of a single stream
        {"name": "attn_decode_1", "op": "attn", "B": 1, "n_lo": 1, "n_hi": 1, "H": 128, "L": 131072, "lo": 131072,
         "page": 64, "pad": 0, "empty": False, "sink": False},
        # the framework's headline decode batch: 4 sequences of 64K rows, 2 tokens each
        {"name": "attn_decode_8", "op": "attn", "B": 4, "n_lo": 2, "n_hi": 2, "H": 128, "L": 65536, "lo": 65536,
         "page": 0, "pad": 0, "empty": False, "sink": False},
        # the framework's ragged paged decode: 32 sequences of 4K to 128K rows
        {"name": "attn_ragged_32", "op": "attn", "B": 32, "n_lo": 1, "n_hi": 1, "H": 128, "L": 131072, "lo": 4096,
         "page": 64, "pad": 0, "empty": False, "sink": False},
        # heads spread over eight GPUs (16 here), 0 to 4 new tokens a sequence, padded batch, small pages, a sequence
        # without a row, a sink
        {"name": "attn_heads_16", "op": "attn", "B": 48, "n_lo": 0, "n_hi": 4, "H": 16, "L": 9000, "lo": 700,
         "page": 16, "pad": 5, "empty": True, "sink": True},
        # a chunk of a prompt: 1024 tokens, the last of up to 8192 rows
        {"name": "attn_chunk_1024", "op": "attn", "B": 1, "n_lo": 1024, "n_hi": 1024, "H": 128, "L": 8192, "lo": 8192,
         "page": 64, "pad": 0, "empty": False, "sink": False},
        # the tables of one decode step of the ragged batch
        {"name": "maps_decode_32", "op": "maps", "B": 32, "n_lo": 1, "n_hi": 1, "chunks": 0, "L": 131072, "page": 64,
         "pad": 0, "short": False},
        # decode tokens, prompt chunks and idle requests in one padded batch, small pages
        {"name": "maps_mixed_300", "op": "maps", "B": 300, "n_lo": 0, "n_hi": 4, "chunks": 5, "L": 20000, "page": 16,
         "pad": 1000, "short": False},
        # many requests, several prompts among them
        {"name": "maps_batch_4096", "op": "maps", "B": 4096, "n_lo": 1, "n_hi": 2, "chunks": 40, "L": 65536,
         "page": 64, "pad": 0, "short": False},
        # the hidden states of one decode step, normalised for the prologs
        {"name": "norm_decode_8", "op": "norm", "rows": 8, "D": 7168, "x": "bf16", "res": "bf16", "y": True,
         "int8": False, "pow2": False, "gap": 0},
        # an int8 product's fp16 output (rows of a wider buffer) onto an fp32 residual, quantised for the next product
        {"name": "norm_int8_1001", "op": "norm", "rows": 1001, "D": 7168, "x": "fp16", "res": "fp32", "y": False,
         "int8": True, "pow2": False, "gap": 64},
        # prompts' hidden states, for the prologs and for an int8 product
        {"name": "norm_prompt_16384", "op": "norm", "rows": 16384, "D": 7168, "x": "bf16", "res": "bf16", "y": True,
         "int8": True, "pow2": False, "gap": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "chunk", "maps", "norm", "norm"])
    if op == "norm":
        y, int8 = rng.choice([(True, False), (False, True), (True, True)])
        return {"op": op, "rows": _log(rng, 1, 16384),
                "D": rng.choice([_log(rng, 1, 7168), 8 * _log(rng, 8, 896), 1536, 2048, 4096, 7168]),
                "x": rng.choice(["bf16", "bf16", "fp16"]), "res": rng.choice(["bf16", "bf16", "fp32", "none"]),
                "y": y, "int8": int8, "pow2": rng.random() < 0.25, "gap": rng.choice([0, 0, 1, 8, 136])}
    page = rng.choice([8, 16, 32, 64, 64, 128, 256])
    if op == "maps":
        lo = rng.choice([0, 0, 1])
        return {"op": op, "B": _log(rng, 1, 4096), "n_lo": lo, "n_hi": lo + rng.choice([1, 1, 2, 4]),
                "chunks": rng.choice([0, 0, 1, 7]), "L": _log(rng, 4096, 65536), "page": page,
                "pad": rng.choice([0, 0, 3, 1000]), "short": rng.random() < 0.2}
    page = rng.choice([0, page])
    H = rng.choice([1, 4, 16, 32, 64, 100, 128, 128, 160])
    if op == "chunk":
        n_hi, L, B = _log(rng, 16, 1024), _log(rng, 1024, 8192), 1
        n_lo = n_hi
    else:
        B, L = _log(rng, 1, 64), _log(rng, 1, 131072)
        while B * L > 2200000:
            L = L // 2
        n_lo, n_hi = rng.choice([(1, 1), (1, 1), (2, 2), (0, 3), (1, 4)])
    return {"op": "attn", "B": B, "n_lo": n_lo, "n_hi": n_hi, "H": H, "L": max(L, n_hi), "lo": _log(rng, 1, max(L, n_hi)),
            "page": page, "pad": rng.choice([0, 0, 2]), "empty": rng.random() < 0.2, "sink": rng.random() < 0.3}


# --------------------------------------------------------------------------- inputs
def _normal_rows(g, rows):
    """bf16 rows of normal values, made a piece at a time."""
    kv = torch.empty(rows, D, dtype=torch.bfloat16, device=DEV)
    for r in range(0, rows, 262144):
        n = min(262144, rows - r)
        kv[r:r + n] = torch.randn(n, D, device=DEV, generator=g)
    return kv


def _randint(g, lo, hi, n):
    """n integers of [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), device=DEV, generator=g)


def _pages(g, used, extra):
    """A block table [B, max_blocks] whose first used[b] pages are mapped, and a shuffled list of the free pages."""
    blocks = used["blocks"]
    on = torch.arange(blocks, device=DEV)[None, :] < used["count"][:, None]
    taken = int(used["count"].sum())
    ids = torch.randperm(taken + extra, device=DEV, generator=g).int()
    table = torch.full((used["count"].shape[0], blocks), -1, dtype=torch.int32, device=DEV)
    table[on] = ids[:taken]
    return table, ids[taken:].contiguous()


def _prepare_maps(case, g):
    B, page, L = case["B"], case["page"], case["L"]
    blocks = -(-L // page)
    fresh = _randint(g, case["n_lo"], case["n_hi"], B)
    longest = min(L, 2048)
    chunks = min(case["chunks"], B)
    at = torch.randperm(B, device=DEV, generator=g)[:chunks]
    fresh[at] = _randint(g, min(100, longest), longest, chunks)
    cached = (torch.rand(B, device=DEV, generator=g) * (L - fresh + 1)).long().clamp_(max=L)
    cached = torch.minimum(cached, L - fresh)
    cached[at[:chunks // 2]] = 0  # prompts that begin
    old = -(-cached // page)
    need = int((-(-(cached + fresh) // page) - old).sum())
    table, free = _pages(g, {"count": old, "blocks": blocks}, need + 100)
    head = 7
    if case["short"]:
        free = free[:max(head, head + need // 2)].contiguous()
    T = B * case["n_hi"] + chunks * longest + case["pad"]
    new = lambda n, t=torch.int32: torch.empty(n, dtype=t, device=DEV)  # noqa: E731
    return {"B": B, "T": T, "page": page, "cached": cached.int(), "fresh": fresh.int(), "free": free, "table": table,
            "head": torch.full((1,), head, dtype=torch.int32, device=DEV), "cu": new(B + 1), "kv_len": new(B),
            "counts": new(3), "seq": new(T), "pos": new(T), "slot": new(T, torch.int64)}


def _prepare_attn(case, g):
    B, H, page, L = case["B"], case["H"], case["page"], case["L"]
    n = _randint(g, case["n_lo"], case["n_hi"], B)
    lens = torch.maximum(_randint(g, case["lo"], L, B), n)
    if case["empty"]:
        lens[B - 1] = 0
    T = B * case["n_hi"] + case["pad"]
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    cu[1:] = n.cumsum(0)
    table = None
    if page:
        count = -(-lens // page)
        table, _ = _pages(g, {"count": count, "blocks": -(-L // page)}, 0)
        rows, L = max(1, int(count.sum())) * page, -(-L // page) * page
    else:
        rows = B * L
    st = {"B": B, "T": T, "H": H, "L": L, "page": page, "most": case["n_hi"], "table": table, "cu": cu,
          "kv_len": lens.int(), "kv": _normal_rows(g, rows),
          "q": torch.randn(T, H, D, device=DEV, generator=g).bfloat16(),
          "out": torch.zeros(T, H, DV, dtype=torch.bfloat16, device=DEV),
          "lse": torch.zeros(T, H, dtype=torch.float32, device=DEV),
          "sink": torch.randn(H, device=DEV, generator=g) * 2 if case["sink"] else None}
    if own:  # the argument block and the workspace that a serving loop keeps
        from sparse_attention_prolog_gb300 import binding as fw
        st["args"] = fw.latent_attn_args(T, B, H, L, SCALE, st["q"], st["kv"], st["kv_len"], st["out"], st["lse"],
                                         cu_tokens=cu, block_table=table, block_size=page, sink=st["sink"])
        st["ws"] = torch.zeros(max(fw.workspace_bytes("latent_attn", st["args"]), 256), dtype=torch.uint8, device=DEV)
    return st


def _prepare_norm(case, g):
    rows, wide = case["rows"], case["D"]
    size = torch.exp(torch.randn(rows, 1, device=DEV, generator=g))  # rows of very different sizes
    x = torch.empty(rows, wide + case["gap"], dtype=torch.float16 if case["x"] == "fp16" else torch.bfloat16, device=DEV)
    x.copy_(torch.randn(rows, wide + case["gap"], device=DEV, generator=g) * size)
    st = {"x": x[:, :wide], "gamma": 1 + 0.1 * torch.randn(wide, device=DEV, generator=g), "res": None, "res_out": None,
          "y": None, "codes": None, "scale": None, "values": None, "pow2": case["pow2"]}
    if case["res"] != "none":
        kind = torch.float32 if case["res"] == "fp32" else torch.bfloat16
        st["res"] = (torch.randn(rows, wide, device=DEV, generator=g) * 4).to(kind)
        st["res_out"] = torch.empty_like(st["res"])
    if case["y"]:
        st["y"] = torch.empty(rows, wide, dtype=torch.bfloat16, device=DEV)
    if case["int8"]:
        st["codes"] = torch.empty(rows, wide, dtype=torch.int8, device=DEV)
        st["scale"] = torch.empty(rows, dtype=torch.float32, device=DEV)
        st["values"] = torch.empty(rows, wide, dtype=torch.bfloat16, device=DEV)
    return st


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = {"maps": _prepare_maps, "attn": _prepare_attn, "norm": _prepare_norm}[case["op"]](case, g)
    st["op"] = case["op"]
    return st


# --------------------------------------------------------------------------- plain forms
def _maps(st):
    page, T, blocks = st["page"], st["T"], st["table"].shape[1]
    cached, fresh, head = st["cached"].long(), st["fresh"].long(), st["head"].long()
    old = (cached + page - 1) // page
    last = (cached + fresh + page - 1) // page
    tokens, pages = fresh.cumsum(0), (last - old).cumsum(0)
    bad = (tokens > T) | (pages > st["free"].shape[0] - head) | (last > blocks) | (cached < 0) | (fresh < 0)
    on = bad.long().cumsum(0) == 0
    fresh = torch.where(on, fresh, 0)
    last = torch.where(on, last, old)
    start = (last - old).cumsum(0) - (last - old)  # of each request's pages in the list
    j = torch.arange(blocks, device=DEV)[None, :]
    fill = (j >= old[:, None]) & (j < last[:, None])
    at = (head + start[:, None] + j - old[:, None]).clamp(0, max(st["free"].shape[0] - 1, 0))
    table = torch.where(fill, st["free"][at] if st["free"].shape[0] else -1, st["table"]).int()
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), fresh.cumsum(0)])
    total = cu[-1:]
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(cu[1:], torch.minimum(t, total - 1).clamp(min=0), right=True).clamp(max=st["B"] - 1)
    seq = torch.where(total > 0, seq, 0)
    real = t < total
    pos = torch.where(real, cached[seq] + t - cu[seq], 0)
    slot = torch.where(real, table[seq, pos // page].long() * page + pos % page, -1)
    counts = torch.cat([total, head + (last - old).sum(), on.sum()[None]])
    return {"table": table, "cu": cu.int(), "kv_len": (cached + fresh).int(), "counts": counts.int(), "seq": seq.int(),
            "pos": pos.int(), "slot": slot}


def _attention(st):
    B, H, L, T, most, page = (st[k] for k in ("B", "H", "L", "T", "most", "page"))
    cu, lens = st["cu"].long(), st["kv_len"].long()
    s = torch.arange(L, device=DEV)[None, :]
    b = torch.arange(B, device=DEV)[:, None]
    row = b * L + s if st["table"] is None else st["table"][b, s // page].long() * page + s % page
    row = torch.where(s < lens[:, None], row, 0)
    kv = st["kv"][row].float()  # [B, L, 576]
    i = torch.arange(most, device=DEV)[None, :]
    n = (cu[1:] - cu[:-1])[:, None]
    token = (cu[:-1, None] + i).clamp(max=max(T - 1, 0))  # [B, most]
    q = st["q"][token].float().reshape(B, most * H, D)
    S = torch.matmul(q, kv.transpose(1, 2)).reshape(B, most, H, L) * SCALE
    sees = s[:, None, :] < (lens[:, None] - n + i + 1)[:, :, None]  # [B, most, L]
    S.masked_fill_(~sees[:, :, None, :], float("-inf"))
    sink = torch.full((H,), float("-inf"), device=DEV) if st["sink"] is None else st["sink"]
    m = torch.maximum(S.amax(-1), sink)
    shift = torch.where(torch.isinf(m), 0.0, m)
    S = S.sub_(shift[..., None]).exp_()
    den = S.sum(-1) + torch.exp(sink - shift)
    out = torch.matmul(S.reshape(B, most * H, L), kv[..., :DV]).reshape(B, most, H, DV)
    out = out / torch.where(den > 0, den, 1.0)[..., None]
    real = i < n
    whole, lse = torch.zeros(T, H, DV, dtype=torch.bfloat16, device=DEV), torch.zeros(T, H, device=DEV)
    whole[token[real]] = out[real].bfloat16()
    lse[token[real]] = (shift + torch.log(den))[real]
    return {"out": whole, "lse": lse}


def _norm(st):
    h = st["x"].float()
    said = {}
    if st["res"] is not None:
        h = (h + st["res"].float()).to(st["res"].dtype)
        said["residual"] = h
        h = h.float()
    z = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["gamma"]
    if st["y"] is not None:
        said["y"] = z.bfloat16()
    if st["codes"] is not None:
        top = z.abs().amax(-1, keepdim=True)
        scale = top / torch.full_like(top, 127)  # divided: x / 127 multiplies by 1 / 127
        if st["pow2"]:
            m, e = torch.frexp(scale)
            scale = torch.where(scale > 0, torch.ldexp(torch.ones_like(scale), e - (m == 0.5).int()), scale)
        code = torch.where(scale > 0, torch.round((z / scale).clamp(-127, 127)), 0.0)
        said["scale"] = scale[:, 0]
        said["values"] = (code * scale).bfloat16()
    return said


def run(st):
    if own:
        from sparse_attention_prolog_gb300 import binding as fw
        if st["op"] == "maps":
            fw.dsa_step_maps(st["cached"], st["fresh"], st["free"], st["table"], st["page"], st["cu"], st["kv_len"],
                             st["counts"], st["seq"], st["pos"], st["slot"], free_head=st["head"])
            return {k: st[k] for k in ("table", "cu", "kv_len", "counts", "seq", "pos", "slot")}
        if st["op"] == "attn":
            fw.dsa_latent_attn(st["args"], st["ws"])
            return {"out": st["out"], "lse": st["lse"]}
        fw.dsa_add_rmsnorm(st["x"], st["gamma"], EPS, residual=st["res"], residual_out=st["res_out"], y=st["y"],
                           codes=st["codes"], scale=st["scale"], round_scale=st["pow2"])
        said = {"residual": st["res_out"], "y": st["y"], "scale": st["scale"]}
        if st["codes"] is not None:
            said["values"] = torch.mul(st["codes"], st["scale"][:, None], out=st["values"])
        return {k: v for k, v in said.items() if v is not None}
    return {"maps": _maps, "attn": _attention, "norm": _norm}[st["op"]](st)


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "maps":
        B, chunk = case["B"], min(case["L"], 2048)
        tokens = B * (case["n_lo"] + case["n_hi"]) / 2 + min(case["chunks"], B) * (min(100, chunk) + chunk) / 2
        rows = B * case["n_hi"] + min(case["chunks"], B) * chunk + case["pad"]  # of the token tables
        return {"bytes": 16 * rows + 20 * B + 8 * tokens / case["page"], "flops": 0}
    if case["op"] == "norm":
        res = {"bf16": 4, "fp32": 8, "none": 0}[case["res"]]
        each = 2 + res + 2 * case["y"] + 2 * case["int8"]  # 8-bit codes come back as bf16 values
        return {"bytes": case["rows"] * (case["D"] * each + 4 * case["int8"]) + 4 * case["D"],
                "flops": 8 * case["rows"] * case["D"]}
    B, H = case["B"], case["H"]
    n = (case["n_lo"] + case["n_hi"]) / 2
    some = B - 1 if case["empty"] else B  # sequences that have rows
    mean = max((case["lo"] + case["L"]) / 2, n)
    read = some * (1 if case["n_lo"] > 0 else case["n_hi"] / (case["n_hi"] + 1)) * mean
    return {"bytes": read * 2 * D + B * n * H * (2 * D + 2 * DV + 4),
            "flops": 2 * some * n * H * max(1.0, mean - (n - 1) / 2) * (D + DV)}


# --------------------------------------------------------------------------- the definitions in 64 bits
def _exact_norm(case, st):
    h = st["x"].double()
    said = {}
    if st["res"] is not None:
        said["residual"] = h + st["res"].double()
        h = (st["x"].float() + st["res"].float()).to(st["res"].dtype).double()  # the definition rounds h
    z = h / (h.pow(2).sum(1, keepdim=True) / case["D"] + EPS).sqrt() * st["gamma"].double()
    if case["y"]:
        said["y"] = z
    if case["int8"]:
        s = z.abs().max(1, keepdim=True).values / 127.0
        if case["pow2"]:
            p = (s.view(torch.int64) >> 52 << 52).view(torch.float64)  # the power of two at or below it
            s = torch.where(s > p, 2 * p, p)
        said["scale"] = s[:, 0]
        said["values"] = torch.where(s > 0, (z / s).round() * s, torch.zeros_like(z))
    return said


def exact(case, seed):
    if case["op"] == "maps":
        return None  # whole numbers only
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, st)
    out = torch.zeros(st["T"], st["H"], DV, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["T"], st["H"], dtype=torch.float64, device=DEV)
    cu, lens = st["cu"].tolist(), st["kv_len"].tolist()
    for b in range(st["B"]):
        n = cu[b + 1] - cu[b]
        if st["table"] is None:
            kv = st["kv"][b * st["L"]:b * st["L"] + lens[b]]
        else:
            s = torch.arange(lens[b], device=DEV)
            kv = st["kv"][st["table"][b, s // st["page"]].long() * st["page"] + s % st["page"]]
        kv = kv.double()
        for i in range(0, n, 16):
            k = min(16, n - i)
            t = slice(cu[b] + i, cu[b] + i + k)
            S = torch.einsum("thd,sd->ths", st["q"][t].double(), kv) * SCALE
            hidden = torch.arange(lens[b], device=DEV)[None, :] > lens[b] - n + i + torch.arange(k, device=DEV)[:, None]
            S.masked_fill_(hidden[:, None, :], -math.inf)
            if st["sink"] is not None:
                S = torch.cat([S, st["sink"].double()[None, :, None].expand(k, -1, 1)], 2)
            top = torch.logsumexp(S, 2) if S.shape[2] else torch.full((k, st["H"]), -math.inf, device=DEV).double()
            lse[t] = top
            P = torch.exp(S - torch.where(top > -math.inf, top, 0.0)[..., None])[..., :lens[b]]
            out[t] = torch.einsum("ths,sd->thd", P, kv[:, :DV])
    return {"out": out, "lse": lse}
