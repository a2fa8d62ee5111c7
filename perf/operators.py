"""The operators of the 4-bit latent cache: what is measured, on which inputs,
and what each computes in plain torch.

A row of the cache is 416 bytes: 512 latent dims as signed 4-bit codes
(bytes 0..255; the 4 bytes of dims 8j..8j+7 hold, from the lowest nibble, dims
0, 2, 4, 6, 1, 3, 5, 7 of the eight), one scale byte u for each 16 dims (bytes
256..287; scale (1 + (u mod 8) / 8) 2^(u div 8 - 15), u = 255: not a number),
and 64 rotary dims in bf16 (bytes 288..415).  A latent value is code x scale.

  write: rows of [512 latent | 64 rotary] bf16 values are quantised into the
         rows of a cache that their slots name, and read back;
  read:  rows of the cache, named by slots, come back as bf16 values;
  attn:  softmax attention of each token's heads over the rows of its
         sequence that an index row selects (-1 selects nothing), the value of
         a row being its latent part, with an optional sink in each head's
         denominator; the output in bf16 and the log-sum-exp in fp32.
"""
import math

import torch

own = False

D, DV, ROPE, ROW = 576, 512, 64, 416
SCALE = 192.0 ** -0.5
DEV = "cuda"


def listed():
    return [
        # one decode step's first tokens: two tokens of a short sequence, 4 heads, the smallest call
        {"name": "attn_tiny", "op": "attn", "T": 2, "B": 1, "H": 4, "topk": 32, "L": 256, "lo": 256, "page": 0,
         "holes": 0, "empty": False, "sink": False},
        # one token of one user over a 128K context, all heads on one GPU: latency of a single stream
        {"name": "attn_decode_1", "op": "attn", "T": 1, "B": 1, "H": 128, "topk": 2048, "L": 131072, "lo": 131072,
         "page": 64, "holes": 0, "empty": False, "sink": False},
        # the framework's headline decode step: 4 sequences of 64K keys, 2 tokens each
        {"name": "attn_decode_8", "op": "attn", "T": 8, "B": 4, "H": 128, "topk": 2048, "L": 65536, "lo": 65536,
         "page": 0, "holes": 0, "empty": False, "sink": False},
        # the framework's ragged paged decode: 32 sequences of 4K to 128K keys in pages of 64 rows
        {"name": "attn_ragged_32", "op": "attn", "T": 32, "B": 32, "H": 128, "topk": 2048, "L": 131072, "lo": 4096,
         "page": 64, "holes": 0, "empty": False, "sink": False},
        # a batch whose heads are spread over eight GPUs (16 here), odd selection size and pages, holes, a token
        # with nothing selected, a sink
        {"name": "attn_heads_16", "op": "attn", "T": 48, "B": 16, "H": 16, "topk": 1001, "L": 9000, "lo": 700,
         "page": 3, "holes": 10, "empty": True, "sink": True},
        # the second half of an 8192-token prompt: every token with 2048 of its 4097 to 8192 visible rows
        {"name": "attn_prefill_4096", "op": "attn", "T": 4096, "B": 1, "H": 128, "topk": 2048, "L": 8192, "lo": 8192,
         "page": 0, "holes": 0, "empty": False, "sink": False},
        # the rows of one decode step, written and read back
        {"name": "write_decode_8", "op": "write", "n": 8, "rows": 262144, "pad": 0, "skip": 0},
        # an 8192-token prompt's rows out of a wider projection output, a few tokens without a slot
        {"name": "write_prompt_8192", "op": "write", "n": 8192, "rows": 65536, "pad": 64, "skip": 5},
        # several prompts at once
        {"name": "write_batch_131071", "op": "write", "n": 131071, "rows": 262144, "pad": 0, "skip": 0},
        # the selected rows of one token, gathered as bf16
        {"name": "read_2048", "op": "read", "n": 2048, "rows": 131072, "pad": 0, "skip": 0},
        # the whole latent context of four 64K sequences, for work that wants it in bf16
        {"name": "read_262144", "op": "read", "n": 262144, "rows": 262144, "pad": 0, "skip": 1},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "prefill", "write", "read"])
    if op in ("write", "read"):
        n = _log(rng, 1, 131072)
        return {"op": op, "n": n, "rows": n + _log(rng, 1, 100000), "pad": rng.choice([0, 0, 8, 64, 136]),
                "skip": rng.choice([0, 0, 3, 20])}
    page = rng.choice([0, 0, 1, 3, 16, 64, 256])
    H = rng.choice([1, 4, 16, 32, 64, 100, 128, 128, 160])
    if op == "prefill":
        B, n_q, L, topk = 1, _log(rng, 64, 2048), _log(rng, 2048, 16384), _log(rng, 64, 2048)
    else:
        B, n_q, L, topk = _log(rng, 1, 32), rng.choice([1, 1, 2, 3, 4]), _log(rng, 64, 131072), _log(rng, 1, 4096)
    if page:
        L = -(-L // page) * page
    lo = min(L, n_q + rng.randrange(max(1, L - n_q)))
    return {"op": "attn", "T": B * n_q, "B": B, "H": H, "topk": topk, "L": L, "lo": lo, "page": page,
            "holes": rng.choice([0, 0, 5, 40]), "empty": rng.random() < 0.3, "sink": rng.random() < 0.3}


# --------------------------------------------------------------------------- inputs
def _random_cache(g, rows):
    """A cache of quantised normal rows, made a piece at a time."""
    kv4 = torch.empty(rows, ROW, dtype=torch.uint8, device=DEV)
    for r in range(0, rows, 131072):
        n = min(131072, rows - r)
        kv4[r:r + n] = _quantise(torch.randn(n, D, device=DEV, generator=g).bfloat16())
    return kv4


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = {"op": case["op"]}
    if case["op"] in ("write", "read"):
        n, rows, wide = case["n"], case["rows"], D + case["pad"]
        slot = torch.randperm(rows, device=DEV, generator=g)[:n]
        if case["op"] == "read" and n > 1:
            slot[n // 2:] = slot[n // 2:].sort().values  # runs of rows among scattered ones
        if case["skip"]:
            slot[torch.rand(n, device=DEV, generator=g) * 100 < case["skip"]] = -1
        st["slot"] = slot
        st["kv4"] = _random_cache(g, rows)
        if case["op"] == "write":
            x = torch.randn(n, wide, device=DEV, generator=g) * torch.exp(torch.randn(n, 1, device=DEV, generator=g))
            st["x"] = x.bfloat16()[:, :D]
        st["out"] = torch.empty(n, D if case["op"] == "write" else wide, dtype=torch.bfloat16, device=DEV)[:, :D]
        return st
    T, B, H, k, L, page = (case[x] for x in ("T", "B", "H", "topk", "L", "page"))
    n_q = T // B
    lens = torch.randint(case["lo"], L + 1, (B,), device=DEV, generator=g).clamp_(min=n_q)
    seq = torch.arange(T, device=DEV) // n_q
    pos = lens[seq] - n_q + torch.arange(T, device=DEV) % n_q
    pick = torch.rand(T, L, device=DEV, generator=g)
    pick.masked_fill_(torch.arange(L, device=DEV)[None, :] > pos[:, None], -1.0)
    top = pick.topk(min(k, L), dim=1)
    idx = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    idx[:, :min(k, L)] = torch.where(top.values >= 0, top.indices, -1).int()
    if case["holes"]:
        idx[torch.rand(T, k, device=DEV, generator=g) * 100 < case["holes"]] = -1
    if case["empty"]:
        idx[T - 1] = -1
    table = None
    if page:
        per = L // page if L % page == 0 else -(-L // page)
        L = per * page
        used = (torch.arange(per, device=DEV)[None, :] * page < lens[:, None])
        n_pages = int(used.sum())
        table = torch.full((B, per), -1, dtype=torch.int32, device=DEV)
        table[used] = torch.randperm(n_pages, device=DEV, generator=g).int()
        rows = n_pages * page
    else:
        rows = B * L
    st.update(T=T, B=B, n_q=n_q, H=H, k=k, L=L, page=page, idx=idx, table=table, kv4=_random_cache(g, rows),
              q=torch.randn(T, H, D, device=DEV, generator=g).bfloat16(),
              out=torch.empty(T, H, DV, dtype=torch.bfloat16, device=DEV),
              lse=torch.empty(T, H, dtype=torch.float32, device=DEV),
              sink=torch.randn(H, device=DEV, generator=g) * 2 if case["sink"] else None)
    if own:  # the argument block and the workspace that a serving loop keeps
        from sparse_attention_prolog_gb300 import binding as fw
        st["args"] = fw.attn_kv4_args(T, B, n_q, H, k, L, SCALE, st["q"], st["kv4"], idx, st["out"], st["lse"],
                                      block_table=table, block_size=page, sink=st["sink"])
        st["ws"] = torch.zeros(max(fw.workspace_bytes("attn_kv4", st["args"]), 256), dtype=torch.uint8, device=DEV)
    return st


# --------------------------------------------------------------------------- plain forms
def _power(e):
    """2^e in fp32, exactly (pow() may be an ulp off, and ties would then round the wrong way)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """Rows of the cache from bf16 rows [n, 576]."""
    n = x.shape[0]
    v = x[:, :DV].float().reshape(n, 32, 16)
    amax = v.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(amax)
    m, e = torch.frexp(torch.where(bad, 1.0, amax) / torch.full_like(amax, 7))  # divided: x / 7 multiplies by 1/7
    s = (torch.round(m * 16) * _power(e.clamp(min=-100) - 4)).clamp(2.0 ** -15, 1.75 * 2.0 ** 16)  # 4 significant bits
    code = torch.where(bad, 0.0, torch.round(v / s).clamp(-7, 7)).int() & 15
    m, e = torch.frexp(s)
    u = torch.where(bad, 255.0, (e.float() + 14) * 8 + (m * 16 - 8))[..., 0].to(torch.uint8)
    nib = code.reshape(n, 64, 4, 2).transpose(-1, -2).reshape(n, 64, 4, 2)  # nibble order 0 2 4 6 1 3 5 7, in pairs
    return torch.cat([(nib[..., 0] | nib[..., 1] << 4).to(torch.uint8).reshape(n, 256), u,
                      x[:, DV:].contiguous().view(torch.uint8)], 1)


def _values(rows):
    """fp32 values [..., 576] of rows of the cache [..., 416]."""
    lead = rows.shape[:-1]
    b = rows[..., :256]
    nib = torch.stack([b & 15, b >> 4], -1).reshape(*lead, 64, 2, 4).transpose(-1, -2)
    code = (nib.float() + 8) % 16 - 8
    u = rows[..., 256:288].float()
    s = _power(torch.floor(u / 8) - 15) * (1 + u % 8 / 8)
    s = torch.where(rows[..., 256:288] == 255, float("nan"), s)
    return torch.cat([(code.reshape(*lead, 32, 16) * s[..., None]).reshape(*lead, DV),
                      rows[..., 288:].contiguous().view(torch.bfloat16).float()], -1)


def _read(kv4, slot):
    return torch.where((slot >= 0)[:, None], _values(kv4[slot.clamp(min=0)]), 0.0)


def _cache_row(st):
    """Physical row of every selected position, and which slots select one."""
    idx = st["idx"].long()
    s = idx.clamp(min=0)
    b = (torch.arange(st["T"], device=idx.device) // st["n_q"])[:, None]
    if st["table"] is None:
        return b * st["L"] + s, idx >= 0
    return st["table"][b, s // st["page"]].long() * st["page"] + s % st["page"], idx >= 0


def _attention(st):
    row, on = _cache_row(st)
    kv = _values(st["kv4"][row.clamp(min=0)])
    S = torch.matmul(st["q"].float(), kv.transpose(1, 2)) * SCALE
    S.masked_fill_(~on[:, None, :], float("-inf"))
    sink = torch.full((st["H"],), float("-inf"), device=S.device) if st["sink"] is None else st["sink"]
    m = torch.maximum(S.amax(-1), sink[None, :])
    shift = torch.where(torch.isinf(m), 0.0, m)
    S = torch.exp(S - shift[..., None])
    den = S.sum(-1) + torch.exp(sink - shift)
    out = torch.matmul(S, kv[..., :DV]) / torch.where(den > 0, den, 1.0)[..., None]
    return out, shift + torch.log(den)


def run(st):
    if own:
        from sparse_attention_prolog_gb300 import binding as fw
        if st["op"] == "attn":
            fw.dsa_sparse_attn_kv4(st["args"], st["ws"])
            return {"out": st["out"], "lse": st["lse"]}
        if st["op"] == "write":
            fw.dsa_kv4_write(st["x"], st["kv4"], st["slot"])
        fw.dsa_kv4_read(st["kv4"], st["slot"], st["out"])
        return {"out": st["out"]}
    if st["op"] == "attn":
        out, lse = _attention(st)
        return {"out": out.bfloat16(), "lse": lse}
    if st["op"] == "write":
        on = st["slot"] >= 0
        st["kv4"][st["slot"][on]] = _quantise(st["x"])[on]
    return {"out": _read(st["kv4"], st["slot"]).bfloat16()}


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "read":
        return {"bytes": case["n"] * (8 + ROW + 2 * D), "flops": 2 * case["n"] * DV}
    if case["op"] == "write":  # quantised and stored, then read back and returned
        return {"bytes": case["n"] * (8 + 2 * D + ROW + ROW + 2 * D), "flops": 6 * case["n"] * DV}
    T, B, H, k, L = (case[x] for x in ("T", "B", "H", "topk", "L"))
    n_q, mean = T // B, (max(case["lo"], T // B) + L) / 2
    sel = sum(min(k, max(1.0, mean - n_q + j + 1)) for j in range(n_q)) / n_q * (1 - case["holes"] / 100)
    tokens = T - (1 if case["empty"] else 0)
    distinct = B * mean * (1 - (1 - min(1.0, sel / mean)) ** n_q)  # rows that the tokens of a sequence share
    return {"bytes": distinct * ROW + T * (k * 4 + H * (2 * D + 2 * DV + 4)), "flops": 2 * tokens * sel * H * (D + DV)}


# --------------------------------------------------------------------------- the definitions in 64 bits
def _exact_values(rows):
    """float64 values of cache rows: tables for the nibbles and the scale bytes."""
    n = rows.shape[0]
    i4 = torch.tensor([*range(8), *range(-8, 0)], dtype=torch.float64, device=rows.device)
    sc = torch.tensor([(8 + u % 8) * 2.0 ** (u // 8 - 18) for u in range(255)] + [math.nan], dtype=torch.float64,
                      device=rows.device)
    val = torch.empty(n, D, dtype=torch.float64, device=rows.device)
    for nibble, dim in enumerate((0, 2, 4, 6, 1, 3, 5, 7)):
        at = rows[:, nibble // 2:256:4].long()
        val[:, dim:DV:8] = i4[at >> 4 if nibble % 2 else at & 15]
    val[:, :DV] *= sc[rows[:, 256:288].long()].repeat_interleave(16, 1)
    val[:, DV:] = rows[:, 288:].contiguous().view(torch.bfloat16).double()
    return val


def _exact_quantised(x):
    """float64 values that 4 bits hold of rows x [n, 576]."""
    v = x.double()
    g = v[:, :DV].reshape(-1, 16)
    top = g.abs().amax(1)
    ideal = (top / torch.full_like(top, 7)).clamp(min=2.0 ** -15)
    octave = (ideal.view(torch.int64) >> 52 << 52).view(torch.float64)  # the power of two at or below it
    s = (torch.round(ideal / octave * 8) / 8 * octave).clamp(max=1.75 * 2.0 ** 16)[:, None]
    q = torch.round(g / s).clamp(-7, 7) * s
    return torch.cat([q.reshape(-1, DV), v[:, DV:]], 1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] != "attn":
        if case["op"] == "write":
            val = _exact_quantised(st["x"])
        else:
            val = _exact_values(st["kv4"][st["slot"].clamp(min=0)])
        val[st["slot"] < 0] = 0.0
        return {"out": val}
    out, lse = [], []
    for t in range(st["T"]):
        idx = st["idx"][t].long()
        idx = idx[idx >= 0]
        b = t // st["n_q"]
        row = b * st["L"] + idx if st["table"] is None else \
            st["table"][b, idx // st["page"]].long() * st["page"] + idx % st["page"]
        kv = _exact_values(st["kv4"][row])
        S = st["q"][t].double() @ kv.T * SCALE
        if st["sink"] is not None:
            S = torch.cat([S, st["sink"].double()[:, None]], 1)
            kv = torch.cat([kv, torch.zeros(1, D, dtype=torch.float64, device=kv.device)])
        if S.shape[1] == 0:
            out.append(torch.zeros(st["H"], DV, dtype=torch.float64, device=DEV))
            lse.append(torch.full((st["H"],), -math.inf, dtype=torch.float64, device=DEV))
            continue
        out.append(torch.softmax(S, 1) @ kv[:, :DV])
        lse.append(torch.logsumexp(S, 1))
    return {"out": torch.stack(out), "lse": torch.stack(lse)}
