"""Step maps on the GPU against a plain loop over the requests, exactly, and the
calls that they refuse or report."""
import numpy as np
import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DATA_ERROR = 6


def reference(cached, fresh, free, head, table, bs, T):
    """The maps by a loop; table is changed in place."""
    n, blocks = table.shape
    cu, kv_len, seq, pos, slot = [0], [], [], [], []
    taken = served = 0
    for b in range(n):
        c, f = int(cached[b]), int(fresh[b])
        on = served == b and head >= 0 and c >= 0 and f >= 0 and c + f <= blocks * bs and cu[-1] + f <= T
        if on:
            old, last = -(-c // bs), -(-(c + f) // bs)
            on = head + taken + last - old <= len(free)
        if not on:
            cu.append(cu[-1])
            kv_len.append(c)
            continue
        served += 1
        table[b, old:last] = free[head + taken:head + taken + last - old]
        taken += last - old
        cu.append(cu[-1] + f)
        kv_len.append(c + f)
        for p in range(c, c + f):
            seq.append(b)
            pos.append(p)
            page = int(table[b, p // bs])
            slot.append(page * bs + p % bs if page >= 0 else -1)
    k = T - len(seq)
    counts = [cu[-1], head + taken, served]
    return cu, kv_len, counts, seq + [seq[-1] if seq else 0] * k, pos + [0] * k, slot + [-1] * k


class Step:
    def __init__(self, cached, fresh, bs, blocks, free, head=None, T=None, table=None, seed=0):
        rng = np.random.default_rng(seed)
        self.bs, self.head = bs, head
        self.cached, self.fresh = np.asarray(cached, dtype=np.int32), np.asarray(fresh, dtype=np.int32)
        n = len(self.cached)
        self.free = np.asarray(free, dtype=np.int32)
        self.T = int(np.maximum(self.fresh, 0).sum()) + 3 if T is None else T
        if table is None:
            table = rng.integers(0, 1 << 20, (n, blocks)).astype(np.int32)  # what a step does not enter stays
        self.table = table.copy()
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
        i32 = lambda k: torch.full((k,), -77, dtype=torch.int32, device=DEV)  # noqa: E731
        self.d = {"cached": up(self.cached), "fresh": up(self.fresh), "free_pages": up(self.free),
                  "block_table": up(self.table), "block_size": bs, "cu_tokens": i32(n + 1), "kv_len": i32(n),
                  "counts": i32(3), "seq_of_token": i32(self.T), "pos": i32(self.T),
                  "slot": torch.full((self.T,), -77, dtype=torch.int64, device=DEV),
                  "free_head": None if head is None else torch.tensor([head], dtype=torch.int32, device=DEV)}

    def run(self, stream=None):
        B.dsa_step_maps(stream=stream, **self.d)

    def check(self, error=False):
        torch.cuda.synchronize()
        assert B.device_error() == (DATA_ERROR if error else 0)
        table = self.table.copy()
        want = reference(self.cached, self.fresh, self.free, self.head or 0, table, self.bs, self.T)
        for name, w in zip(("cu_tokens", "kv_len", "counts", "seq_of_token", "pos", "slot"), want):
            assert self.d[name].tolist() == w, name
        assert np.array_equal(self.d["block_table"].cpu().numpy(), table)


def _random(n, bs, blocks, most, seed, idle=0.3):
    rng = np.random.default_rng(seed)
    fresh = rng.integers(1, most + 1, n) * (rng.random(n) > idle)
    cached = rng.integers(0, blocks * bs - fresh + 1)
    need = int((-(-(cached + fresh) // bs) - -(-cached // bs)).sum())
    return cached, fresh, rng.permutation(1 << 21)[:need + 9], need


@pytest.mark.parametrize("n,bs,blocks,most", [(1, 64, 4, 1), (1, 64, 4, 200), (2, 1, 50, 3), (32, 64, 2048, 1),
                                              (33, 16, 20, 4), (255, 8, 30, 9), (256, 3, 40, 5), (257, 64, 10, 2),
                                              (1000, 128, 8, 40), (1025, 16, 64, 4), (4099, 64, 32, 3), (8192, 7, 9, 2)])
@pytest.mark.parametrize("head", [None, 5])
def test_against_a_loop(n, bs, blocks, most, head, cuda_lib):
    cached, fresh, free, need = _random(n, bs, blocks, most, n + bs)
    s = Step(cached, fresh, bs, blocks, free, head, seed=n)
    s.run()
    s.check()


@pytest.mark.parametrize("cached,fresh,T", [
    ([0], [1], 1), ([63], [1], 1), ([64], [1], 1), ([63], [2], 2), ([0], [64], 64), ([0], [256], 300), ([255], [1], 1),
    ([10, 20, 30], [0, 0, 0], 0), ([10, 20, 30], [0, 0, 0], 5), ([0, 0], [0, 3], 3), ([5, 0, 7], [2, 0, 0], 8),
    ([100], [0], 4),
])
def test_edges(cached, fresh, T, cuda_lib):
    s = Step(cached, fresh, 64, 4, np.arange(50, 80), T=T)
    s.run()
    s.check()


def test_a_long_prompt_and_padding(cuda_lib):
    s = Step([0, 70000, 5], [70000, 1, 0], 64, 1200, np.random.default_rng(1).permutation(5000), 17, T=100000)
    s.run()
    s.check()


@pytest.mark.parametrize("cached,fresh,kw", [
    ([0, 0, 0], [100, 300, 1], {"blocks": 4}),                      # a request past its table's end
    ([0, 10, 20], [30, 30, 30], {"T": 89}),                         # more tokens than rows
    ([0, 10, 20], [30, 30, 30], {"T": 59}),
    ([0, 0, 0], [64, 64, 64], {"free": [3, 4]}),                    # too few pages
    ([0, 0, 0], [64, 64, 64], {"free": [3, 4, 5, 6], "head": 2}),
    ([0, 0, 0], [64, 64, 64], {"free": []}),
    ([64, 64], [0, 1], {"free": []}),
    ([64, 64], [0, 0], {"free": [1], "head": 9}),                   # a head past the list, or before it
    ([64, 64], [0, 1], {"head": -1}),
    ([5, -1, 7], [1, 1, 1], {}), ([5, 6, 7], [1, -2, 1], {}),       # negative lengths
    ([2 ** 31 - 1, 0], [2 ** 31 - 1, 1], {}), ([0, 2 ** 31 - 1], [1, 1], {}),
    ([0] * 300, [1] * 299 + [-1], {}), ([0] * 3000, [1] * 1500 + [-1] + [1] * 1499, {"free": np.arange(4000)}),
])
def test_requests_that_do_not_fit(cached, fresh, kw, cuda_lib):
    kw = dict(kw)
    blocks, free, head, T = kw.get("blocks", 8), kw.get("free", np.arange(400)), kw.get("head"), kw.get("T", 5000)
    s = Step(cached, fresh, 64, blocks, free, head, T=T)
    s.run()
    s.check(error=True)


def test_a_page_that_is_not_mapped(cuda_lib):
    table = np.full((2, 8), -1, dtype=np.int32)
    table[0, :2] = [7, -3]
    s = Step([100, 0], [40, 10], 64, 8, [9, 11, -5], T=60, table=table)
    s.run()
    s.check(error=True)
    assert (s.d["slot"][:28] == -1).all() and (s.d["slot"][28:40] >= 0).all()


def test_steps_in_a_row_captured_and_replayed(cuda_lib):
    """Two steps a replay, each taking the other's lengths and head; the tables grow
    as a loop on the host says."""
    rng = np.random.default_rng(3)
    n, bs, blocks, T = 40, 8, 60, 128
    free = rng.permutation(4000).astype(np.int32)
    lens, head = np.zeros(n, dtype=np.int32), 0
    table = np.full((n, blocks), -1, dtype=np.int32)
    a = Step(lens, np.zeros(n), bs, blocks, free, 0, T=T, table=table)
    d = a.d
    state = [(d["cached"], d["free_head"]), (torch.empty_like(d["kv_len"]), torch.empty(1, dtype=torch.int32, device=DEV))]
    fresh = [torch.zeros(n, dtype=torch.int32, device=DEV) for _ in range(2)]
    counts = [torch.zeros(3, dtype=torch.int32, device=DEV) for _ in range(2)]
    rest = {k: d[k] for k in ("free_pages", "block_table", "block_size", "cu_tokens", "seq_of_token", "pos", "slot")}

    def both():
        for i in range(2):
            B.dsa_step_maps(cached=state[i][0], fresh=fresh[i], kv_len=state[1 - i][0], counts=counts[i],
                            free_head=state[i][1], **rest)
            state[1 - i][1].copy_(counts[i][1:2])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()  # (nothing new: the state stays)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for _ in range(4):
        new = [rng.integers(0, 4, n).astype(np.int32) for _ in range(2)]
        for f, x in zip(fresh, new):
            f.copy_(torch.from_numpy(x))
        g.replay()
        torch.cuda.synchronize()
        assert B.device_error() == 0
        for x in new:
            want = reference(lens, x, free, head, table, bs, T)
            lens, head = np.asarray(want[1], dtype=np.int32), want[2][1]
        assert state[0][0].tolist() == want[1] and int(state[0][1]) == head
        assert d["slot"].tolist() == want[5] and d["pos"].tolist() == want[4]
        assert np.array_equal(d["block_table"].cpu().numpy(), table)


def test_refusals(cuda_lib):
    def bad(**kw):
        s = Step([5, 6], [1, 1], 64, 4, np.arange(50, 80))
        s.d.update(kw)
        with pytest.raises(B.DSAError):
            s.run()

    s = Step([5, 6], [1, 1], 64, 4, np.arange(50, 80))
    both = torch.zeros(4, dtype=torch.int32, device=DEV)
    bad(kv_len=s.d["cached"], cached=s.d["cached"])
    bad(cached=both[:2], kv_len=both[1:3])
    bad(counts=both[:3], free_head=both[2:3])
    bad(block_size=0)
    bad(block_size=2 ** 31)
    bad(block_size=2 ** 30)
    bad(fresh=s.d["fresh"].long())
    bad(fresh=s.d["fresh"].cpu())
    bad(slot=s.d["slot"][:-1])
    bad(slot=s.d["slot"].int())
    bad(block_table=s.d["block_table"][:, ::2])
    bad(cu_tokens=s.d["cu_tokens"][:2])
    big = torch.zeros(8193, dtype=torch.int32, device=DEV)
    bad(cached=big, fresh=big.clone(), kv_len=big.clone(), cu_tokens=torch.zeros(8194, dtype=torch.int32, device=DEV),
        block_table=torch.zeros(8193, 2, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert B.device_error() == 0
    Step([], [], 64, 4, [], T=0, table=np.zeros((0, 4), dtype=np.int32)).run()
