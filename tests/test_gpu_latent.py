"""The attention over the whole latent cache against a float64 form on the same
bf16 values, with bounds worked out from its roundings, and its refusals that
need a GPU.

Per output element, with A = sum_j p_j |v_j| (p_j the softmax weights): the
probabilities are rounded to bf16 (at most 2^-8 of each: 2^-8 A; half a step
relative to the value is 2^-8) and so is the result (2^-8 |out|).  A logit is a
sum of 576 exact products held in fp32, off by at most 576 * 2^-23 of the largest
sum of their magnitudes, and its product with scale / ln 2 is rounded three times
(the factor, the product, the exponent's argument: 3 * 2^-23 of the magnitude);
together delta.  An error of delta in a logit changes a weight by delta of itself,
and the normalisation by as much again: 2 delta A.  Every exponential (the weight,
the rescaling between tiles, the merge) is within 2^-22 of itself plus what its
argument, at most the logits' spread, loses to rounding: 2^-16 in all below a
spread of 32.  The fp32 sums of L terms are off by at most L * 2^-23 of A.  lse moves
by delta, by the sums' L * 2^-23 + 2^-16 and by 2^-22 of itself."""
import math

import numpy as np
import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DATA_ERROR = 6
TIMEOUT = 5
SCALE = 192.0 ** -0.5
NAN = float("nan")


def ok():
    torch.cuda.synchronize()
    assert B.device_error() == 0


class Case:
    """A batch: n[b] new tokens of sequences of lens[b] rows.  Rows of the cache that
    no sequence has, and q's padding, are NaN; out and lse start as 7."""

    def __init__(self, n, lens, H, page=0, pad=0, sink=False, seed=0, size=1.0, scale=SCALE, spare_rows=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.n, self.lens, self.H, self.scale = list(n), list(lens), H, scale
        self.B, self.T = len(n), sum(n) + pad
        most = max(max(lens), 1)
        self.page = page
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.cu = torch.tensor([0, *np.cumsum(n)], dtype=torch.int32, device=DEV)
        self.table = None
        rng = np.random.default_rng(seed)
        if page:
            blocks = -(-most // page)
            self.L = blocks * page
            used = [-(-x // page) for x in lens]
            pages = sum(used) + 2
            ids = rng.permutation(pages)
            table = np.full((self.B, blocks), -1, dtype=np.int32)
            at = 0
            for b, u in enumerate(used):
                table[b, :u] = ids[at:at + u]
                at += u
            self.table = torch.from_numpy(table).to(DEV)
            rows = pages * page
            self.rows_of = [torch.tensor([table[b, s // page] * page + s % page for s in range(lens[b])],
                                         dtype=torch.long, device=DEV) for b in range(self.B)]
        else:
            self.L = most
            rows = self.B * most + spare_rows
            self.rows_of = [b * most + torch.arange(lens[b], device=DEV) for b in range(self.B)]
        self.kv = torch.full((rows, 576), NAN, dtype=torch.bfloat16, device=DEV)
        for r in self.rows_of:
            self.kv[r] = (torch.randn(len(r), 576, device=DEV, generator=g) * size).bfloat16()
        self.q = torch.full((self.T, H, 576), NAN, dtype=torch.bfloat16, device=DEV)
        self.q[:sum(n)] = torch.randn(sum(n), H, 576, device=DEV, generator=g).bfloat16()
        self.sink = None
        if sink:
            self.sink = torch.randn(H, device=DEV, generator=g) * 3
            self.sink[::3] = -math.inf
        self.fresh()

    def fresh(self):
        self.out = torch.full((self.T, self.H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.T, self.H), 7.0, device=DEV)

    def args(self, **kw):
        kw = {"lse": self.lse, "cu_tokens": self.cu, "block_table": self.table, "block_size": self.page,
              "sink": self.sink, **kw}
        return B.latent_attn_args(self.T, self.B, self.H, self.L, self.scale, self.q, self.kv, self.kv_len, self.out,
                                  **kw)

    def run(self, ws=None, stream=None, **kw):
        return B.dsa_latent_attn(self.args(**kw), ws, stream)

    def check(self, lse=True, tokens=None):
        """Every token (or some) against float64, and the padding as it was."""
        at = 0
        for b in range(self.B):
            kv_all = self.kv[self.rows_of[b]].double()
            for i in range(self.n[b]):
                t = at + i
                if tokens is not None and t not in tokens:
                    continue
                kv = kv_all[:max(0, self.lens[b] - self.n[b] + i + 1)]
                self._token(t, kv, lse)
            at += self.n[b]
        assert bool((self.out[at:] == 7.0).all()) and bool((self.lse[at:] == 7.0).all())

    def _token(self, t, kv, lse):
        q = self.q[t].double()
        S = q @ kv.T * self.scale
        mag = q.abs() @ kv.abs().T * self.scale
        L = kv.shape[0]
        delta = float(mag.max()) * (576 + 3) * 2.0 ** -23 if L else 0.0
        if self.sink is not None:
            S = torch.cat([S, self.sink.double()[:, None]], 1)
            kv = torch.cat([kv, torch.zeros(1, 576, dtype=torch.float64, device=DEV)])
        want_lse = torch.logsumexp(S, 1) if S.shape[1] else torch.full((self.H,), -math.inf, device=DEV).double()
        p = torch.exp(S - torch.where(torch.isinf(want_lse), 0.0, want_lse)[:, None])
        want, A = p @ kv[:, :512], p @ kv[:, :512].abs()
        got = self.out[t].double()
        sums = L * 2.0 ** -23
        bound = A * (2.0 ** -8 + 2 * delta + sums + 2.0 ** -16) * (1 + 2.0 ** -7) + want.abs() * 2.0 ** -8 + 1e-30
        off = (got - want).abs()
        assert bool((off <= bound).all()), f"token {t}: {float((off / bound).max()):.3g} of its bound"
        # the roundings of the weights are independent: they do not add up to their bound
        rms = float((off.square().mean() / want.square().mean().clamp(min=1e-300)).sqrt())
        assert rms < 5e-3, f"token {t}: rms {rms:.3g}"
        if lse:
            got = self.lse[t].double()
            inf = torch.isinf(want_lse)
            assert torch.equal(got[inf], want_lse[inf])
            off = (got - want_lse)[~inf].abs()
            assert bool((off <= delta + sums + 2.0 ** -16 + 2.0 ** -22 * want_lse[~inf].abs()).all()), f"token {t}: lse {float(off.max()):.3g}"


SMALL = [
    # n, lens, H, page
    ([1], [1], 1, 0),
    ([2], [256], 4, 0),
    ([1], [63], 128, 0), ([1], [64], 128, 0), ([1], [65], 128, 64), ([1], [129], 128, 128),
    ([1], [1000], 128, 64),
    ([2], [300], 128, 0),
    ([3, 1, 2], [200, 1, 77], 128, 64),
    ([1, 0, 4, 2, 0], [500, 90, 700, 2, 0], 16, 16),
    ([5, 5], [130, 131], 100, 8),
    ([2, 1], [400, 64], 160, 32),
    ([1, 2], [70, 200], 1024, 64),
    ([7, 3], [7, 100], 3, 192),
    ([1, 1, 1], [0, 5, 0], 128, 64),
    ([4, 2], [2, 0], 16, 0),
    ([33], [40], 1, 8),
    ([130], [257], 2, 16),
]


@pytest.mark.parametrize("n,lens,H,page", SMALL)
def test_small_shapes(n, lens, H, page, cuda_lib):
    c = Case(n, lens, H, page, pad=2, seed=len(n) + H)
    c.run()
    ok()
    c.check()


@pytest.mark.parametrize("n,lens,H,page", [
    ([1], [20000], 128, 64), ([1], [20000], 16, 0), ([2, 2, 2, 2], [4100, 5000, 64, 3000], 128, 0),
    ([1] * 9, [4096, 1, 8191, 300, 2048, 10000, 64, 65, 7000], 128, 64),
    ([0, 3, 1, 4, 2, 0, 1] * 5, [700, 1000, 9000, 64, 3000, 50, 128] * 5, 16, 16),
    ([300], [1000], 128, 64),
])
def test_split_sequences(n, lens, H, page, cuda_lib):
    c = Case(n, lens, H, page, pad=3, seed=H + len(n))
    c.run()
    ok()
    tokens = None if sum(n) < 100 else {0, 1, 63, 64, 150, 298, 299}
    c.check(tokens=tokens)


@pytest.mark.parametrize("n,lens,H,page", [([1], [65], 128, 64), ([1, 1], [5000, 0], 128, 64),
                                           ([2, 4, 0], [900, 3, 7], 16, 16)])
def test_a_sink(n, lens, H, page, cuda_lib):
    c = Case(n, lens, H, page, sink=True, seed=4)
    c.run()
    ok()
    c.check()


def test_a_uniform_batch_needs_no_token_counts(cuda_lib):
    c = Case([2] * 5, [300, 64, 2, 1000, 129], 32, 64, seed=3)
    c.run(cu_tokens=None, n_q=2)
    ok()
    c.check()


def test_without_lse(cuda_lib):
    c = Case([1, 2], [3000, 100], 128, 64, seed=3)
    c.run(lse=None)
    ok()
    assert bool((c.lse == 7.0).all())
    c.check(lse=False)


@pytest.mark.parametrize("lens", [[5000], [640, 300]])
def test_a_maximum_that_grows_with_every_tile(lens, cuda_lib):
    """Rows along q, longer and longer: each tile's logits pass the ones before by
    more than 2^8, and the output is the last rows' (spread below 32 in a tile; what
    is further from the maximum has no weight)."""
    c = Case([1] * len(lens), lens, 128, 64, seed=9)
    for r in c.rows_of:
        up = torch.linspace(0.1, 12.0, len(r), device=DEV)[:, None]
        c.kv[r] = (c.kv[r].float() * 0.1 + up * torch.sign(c.q[0, 0].float())).bfloat16()
    c.q.copy_(c.q[:, :1].abs() * torch.sign(c.q[0, 0]) + 0 * c.q)
    c.run()
    ok()
    c.check()


def test_large_and_small_logits(cuda_lib):
    for size, scale in ((1.0, 1e-4), (4.0, SCALE), (1e-3, 1.0)):
        c = Case([1, 2], [2000, 130], 128, 64, seed=2, size=size, scale=scale)
        c.run()
        ok()
        c.check()


def test_rows_that_a_token_does_not_see_may_hold_anything(cuda_lib):
    """The tail of the last page and the cache's other rows are NaN in every case
    here; infinities, and at 128 heads the newer tokens' own rows, as well."""
    c = Case([3, 2], [100, 64], 128, 64, seed=5)
    seen = torch.cat(c.rows_of)
    rest = torch.ones(c.kv.shape[0], dtype=torch.bool, device=DEV)
    rest[seen] = False
    c.kv[rest] = math.inf
    newest = c.rows_of[0][-1]
    kept = c.kv[newest].clone()
    c.kv[newest] = NAN
    c.run()
    ok()
    assert bool(c.out[2].isnan().all()) and bool(c.lse[2].isnan().all())  # that token sees it
    c.check(tokens={0, 1, 3, 4})
    c.kv[newest] = kept
    c.fresh()
    c.run()
    ok()
    c.check()


def test_a_row_that_is_not_a_number_reaches_who_sees_it(cuda_lib):
    c = Case([1, 1], [5000, 300], 128, 64, seed=6)
    c.kv[c.rows_of[0][1234], 17] = NAN
    c.run()
    ok()
    assert bool(c.out[0].isnan().all())
    c.check(tokens={1})


def test_pages_that_do_not_exist_read_as_zeros(cuda_lib):
    for bad in (-5, 1 << 20, 2 ** 31 - 1):
        c = Case([1, 1], [300, 700], 128, 64, seed=7)
        was = int(c.table[1, 3])
        zero = c.kv.clone()
        zero[was * 64:was * 64 + 64] = 0
        c.table[1, 3] = bad
        c.run()
        torch.cuda.synchronize()
        assert B.device_error() == DATA_ERROR
        c.kv = zero
        c.check()
        c.table[1, 3] = was
        c.fresh()
        c.run()
        ok()
        c.check()


def test_lengths_and_counts_out_of_range_are_reported(cuda_lib):
    c = Case([1, 2], [300, 128], 128, 64, seed=8)
    good_len, good_cu = c.kv_len.clone(), c.cu.clone()
    for kv_len, cu, tokens in ([[300, -3], [0, 1, 3], {0}], [[300, 10 ** 6], [0, 1, 3], {0}], [[300, 128], [0, 1, 99], {0}],
                               [[300, 128], [-4, 1, 3], {1, 2}], [[300, 128], [0, 1, -1], {0}]):
        c.fresh()
        c.kv_len.copy_(torch.tensor(kv_len))
        c.cu.copy_(torch.tensor(cu))
        c.run()
        torch.cuda.synchronize()
        assert B.device_error() == DATA_ERROR, (kv_len, cu)
        was = c.out.clone()
        if cu == [0, 1, 99]:
            tokens = {0, 1, 2}  # (clamped to the three that there are)
        c.out[2 if cu[2] < 0 else 3:] = 7.0
        at = c.out
        for t in tokens:
            b, i = (0, 0) if t == 0 else (1, t - 1)
            c._token(t, c.kv[c.rows_of[b]].double()[:c.lens[b] - c.n[b] + i + 1], True)
        c.out = was
        assert at is not None
    c.kv_len.copy_(good_len)
    c.cu.copy_(good_cu)
    c.fresh()
    c.run()
    ok()
    c.check()


def test_refusals(cuda_lib):
    c = Case([1, 2], [300, 128], 16, 64, seed=8)
    ws = c.run()
    ok()
    for kw in ({"n_q": 2, "cu_tokens": None}, {"block_size": 24}, {"block_size": 0}, {"sink": torch.zeros(15, device=DEV)},
               {"lse": c.lse[:, :8]}, {"cu_tokens": c.cu.long()}, {"block_table": c.table.cpu()}, {"block_size": 2 ** 32 + 64}):
        with pytest.raises(B.DSAError):
            c.run(**kw)
    for field, value in (("q", c.q[:, :, ::2]), ("kv", c.kv.float()), ("out", c.out[:1]), ("scale", 0.0),
                         ("scale", math.inf), ("kv_len", c.kv_len[:1]), ("kv", c.kv[:0])):
        kept = getattr(c, field)
        setattr(c, field, value)
        with pytest.raises(B.DSAError):
            c.run()
        setattr(c, field, kept)
    c.table, kept = None, c.table
    with pytest.raises(B.DSAError):  # a contiguous cache of that length has more rows
        c.L = 10 ** 6
        c.run()
    c.table, c.L = kept, kept.shape[1] * 64
    with pytest.raises(B.DSAError):
        B.dsa_latent_attn(c.args(), ws[:-256])
    with pytest.raises(B.DSAError):
        B.dsa_latent_attn(c.args(), ws[8:])
    ok()
    c.T, c.q, c.out, c.lse = 0, c.q[:0], c.out[:0], c.lse[:0]
    c.run()
    ok()


def test_the_same_bits_again_over_a_workspace_of_nan(cuda_lib):
    c = Case([2, 1, 3], [3000, 64, 700], 128, 64, seed=11)
    ws = c.run()
    ok()
    first = c.out.clone(), c.lse.clone()
    ws.view(torch.float32).fill_(NAN)
    c.fresh()
    c.run(ws)
    ok()
    assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


def test_a_captured_call_follows_the_lengths(cuda_lib):
    """A graph of two calls on one workspace, replayed after the lengths and the
    counts have changed."""
    c = Case([1, 2, 1], [900, 300, 2000], 128, 64, pad=1, seed=12)
    d = Case([4], [5000], 16, 16, seed=13)
    need = max(B.workspace_bytes("latent_attn", c.args()), B.workspace_bytes("latent_attn", d.args()))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    ca, da = c.args(), d.args()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.dsa_latent_attn(ca, ws)
        B.dsa_latent_attn(da, ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.dsa_latent_attn(ca, ws)
        B.dsa_latent_attn(da, ws)
    for n, lens in (([1, 2, 1], [900, 300, 2000]), ([0, 1, 2], [900, 299, 64]), ([1, 1, 2], [1, 300, 1999])):
        c.n, c.lens = n, lens
        c.cu.copy_(torch.tensor([0, *np.cumsum(n)], dtype=torch.int32))
        c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        rows_of, c.rows_of = c.rows_of, [r[:x] for r, x in zip(c.rows_of, lens)]
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        d.out.fill_(7.0)
        g.replay()
        ok()
        c.check()
        d.check()
        c.rows_of = rows_of


def test_two_streams_at_once(cuda_lib):
    c, d = Case([2], [9000], 128, 64, seed=14), Case([1, 3], [4000, 100], 64, 32, seed=15)
    s, r = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        c.run(stream=s)
        d.run(stream=r)
    ok()
    c.check()
    d.check()


def test_a_cache_past_4_gb(cuda_lib):
    """Rows whose byte offsets need 33 bits, contiguous and paged."""
    rows = (1 << 32) // 1152 + 5000
    big = torch.zeros(rows, 576, dtype=torch.bfloat16, device=DEV)
    c = Case([1, 1], [200, 150], 128, 64, seed=16)
    pages = int(c.table.max()) + 1
    first = rows // 64 - pages
    for b in range(2):
        big[c.rows_of[b] + first * 64] = c.kv[c.rows_of[b]]
    c.table[c.table >= 0] += first
    c.rows_of = [r + first * 64 for r in c.rows_of]
    c.kv = big
    c.run()
    ok()
    c.check()
    c.table, c.page = None, 0
    c.L = rows // 2
    for b in range(2):
        at = b * c.L + torch.arange(c.lens[b], device=DEV)
        big[at] = big[c.rows_of[b]]
        c.rows_of[b] = at
    c.fresh()
    c.run()
    ok()
    c.check()


def test_more_sequences_than_threads(cuda_lib):
    rng = np.random.default_rng(17)
    n = rng.integers(0, 3, 1000).tolist()
    lens = [int(x) for x in rng.integers(0, 200, 1000)]
    c = Case(n, lens, 4, 16, seed=17)
    c.run()
    ok()
    c.check(tokens=set(rng.integers(0, sum(n), 60).tolist()) | {0, sum(n) - 1})
