"""Residual addition and RMS norm on the GPU against a float64 form on the same
inputs, and its refusals.

h = x + residual is exact in float64 and rounded to the residual's type: the
same bits (the fp32 sum of two bf16 or fp16 values, rounded to bf16, could be a
double rounding: the kernel's h is taken for what follows, and checked against
the fp32 sum's).  z = h r gamma: the D squares are summed with at most
D / n + 12 roundings of a partial sum, n the threads of a row (n >= D / 32), each
2^-24 of the sum, which a square root halves; the mean, the root, the reciprocal
and the two products add six more: (D / n + 24) 2^-24 =: e, at most 2^-18.  y adds
half a step of bf16, 2^-8 of itself.  The scale is the largest |z| over 127: e and
one rounding.  A code is rint(z / scale): off by one only where z / scale is
within 127 * (2 e + 2^-23) + 2^-16 of a tie."""
import numpy as np
import pytest
import torch

from sparse_attention_prolog_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E = 2.0 ** -18


def ok():
    torch.cuda.synchronize()
    assert B.device_error() == 0


class Case:
    def __init__(self, T, D, x="bf16", res=None, y=True, codes=True, gap=0, pow2=False, eps=1e-6, seed=0, off=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        kind = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
        size = torch.exp(3 * torch.randn(T, 1, device=DEV, generator=g)).clamp(max=500)

        def rows(dtype, values):
            wide = torch.full((T * (D + gap) + off + 8,), 9.0, dtype=dtype, device=DEV)
            t = wide[off:off + T * (D + gap)].view(T, D + gap)[:, :D]
            t.copy_(values)
            return t

        self.T, self.D, self.eps, self.pow2 = T, D, eps, pow2
        self.x = rows(kind[x], torch.randn(T, D, device=DEV, generator=g) * size)
        self.gamma = 1 + 0.3 * torch.randn(D, device=DEV, generator=g)
        self.res = rows(kind[res], torch.randn(T, D, device=DEV, generator=g)) if res else None
        self.res_out = rows(kind[res], torch.zeros(T, D, device=DEV)) if res else None
        self.y = torch.full((T, D), 9.0, dtype=torch.bfloat16, device=DEV) if y else None
        self.codes = torch.full((T, D), 99, dtype=torch.int8, device=DEV) if codes else None
        self.scale = torch.full((T,), 9.0, device=DEV) if codes else None

    def run(self, stream=None):
        B.dsa_add_rmsnorm(self.x, self.gamma, self.eps, self.res, self.res_out, self.y, self.codes, self.scale, self.pow2,
                          stream)

    def check(self, res=None):
        ok()
        h = self.x.float()
        if self.res is not None:
            h = (h + (self.res if res is None else res).float()).to(self.res.dtype)
            assert torch.equal(self.res_out, h)
        h = h.double()
        z = h / (h.square().mean(1, keepdim=True) + self.eps).sqrt() * self.gamma.double()
        if self.y is not None:
            off = (self.y.double() - z).abs()
            assert bool((off <= z.abs() * (E + 2.0 ** -8) + 2.0 ** -133).all())
        if self.codes is None:
            return
        scale = z.abs().amax(1) / 127
        got = self.scale.double()
        if self.pow2:
            m, e = np.frexp(scale.cpu().numpy())
            p = torch.from_numpy(np.ldexp(1.0, np.where(m == 0.5, e - 1, e)) * (m > 0)).to(DEV)
            edge = ((scale / p.clamp(min=1e-300)).log2().abs() < 2 * E) | ((2 * scale / p.clamp(min=1e-300)).log2().abs() < 2 * E)
            assert bool(((got == p) | edge).all())
        else:
            assert bool(((got - scale).abs() <= scale * (E + 2.0 ** -23) + 2.0 ** -149).all())
        assert bool((self.codes.int().abs() <= 127).all())
        s = got[:, None]
        t = torch.where(s > 0, z / torch.where(s > 0, s, 1.0), 0.0)
        near = 127 * (2 * E + 2.0 ** -23) + 2.0 ** -16
        assert bool(((self.codes.double() - t).abs() <= 0.5 + near).all())


@pytest.mark.parametrize("T,D", [(1, 1), (1, 7), (3, 8), (5, 64), (9, 255), (8, 256), (7, 257), (17, 264), (2, 1000),
                                 (33, 1536), (8, 7168), (3, 8191), (2, 8192), (2, 8200), (3, 16384), (1, 16385), (2, 20000),
                                 (2, 32767), (2, 32768), (700, 7168), (2000, 64)])
@pytest.mark.parametrize("x,res", [("bf16", None), ("bf16", "bf16"), ("fp16", "fp32"), ("fp16", "bf16"), ("bf16", "fp32")])
def test_shapes_and_types(T, D, x, res, cuda_lib):
    c = Case(T, D, x, res, seed=T + D)
    c.run()
    c.check()


@pytest.mark.parametrize("y,codes,pow2", [(True, False, False), (False, True, False), (False, True, True), (True, True, True)])
@pytest.mark.parametrize("D", [100, 7168])
def test_outputs(y, codes, pow2, D, cuda_lib):
    c = Case(50, D, "bf16", "bf16", y=y, codes=codes, pow2=pow2, seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("gap,off", [(8, 0), (1, 0), (64, 8), (8, 1), (0, 1), (3, 3), (0, 4)])
@pytest.mark.parametrize("x,res", [("bf16", "bf16"), ("fp16", "fp32")])
def test_strides_and_alignment(gap, off, x, res, cuda_lib):
    for D in (1536, 40):
        c = Case(11, D, x, res, gap=gap, off=off, seed=gap + off)
        c.run()
        c.check()
        for t in (c.x, c.res, c.res_out):
            if gap:
                assert bool((t.as_strided((10, gap), (D + gap, 1), t.storage_offset() + D) == 9.0).all())


@pytest.mark.parametrize("D,res", [(7168, "bf16"), (7168, "fp32"), (999, "bf16"), (999, "fp32"), (64, "bf16")])
def test_the_residual_in_place(D, res, cuda_lib):
    c = Case(40, D, "bf16", res, seed=5)
    before = c.res.clone()
    c.res_out = c.res
    c.run()
    c.check(res=before)


def test_rows_of_zeros_and_of_one_value(cuda_lib):
    for eps in (1e-6, 1.0):
        c = Case(6, 512, "bf16", "bf16", eps=eps)
        c.x[1:4] = 0
        c.res[1:3] = 0
        c.res[3] = 2.0
        c.x[5] = -c.res[5]
        c.run()
        c.check()
        assert c.scale[1] == 0 and c.scale[5] == 0 and bool((c.codes[[1, 2, 5]] == 0).all()) and bool((c.y[1] == 0).all())
    c = Case(2, 512, "bf16", None, eps=0.0)
    c.run()
    c.check()


def test_values_of_every_size(cuda_lib):
    """Rows whose squares stay within fp32, down to bf16 subnormals beside them (eps
    hides a row of those alone)."""
    c = Case(5, 1024, "bf16", "fp32", eps=1e-12)
    c.x[0] *= 1e-20
    c.res[0] *= 1e-20
    c.x[1] = c.x[1].sign() * 1e17
    c.x[2, ::2] = 1e-39
    c.res[2, ::2] = 0
    c.x[3] = 0
    c.x[3, 7] = 300.0
    c.res[3] = 0
    c.run()
    c.check()
    assert c.codes[3, 7].abs() == 127 and int((c.codes[3] != 0).sum()) == 1


def test_values_that_are_not_finite(cuda_lib):
    """Such a row has codes 0 and a scale that is not finite, and touches no other."""
    for D in (512, 500, 64, 8192):
        c = Case(9, D, "bf16", "bf16")
        c.x[2, 5] = float("nan")
        c.res[4, D - 1] = float("inf")
        c.x[6, 0] = float("-inf")
        c.run()
        ok()
        for r in (2, 4, 6):
            assert not torch.isfinite(c.scale[r]) and bool((c.codes[r] == 0).all()) and bool(c.y[r].isnan().any())
        keep = [0, 1, 3, 5, 7, 8]
        for name in ("x", "res", "res_out", "y", "codes", "scale"):
            setattr(c, name, getattr(c, name)[keep])
        c.check()


def test_many_rows(cuda_lib):
    """More rows than a grid's second dimension could hold, sampled."""
    c = Case(200000, 24, "fp16", "bf16", seed=8)
    c.run()
    c.check()


def test_captured_and_on_another_stream(cuda_lib):
    c = Case(8, 7168, "bf16", "bf16", seed=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    torch.cuda.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for k in range(3):
        c.x.copy_(torch.randn(8, 7168, device=DEV))
        g.replay()
        c.check()


def test_feeds_the_int8_gemm(cuda_lib):
    """x (fp16, an int8 GEMM's output) + residual -> codes -> the int8 GEMM: within
    the codes' half step of the product in float64."""
    T, D, N = 40, 1536, 256
    c = Case(T, D, "fp16", "fp32", y=False, seed=10)
    b = torch.randint(-127, 128, (N, D), dtype=torch.int8, device=DEV)
    b_scale = torch.rand(N, device=DEV) / 127 / 40
    out = torch.empty(T, N, dtype=torch.float16, device=DEV)
    c.run()
    B.dsa_int8_gemm(c.codes, c.scale, b, b_scale, out)
    c.check()
    w = b.double() * b_scale.double()[:, None]
    h = c.res_out.double()
    z = h / (h.square().mean(1, keepdim=True) + c.eps).sqrt() * c.gamma.double()
    bound = 0.51 * c.scale.double()[:, None] * w.abs().sum(1) + 2.0 ** -11 * (z @ w.T).abs() + 2.0 ** -24
    assert bool(((out.double() - z @ w.T).abs() <= bound * (1 + 2.0 ** -10)).all())


def test_refusals(cuda_lib):
    def bad(change):
        c = Case(4, 64, "bf16", "bf16")
        change(c)
        with pytest.raises(B.DSAError):
            c.run()

    bad(lambda c: setattr(c, "x", c.x.float()))
    bad(lambda c: setattr(c, "x", c.x[:, ::2]))
    bad(lambda c: setattr(c, "x", c.x[:1].expand(4, 64)))
    bad(lambda c: setattr(c, "gamma", c.gamma[:63]))
    bad(lambda c: setattr(c, "gamma", c.gamma.bfloat16()))
    bad(lambda c: setattr(c, "res", None))
    bad(lambda c: setattr(c, "res", c.res.half()))
    bad(lambda c: setattr(c, "res_out", c.res_out.float()))
    bad(lambda c: setattr(c, "scale", None))
    bad(lambda c: setattr(c, "codes", c.codes[:2]))
    bad(lambda c: setattr(c, "y", c.y.cpu()))
    bad(lambda c: setattr(c, "eps", -1.0))
    bad(lambda c: setattr(c, "eps", float("nan")))

    def none(c):
        c.y = c.codes = c.scale = None
    bad(none)
    c = Case(1, 8)
    c.x, c.gamma = torch.zeros(1, 40000, dtype=torch.bfloat16, device=DEV), torch.ones(40000, device=DEV)
    c.y, c.codes = torch.zeros_like(c.x), None
    c.scale = None
    with pytest.raises(B.DSAError):
        c.run()
    ok()
    Case(0, 64, "bf16", "bf16").run()
    ok()
