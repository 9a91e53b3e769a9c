"""The tensor kernel's divisions of work against 64 bits: cut tiles in every width,
pairs of CTAs, several tiles for a worker, f32 tokens through their image, adapters in
all of them.  (test_ffn_plan asserts the plans named here.)  Matrices repeat ROWS rows,
so that the products in float64 stay small.  Bounds as in test_gpu_ffn; adapters of f32
tokens add the split of t, 2^-16, as those of bf16 do."""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import DT, U16, _device, blocks, decoded, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]

ROWS = 64


class Matrix:
    """n rows of Q2_K blocks, ROWS different ones again and again, and those in float64."""

    def __init__(self, n, k, seed):
        w = blocks(np.random.default_rng([91, k, seed]), ROWS, k)
        self.n, self.k = n, k
        self.w = dev(w).repeat(-(-n // ROWS))[:n * (w.size // ROWS)].clone()
        self.f = torch.from_numpy(decoded(w, ROWS, k)[0]).to("cuda:0")

    def times(self, x):
        """x W^T and sum |x w|."""
        at = torch.arange(self.n, device="cuda:0") % ROWS
        return (x @ self.f.T)[:, at], (x.abs() @ self.f.T.abs())[:, at]

    def under(self, dy):
        """dy W and sum |dy w|."""
        pad = torch.nn.functional.pad
        fold = lambda v: pad(v, (0, -self.n % ROWS)).view(len(v), -1, ROWS).sum(1)  # noqa: E731
        return fold(dy) @ self.f, fold(dy.abs()) @ self.f.abs()


def randn(gen, *shape, scale=1.0):
    return scale * torch.randn(shape, device="cuda:0", generator=gen)


def within(got, ref, bound, dtype, what):
    r = U16 if dtype == "bf16" else 2.0 ** -24
    err, limit = (got.double() - ref).abs(), bound + r * (ref.abs() + bound) + 1e-30
    worst = float((err / limit).max())
    assert worst <= 1, f"{what}: {worst:.2f} of the bound"


def silu(g):
    return g / (1 + torch.exp(-g))


GATED = [(20, 12000, 16384), (40, 12000, 16384), (100, 12000, 16384), (1024, 5000, 14336),
         (600, 5000, 4096), (300, 300, 1024), (259, 14335, 2816), (100, 12001, 16128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", GATED)
def test_gated(m, n, k, dtype):
    gen = torch.Generator(device="cuda:0").manual_seed(m)
    a, b = Matrix(n, k, 1), Matrix(n, k, 2)
    x = randn(gen, m, k).to(DT[dtype])
    h, g, u = q2k.gated_ffn(x, a.w, b.w, n, save=True)
    (rg, sg), (ru, su) = a.times(x.double()), b.times(x.double())
    eg, eu, rh = 8e-3 * sg, 8e-3 * su, silu(rg) * ru
    within(g, rg, eg, dtype, "gate")
    within(u, ru, eu, dtype, "up")
    eh = 1.13 * eg * (ru.abs() + eu) + silu(rg).abs() * eu + 4 * 2.0 ** -24 * rh.abs()
    within(h, rh, eh, dtype, "h")
    assert torch.equal(h, q2k.gated_ffn(x, a.w, b.w, n))


@pytest.mark.parametrize("m,n,k", [(2048, 14336, 4096), (600, 14336, 4096), (600, 5000, 4096), (1000, 14000, 2816),
                                   (200, 9800, 14336), (601, 5003, 4096)])
def test_backward(m, n, k):
    gen = torch.Generator(device="cuda:0").manual_seed(m)
    a, b = Matrix(n, k, 1), Matrix(n, k, 2)
    dh, g, u = (randn(gen, m, n, scale=s).bfloat16() for s in (0.3, 2.0, 1.5))
    dx, dg, du = q2k.gated_ffn_backward(dh, g, u, a.w, b.w, k)
    # from the dgate and dup that the call returned, as the product reads them
    (r1, s1), (r2, s2) = a.under(dg.double()), b.under(du.double())
    within(dx, r1 + r2, 8e-3 * (s1 + s2), "bf16", "dx")
    gd = g.double()
    p = torch.sigmoid(gd)
    within(du, dh.double() * gd * p, 1e-6 * dh.double().abs() * gd.abs(), "bf16", "dup")
    slope = p + gd * p * (1 - p)
    within(dg, dh.double() * u.double() * slope,
           36 * 8 * 2.0 ** -24 * (dh.double() * u.double()).abs() * (1 + gd.abs()), "bf16", "dgate")


LORA = [("bf16", 1024, 6000, 14336, 16, 5), ("bf16", 1024, 5000, 14336, 16, 5), ("bf16", 512, 14336, 1024, 64, 7), ("bf16", 600, 5000, 4096, 8, 3),
        ("bf16", 300, 9800, 1024, 40, 9), ("bf16", 512, 14336, 4096, 16, 6), ("bf16", 70, 5000, 4096, 128, 20),
        ("f32", 9, 300, 1024, 16, 3), ("f32", 20, 1000, 2816, 8, 4), ("f32", 45, 1003, 1792, 24, 5),
        ("f32", 64, 500, 4096, 256, 2), ("f32", 100, 5000, 4096, 64, 6), ("f32", 300, 300, 1024, 16, 4),
        ("f32", 300, 9800, 1024, 40, 9), ("f32", 600, 5000, 4096, 8, 3), ("f32", 1024, 6000, 14336, 16, 5),
        ("f32", 512, 7168, 7168, 64, 4)]


@pytest.mark.parametrize("order", ["mixed", "segments"])
@pytest.mark.parametrize("dtype,m,n,k,r,na", LORA)
def test_adapters(dtype, m, n, k, r, na, order):
    gen = torch.Generator(device="cuda:0").manual_seed(m)
    w = Matrix(n, k, 1)
    x = randn(gen, m, k).to(DT[dtype])
    a, b = randn(gen, na, r, k, scale=k ** -0.5).bfloat16(), randn(gen, na, n, r, scale=r ** -0.5).bfloat16()
    s = 0.25 + torch.rand(na, device="cuda:0", generator=gen)
    if order == "mixed":
        ids = torch.randint(-1, na, (m,), device="cuda:0", generator=gen, dtype=torch.int32)
        ids[m // 3] = na  # out of range: a zero row
        ids[m - 1] = -7
    else:
        ids = (torch.arange(m, device="cuda:0") * na // m).int()
    y, bad = q2k.matmul_lora(x, w.w, n, a, b, ids, scales=s, check=False)
    xd = x.double()
    ref, total = w.times(xd)
    bound = 8e-3 * total
    c = (k / 32 + 64 + r) * 2.0 ** -24 + 2.0 ** -16
    for i in range(na):
        at = (ids == i).nonzero().view(-1)
        t, tt = xd[at] @ a[i].double().T, xd[at].abs() @ a[i].double().abs().T
        ref[at] += s[i].double() * (t @ b[i].double().T)
        bound[at] += c * s[i].double() * (tt @ b[i].double().abs().T)
    out = (ids < -1) | (ids >= na)
    assert int(bad.item()) == int(out.sum()) == (2 if order == "mixed" else 0)
    assert not y[out].any()
    within(y[~out], ref[~out], bound[~out], dtype, "y")
    assert torch.equal(y, q2k.matmul_lora(x, w.w, n, a, b, ids, scales=s, check=False)[0])
