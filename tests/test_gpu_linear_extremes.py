"""The projection, its gradient and the moves of rows at the largest n, k and width.

Bounds as test_gpu_linear's, with what long sums add: on the exact path c = max(1e-5, k
2^-31) as documented; on the tensor path each step of 16 terms rounds the sum once more in
f32, by at most 2^-22 of the absolute terms.  Matrices are 64 rows again and again, so that
every result is checked."""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import DT, U16, _device, blocks, decoded, dev, slope

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]

U, MOST = 2.0 ** -24, 1 << 20


def matrix(seed, n, k):
    """(n rows of blocks on the device, the distinct rows W and |dl q| + |ml| in float64)."""
    r = min(n, 64)
    w = blocks(np.random.default_rng(seed), r, k)
    wf, wa = (dev(a) for a in decoded(w, r, k))
    return dev(w).repeat(-(-n // r))[:n * (k // 256) * 84].clone(), wf, wa


@pytest.mark.parametrize("dtype,m,n,k", [("bf16", 2, MOST, 256), ("bf16", 40, MOST - 1, 256), ("f32", 1, 1, MOST),
                                         ("f32", 3, 5, MOST), ("bf16", 16, 12, MOST), ("bf16", 20, 5, MOST)])
def test_forward(dtype, m, n, k):
    w, wf, wa = matrix([601, m], n, k)
    gen = torch.Generator(device="cuda:0").manual_seed(m)
    x = torch.randn(m, k, device="cuda:0", generator=gen).to(DT[dtype])
    b = torch.randn(n, device="cuda:0", generator=gen)
    y = q2k.linear(x, w, n, bias=b)
    exact = m <= (16 if dtype == "bf16" else 8)
    each = torch.arange(n, device="cuda:0") % wf.shape[0]
    ref = (x.double() @ wf.T)[:, each] + b.double()
    c = max(1e-5, k * 2.0 ** -31) if exact else 8e-3 + k / 16 * 2.0 ** -22
    e = c * (x.double().abs() @ (wa if exact else wf.abs()).T)[:, each] + U * ref.abs()
    half = U16 if dtype == "bf16" else U
    assert bool(((y.double() - ref).abs() <= e + half * (ref.abs() + e)).all())


@pytest.mark.parametrize("m,n,k,kind", [(3, MOST, 256, "gelu"), (3, MOST - 4, 256, "silu"), (2, MOST - 1, 256, None),
                                        (3, 4, MOST, "gelu"), (70, 12, MOST, None)])
def test_backward(m, n, k, kind):
    w, wf, _ = matrix([602, m], n, k)
    gen = torch.Generator(device="cuda:0").manual_seed(m)
    dy, z = (torch.randn(m, n, device="cuda:0", generator=gen).bfloat16() for _ in range(2))
    dx, dz, dbias = q2k.linear_backward(dy, w, k, z=z, act=kind, bias=True)
    d, s = dy.double(), 0.0
    if kind is not None:
        s = 1e-5 * d.abs()
        d = d * dev(slope(z.double().cpu().numpy(), kind))
    es = s if kind is not None else torch.zeros_like(d)
    assert bool(((dz.double() - d).abs() <= es + U16 * (d.abs() + es)).all())
    bound = es.sum(0) + (m + 1) * U * d.abs().sum(0)
    assert bool(((dbias.double() - d.sum(0)).abs() <= bound).all())

    def through(v):  # sums over the rows that are the same
        rows = wf.shape[0]
        v = torch.nn.functional.pad(v, (0, -n % rows))
        return v.view(m, -1, rows).sum(1)

    ref = through(d) @ wf
    bound = (8e-3 + n / 16 * 2.0 ** -22) * (through(d.abs()) @ wf.abs()) + through(es) @ wf.abs() + U16 * ref.abs()
    assert bool(((dx.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("dtype,width", [("f32", MOST), ("bf16", MOST), ("bf16", MOST - 1), ("f32", MOST - 1)])
def test_moves(dtype, width):
    tokens, top_k, experts = 3, 3, 5
    rng = np.random.default_rng([603, width])
    routes = q2k.moe_route(dev(rng.integers(-1, experts, (tokens, top_k)).astype(np.int32)), experts)
    gen = torch.Generator(device="cuda:0").manual_seed(1)
    x, r, dy = (torch.randn(tokens, width, device="cuda:0", generator=gen).to(DT[dtype]) for _ in range(3))
    ys = torch.randn(tokens * top_k, width, device="cuda:0", generator=gen).to(DT[dtype])
    weights = torch.rand(tokens, top_k, device="cuda:0", generator=gen)
    end, half = int(routes.offsets[-1]), U16 if dtype == "bf16" else U
    order, real = routes.order.long(), torch.arange(tokens * top_k, device="cuda:0") < end
    assert torch.equal(q2k.moe_sort(x, routes), torch.where(real[:, None], x[order // top_k], 0))
    used = (routes.rows < end).double()[..., None]
    parts = used * ys.double()[routes.rows.long()]
    for got, terms in ((q2k.moe_sort_backward(ys, routes), parts),
                       (q2k.moe_combine(ys, routes, weights=weights, residual=r),
                        torch.cat([parts * weights.double()[..., None], r.double()[:, None]], 1))):
        ref, e = terms.sum(1), (top_k + 1) * U * terms.abs().sum(1)
        assert bool(((got.double() - ref).abs() <= e + half * (ref.abs() + e)).all())
    dys, dw = q2k.moe_combine_backward(dy, ys, routes, weights)
    ref = torch.where(real[:, None], weights.view(-1)[order][:, None].double() * dy.double()[order // top_k], 0)
    assert bool(((dys.double() - ref).abs() <= half * ref.abs()).all())
    terms = parts * dy.double()[:, None]
    # (a thread's chain of f32 sums is at most width / 256 long, then the warps', the
    # CTAs' and the cluster's)
    assert bool(((dw.double() - terms.sum(-1)).abs() <= (width / 256 + 64) * U * terms.abs().sum(-1)).all())
