"""The projection and the products over segments where counts are large: more passes or
tiles than a grid's second dimension holds, thousands of experts; and workspaces of the
caller's.  Bounds as in test_gpu_linear; matrices are small, so that all rows are checked."""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import U16, act, blocks, decoded, dev
from test_gpu_linear import routes_of, takes_rows

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield
    assert q2k.device_error() == 0


def parts(w, n, k):
    """(W, |dl q| + |ml|) in float64 on the device."""
    return [torch.from_numpy(a).to("cuda:0") for a in decoded(w, n, k)]


def check(y, x, w, scale, half, bias=None, residual=None, kind=None):
    """y against act(x W^T + bias) + residual; scale: the path's bound of |x| w."""
    wf, wa = w
    z = x.double() @ wf.T + (0 if bias is None else bias.double())
    ez = scale * (x.double().abs() @ wa.T) + U * z.abs()
    ref = z if kind is None else z / (1 + torch.exp(-z))
    ref = ref + (0 if residual is None else residual.double())
    e = 1.13 * ez + 8 * U * (z.abs() + ref.abs() + (0 if residual is None else residual.double().abs()))
    worst = ((y.double() - ref).abs() / (e + half * (ref.abs() + e) + 1e-30)).max()
    assert float(worst) <= 1, f"{float(worst):.2f} of the bound"


@pytest.mark.parametrize("dtype,m,n,k", [("bf16", 16 * 65535 + 9, 3, 256), ("f32", 8 * 65535 + 13, 5, 2304)])
def test_more_passes_than_a_grid(dtype, m, n, k):
    dt, half = (torch.bfloat16, U16) if dtype == "bf16" else (torch.float32, U)
    w = blocks(np.random.default_rng(1), n, k)
    gen = torch.Generator(device="cuda:0").manual_seed(2)
    x = torch.randn(m, k, device="cuda:0", generator=gen).to(dt)
    r = torch.randn(m, n, device="cuda:0", generator=gen).to(dt)
    b = torch.randn(n, device="cuda:0", generator=gen)
    y, z = q2k.linear(x, dev(w), n, bias=b, act="silu", residual=r, save=True, path="gemv")
    wd = parts(w, n, k)
    check(y, x, wd, 1e-5, half, b, r, "silu")
    check(z, x, wd, 1e-5, half, b)


@pytest.mark.parametrize("path", ["gemv", "tensor"])
@pytest.mark.parametrize("n,k", [(3, 256), (24, 2560)])
def test_more_tiles_than_a_grid(path, n, k):
    """2^20 tokens of two experts, the first with almost all."""
    m = 1 << 20 if k == 256 else 200000
    rng = np.random.default_rng(3)
    each = [blocks(rng, n, k) for _ in range(2)]
    routes, offsets = routes_of([m - 30, 20], 5)
    x = torch.randn(m, k, device="cuda:0").bfloat16()
    y = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda:0")
    q2k.linear(x, dev(np.concatenate(each)), n, out=y, path=path, routes=routes)
    for e in range(2):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        wf, wa = parts(each[e], n, k)
        check(y[lo:hi], x[lo:hi], (wf, wa if path == "gemv" else wf.abs()), 1e-5 if path == "gemv" else 8e-3, U16)
    assert bool((y[:5] == 7).all()) and bool((y[m - 5:] == 7).all())


@pytest.mark.parametrize("path", ["auto", "gemv", "tensor"])
@pytest.mark.parametrize("m", [7, 900, 5000])
def test_thousands_of_experts(path, m):
    experts, n, k = 4096, 9, 256
    rng = np.random.default_rng([4, m])
    w = blocks(rng, experts * n, k)
    ids = rng.integers(0, experts, (m, 1)).astype(np.int32)
    routes = q2k.moe_route(dev(ids), experts)
    x = torch.randn(m, k, device="cuda:0").bfloat16()
    xs = q2k.moe_sort(x, routes)
    b = torch.randn(experts, n, device="cuda:0")
    y = q2k.linear(xs, dev(w), n, bias=b, routes=routes, path=path)
    exact = takes_rows(m, "bf16", experts, path)
    wf, wa = (t.view(experts, n, k) for t in parts(w, experts * n, k))
    whose = dev(np.sort(ids[:, 0]))
    for lo in range(0, m, 1000):
        part = whose[lo:lo + 1000].long()
        a = xs[lo:lo + 1000].double().unsqueeze(-1)
        z = (wf[part] @ a).squeeze(-1) + b[part].double()
        e = ((wa if exact else wf.abs())[part] @ a.abs()).squeeze(-1) * (1e-5 if exact else 8e-3) + U * z.abs()
        assert bool(((y[lo:lo + 1000].double() - z).abs() <= e + U16 * (z.abs() + e)).all())
    dy = torch.randn(m, n, device="cuda:0").bfloat16()
    _, _, dbias = q2k.linear_backward(dy, dev(w), k, bias=True, routes=routes)
    ref = torch.zeros(experts, n, dtype=torch.float64, device="cuda:0").index_add_(0, whose.long(), dy.double())
    top = torch.zeros(experts, n, dtype=torch.float64, device="cuda:0").index_add_(0, whose.long(), dy.double().abs())
    assert bool(((dbias.double() - ref).abs() <= m * U * top).all())


def test_callers_workspace():
    rng = np.random.default_rng(5)
    n, k, m = 40, 1024, 70
    w = dev(np.concatenate([blocks(rng, n, k) for _ in range(3)]))
    routes, _ = routes_of([30, 0, 40], 0)
    x, dy = (torch.randn(m, c, device="cuda:0").bfloat16() for c in (k, n))
    ws = torch.full((1 << 22,), 0xEE, dtype=torch.uint8, device="cuda:0")
    for path in ("gemv", "tensor"):
        for call in (lambda **kw: q2k.linear(x, w, n, routes=routes, path=path, **kw),
                     lambda **kw: q2k.gated_ffn(x, w, w, n, routes=routes, path=path, **kw),
                     lambda **kw: q2k.linear_backward(dy, w, k, z=dy, act="gelu", bias=True, routes=routes, **kw),
                     lambda **kw: q2k.gated_ffn_backward(dy, dy, dy, w, w, k, routes=routes, **kw)):
            want, got = call(), call(workspace=ws)
            for a, b in zip(want if isinstance(want, tuple) else (want,), got if isinstance(got, tuple) else (got,)):
                assert torch.equal(a, b)
            with pytest.raises(q2k.InvalidArgument, match="workspace"):
                call(workspace=None)
            with pytest.raises(q2k.InvalidArgument, match="workspace has 16"):
                call(workspace=ws[:16])
            with pytest.raises(TypeError):
                call(workspace=ws.view(torch.int8))
    plain = q2k.linear(x, w[:w.numel() // 3], n, act="silu")
    assert torch.equal(plain, q2k.linear(x, w[:w.numel() // 3], n, act="silu", workspace=ws))


def test_act_of_the_reference():
    """(the bounds above take silu as z / (1 + e^-z))"""
    z = np.linspace(-9, 9, 19)
    assert np.allclose(act(z, "silu"), z / (1 + np.exp(-z)))
