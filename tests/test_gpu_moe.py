"""Tokens to their experts and back on the GPU, against the definitions in 64 bits.

Bounds, per output, with u = 2^-24 and r half a step of the output's type (bf16 2^-8,
f32 2^-24) of its magnitude:
- the places and the moved rows are exact;
- a sum over S slots and a residual: S + 1 fused roundings, (S + 1) u sum |terms|, and r;
- a router weight's gradient, a sum over n products: each product and each addition
  rounded once, in whatever grouping: (n + 1) u sum |products|;
- dys, one product: r.
"""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield
    assert q2k.device_error() == 0


def host(t):
    return t.to(torch.float64).cpu().numpy()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")
    return t if dtype is None else t.to(dtype)


def reference_route(ids, n_experts):
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < n_experts), flat, n_experts)
    order = np.argsort(key, kind="stable")
    rows = np.empty_like(order)
    rows[order] = np.arange(order.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=n_experts + 1))[:n_experts]])
    return rows.reshape(ids.shape), order, offsets


def make_ids(rng, n_tokens, top_k, n_experts, pad=0.0):
    ids = rng.integers(0, n_experts, (n_tokens, top_k)).astype(np.int32)
    ids[rng.random((n_tokens, top_k)) < pad] = -1
    return ids


def check_route(routes, ids, n_experts):
    for got, want in zip(routes, reference_route(ids, n_experts)):
        assert got.dtype == torch.int32
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("n_tokens,top_k,n_experts,pad", [
    (1, 1, 1, 0), (1, 8, 64, 0), (1, 4, 4, 1.0), (3, 2, 5, 0.5), (31, 1, 7, 0), (33, 1, 2, 0.1),
    (64, 8, 64, 0), (77, 3, 10, 0.3), (512, 8, 64, 0), (511, 8, 1, 0.2), (1025, 7, 256, 0),
    (5000, 8, 2047, 0.1), (5001, 5, 2048, 0.1), (700, 256, 4096, 0.05), (1 << 17, 8, 60, 0.01),
    (4096, 1, 4096, 0)])
def test_route(n_tokens, top_k, n_experts, pad):
    rng = np.random.default_rng([1, n_tokens, top_k, n_experts])
    ids = make_ids(rng, n_tokens, top_k, n_experts, pad)
    routes, bad = q2k.moe_route(dev(ids), n_experts, check=False)
    check_route(routes, ids, n_experts)
    assert int(bad) == 0 and routes.n_experts == n_experts
    check_route(q2k.moe_route(dev(ids), n_experts), ids, n_experts)


def test_route_one_expert_takes_all():
    ids = np.full((300, 4), 5, np.int32)
    check_route(q2k.moe_route(dev(ids), 9), ids, 9)


def test_route_counts_bad_ids():
    ids = np.array([[0, 7], [-1, 3], [-2, 1 << 30], [2, -1 << 31]], np.int32)
    routes, bad = q2k.moe_route(dev(ids), 7, check=False)
    assert int(bad) == 4
    check_route(routes, ids, 7)
    with pytest.raises(q2k.InvalidArgument, match="4 expert id"):
        q2k.moe_route(dev(ids), 7)
    many = np.full((3000, 8), 99, np.int32)
    assert int(q2k.moe_route(dev(many), 64, check=False)[1]) == 24000


MOVES = [(1, 8, 64, 7168, 0), (1, 1, 1, 1, 0), (5, 2, 3, 33, 0.3), (77, 3, 10, 1001, 0.2),
         (64, 8, 64, 256, 0), (130, 6, 17, 2050, 0.1), (9, 11, 4, 520, 0.4), (40, 4, 8, 4100, 1.0),
         (300, 8, 60, 7168, 0.1), (2, 20, 7, 14336, 0),
         # words of every size, one row of them more or less than a CTA's or a cluster's
         (1, 2, 9, 14335, 0), (3, 1, 4, 2047, 0), (3, 4, 9, 2049, 0.2), (6, 5, 9, 4097, 0.2),
         (2, 3, 9, 14334, 0.3), (400, 2, 5, 2046, 0.1), (400, 1, 5, 4100, 0.1), (401, 4, 5, 513, 0.1),
         (700, 2, 64, 4104, 0.1), (700, 9, 64, 515, 0.1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n_tokens,top_k,n_experts,width,pad", MOVES)
def test_moves(n_tokens, top_k, n_experts, width, pad, dtype):
    rng = np.random.default_rng([2, n_tokens, width])
    ids = make_ids(rng, n_tokens, top_k, n_experts, pad)
    routes = q2k.moe_route(dev(ids), n_experts)
    rows, order, offsets = reference_route(ids, n_experts)
    end, choices = offsets[-1], n_tokens * top_k
    real = (rows < end)[..., None]

    x = dev(rng.standard_normal((n_tokens, width)).astype(np.float32), DT[dtype])
    xs = q2k.moe_sort(x, routes)
    want = host(x)[order // top_k]
    want[end:] = 0
    assert np.array_equal(host(xs), want)

    dxs = dev(rng.standard_normal((choices, width)).astype(np.float32), DT[dtype])
    dxs[end:] = float("nan")  # (never read)
    parts = np.where(real, host(dxs)[rows], 0)
    ref = parts.sum(1)
    bound = (top_k + 1) * U * np.abs(parts).sum(1)
    bound = bound + HALF[dtype] * (np.abs(ref) + bound)
    assert np.all(np.abs(host(q2k.moe_sort_backward(dxs, routes)) - ref) <= bound)

    weights = dev(rng.random((n_tokens, top_k)).astype(np.float32))
    weights[dev(rows >= end)] = float("inf")  # (nor these)
    w = np.where(real, host(weights)[..., None], 0)
    residual = dev(rng.standard_normal((n_tokens, width)).astype(np.float32), DT[dtype])
    for res in (None, residual):
        base = 0 if res is None else host(res)
        ref = base + (w * parts).sum(1)
        bound = (top_k + 1) * U * (np.abs(base) + np.abs(w * parts).sum(1))
        bound = bound + HALF[dtype] * (np.abs(ref) + bound)
        y = q2k.moe_combine(dxs, routes, weights=weights, residual=res)
        assert np.all(np.abs(host(y) - ref) <= bound)

    dy = dev(rng.standard_normal((n_tokens, width)).astype(np.float32), DT[dtype])
    dys, dw = q2k.moe_combine_backward(dy, dxs, routes, weights)
    ref = np.zeros((choices, width))
    ref[rows.reshape(-1)] = (w * host(dy)[:, None]).reshape(choices, width)
    assert np.all(np.abs(host(dys) - ref) <= HALF[dtype] * np.abs(ref))
    products = parts * host(dy)[:, None]
    assert np.all(np.abs(host(dw) - products.sum(-1)) <= (width + 1) * U * np.abs(products).sum(-1))
    again = q2k.moe_combine_backward(dy, dxs, routes, weights)
    assert torch.equal(again[0], dys) and torch.equal(again[1], dw)


def test_gradients_against_differences():
    """<dy, y(ys + d) - y(ys)> and <dy, y(w + d) - y(w)>: y is linear in each."""
    rng = np.random.default_rng(3)
    ids = make_ids(rng, 20, 3, 6, 0.2)
    routes = q2k.moe_route(dev(ids), 6)
    ys, d = (dev(rng.standard_normal((60, 24)).astype(np.float32)) for _ in range(2))
    w, e = (dev(rng.random((20, 3)).astype(np.float32)) for _ in range(2))
    dy = dev(rng.standard_normal((20, 24)).astype(np.float32))
    x, dx = (dev(rng.standard_normal((20, 24)).astype(np.float32)) for _ in range(2))
    dys, dw = q2k.moe_combine_backward(dy, ys, routes, w)

    def dot(a, b):
        return float((a.double() * b.double()).sum())

    base = q2k.moe_combine(ys, routes, weights=w)
    # f32 sums of a few terms of order one: 60 * 24 of them, each within 8 u of terms below 8
    tol = 60 * 24 * 8 * 8 * U
    assert abs(dot(dy, q2k.moe_combine(ys + d, routes, weights=w) - base) - dot(dys, d)) < tol
    assert abs(dot(dy, q2k.moe_combine(ys, routes, weights=w + e) - base) - dot(dw, e)) < tol
    moved = dot(d, q2k.moe_sort(x + dx, routes) - q2k.moe_sort(x, routes))
    assert abs(moved - dot(q2k.moe_sort_backward(d, routes), dx)) < tol


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [1, 2, 3, 4])
def test_rows_off_sixteen_bytes(dtype, shift):
    """Buffers that start `shift` elements into an allocation; what lies around stays."""
    rng = np.random.default_rng([4, shift])
    ids = make_ids(rng, 12, 3, 5, 0.2)
    routes = q2k.moe_route(dev(ids), 5)
    width = 72

    def cut(rows):
        buf = torch.full((rows * width + shift + 5,), 7.0, dtype=DT[dtype], device="cuda:0")
        return buf, buf[shift:shift + rows * width].view(rows, width)

    whole, x = cut(12)
    x.copy_(dev(rng.standard_normal((12, width)).astype(np.float32)))
    wide, xs = cut(36)
    assert q2k.moe_sort(x, routes, out=xs) is xs
    assert torch.equal(xs, q2k.moe_sort(x.clone(), routes))
    back, dx = cut(12)
    q2k.moe_sort_backward(xs, routes, out=dx)
    assert torch.equal(dx, q2k.moe_sort_backward(xs.clone(), routes))
    y = q2k.moe_combine(xs, routes, residual=x)
    assert torch.equal(y, q2k.moe_combine(xs.clone(), routes, residual=x.clone()))
    for buf, rows in ((whole, 12), (wide, 36), (back, 12)):
        assert bool((buf[:shift] == 7).all()) and bool((buf[shift + rows * width:] == 7).all())


def test_infinities_and_nan_pass():
    routes = q2k.moe_route(dev(np.array([[0, 1], [1, -1]], np.int32)), 2)
    ys = torch.ones(4, 8, device="cuda:0")
    ys[0, 0], ys[1, 1] = float("inf"), float("nan")
    w = torch.tensor([[0.5, 2.0], [0.0, 1.0]], device="cuda:0")
    y = host(q2k.moe_combine(ys, routes, weights=w))
    assert y[0, 0] == np.inf and np.isnan(y[0, 1]) and y[0, 2] == 2.5
    assert np.array_equal(y[1], np.zeros(8))
    x = torch.tensor([[float("inf"), -0.0], [float("nan"), 1.0]], device="cuda:0")
    xs = q2k.moe_sort(x, routes)
    assert torch.equal(xs[0].view(torch.int32), x[0].view(torch.int32))


def test_places_out_of_range_are_skipped():
    rows = torch.tensor([[0, 99], [-7, 1 << 30]], dtype=torch.int32, device="cuda:0")
    offsets = torch.tensor([0, 1 << 20], dtype=torch.int32, device="cuda:0")
    routes = q2k.Routes(rows, rows.view(-1), offsets)
    x = torch.randn(2, 16, device="cuda:0")
    out = torch.zeros(4, 16, device="cuda:0")
    q2k.moe_sort(x, routes, out=out)
    assert torch.equal(out[0], x[0]) and not bool(out[1:].any())
    y = q2k.moe_combine(out, routes)
    assert torch.equal(y[0], x[0]) and not bool(y[1].any())
    w = torch.ones(2, 2, device="cuda:0")
    _, dw = q2k.moe_combine_backward(x, out, routes, w)
    assert dw[0, 0] > 0 and not bool(dw.view(-1)[1:].any())


def test_streams_and_graphs():
    """On a side stream, and captured once and replayed on new contents."""
    rng = np.random.default_rng(5)
    n_tokens, top_k, n_experts, width = 50, 4, 12, 320
    ids = dev(make_ids(rng, n_tokens, top_k, n_experts))
    x = dev(rng.standard_normal((n_tokens, width)).astype(np.float32))
    w = dev(rng.random((n_tokens, top_k)).astype(np.float32))

    def path():
        routes, _ = q2k.moe_route(ids, n_experts, check=False)
        xs = q2k.moe_sort(x, routes)
        y = q2k.moe_combine(xs, routes, weights=w, residual=x)
        dys, dw = q2k.moe_combine_backward(y, xs, routes, w)
        return y, dys, dw, q2k.moe_sort_backward(dys, routes)

    want = path()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = path()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = path()
    ids.copy_(dev(make_ids(rng, n_tokens, top_k, n_experts, 0.3)))
    x.copy_(dev(rng.standard_normal((n_tokens, width)).astype(np.float32)))
    want = path()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_python_refuses():
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda:0")
    routes = q2k.moe_route(ids, 3)
    x = torch.zeros(4, 8, device="cuda:0")
    for bad, err in ((ids.long(), TypeError), (ids.view(-1), ValueError), (ids.t(), ValueError),
                     (ids[:0], q2k.InvalidArgument)):
        with pytest.raises(err):
            q2k.moe_route(bad, 3)
    for n in (0, -1, 4097, 1 << 32):
        with pytest.raises(ValueError, match="n_experts"):
            q2k.moe_route(ids, n)
    for bad, err in ((x.half(), TypeError), (x[:3], ValueError), (x.view(-1), ValueError),
                     (torch.zeros(8, 4, device="cuda:0").t(), ValueError),
                     (x[:, :0].contiguous(), q2k.InvalidArgument), (x.cpu(), TypeError)):
        with pytest.raises(err):
            q2k.moe_sort(bad, routes)
    with pytest.raises(ValueError):
        q2k.moe_sort_backward(x, routes)
    ys = torch.zeros(8, 8, device="cuda:0")
    w = torch.zeros(4, 2, device="cuda:0")
    for kw in ({"weights": w.double()}, {"weights": w.view(2, 4)}, {"residual": x.bfloat16()},
               {"residual": ys}, {"out": ys}, {"out": x.bfloat16()}):
        with pytest.raises((TypeError, ValueError)):
            q2k.moe_combine(ys, routes, **kw)
    with pytest.raises(ValueError):
        q2k.moe_combine_backward(ys, ys, routes, w)
    with pytest.raises(q2k.InvalidArgument, match="alias"):
        q2k.moe_combine(ys, routes, residual=x, out=x)
    with pytest.raises(TypeError):
        q2k.moe_sort(x, q2k.Routes(ids.long(), ids.view(-1), routes.offsets))
