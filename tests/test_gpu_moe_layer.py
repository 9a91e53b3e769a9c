"""A mixture-of-experts feed-forward layer as a user runs it (route, sort, the experts'
gated block and down projection, combine onto the residual; and backwards) against its
formula in 64 bits, and how its calls behave together: in graphs, on several streams at
once, through ctypes, with bad rows and weights, and past 32-bit offsets.

The layer's bounds follow the rounding through it.  Every step's inputs are the outputs
of the step before as they are (rounded), so that each step is checked by itself with
the bounds of test_gpu_moe and test_gpu_linear.
"""

import threading

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import U16, act, blocks, decoded, dev, host, slope
from test_gpu_moe import make_ids, reference_route

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


def bf16(rng, *shape, scale=1.0):
    return dev((scale * rng.standard_normal(shape)).astype(np.float32), torch.bfloat16)


class Layer:
    """Experts of `inner` x `hidden` gated blocks and their down projections with biases."""

    def __init__(self, rng, experts, hidden, inner):
        self.experts, self.hidden, self.inner = experts, hidden, inner
        self.gate, self.up = ([blocks(rng, inner, hidden) for _ in range(experts)] for _ in range(2))
        self.down = [blocks(rng, hidden, inner) for _ in range(experts)]
        self.wg, self.wu, self.wd = (dev(np.concatenate(w)) for w in (self.gate, self.up, self.down))
        self.bias = dev(rng.standard_normal((experts, hidden)).astype(np.float32))

    def forward(self, x, ids, weights):
        routes, bad = q2k.moe_route(ids, self.experts, check=False)
        xs = q2k.moe_sort(x, routes)
        h, gate, up = q2k.gated_ffn(xs, self.wg, self.wu, self.inner, save=True, routes=routes)
        ys = q2k.linear(h, self.wd, self.hidden, bias=self.bias, routes=routes)
        y = q2k.moe_combine(ys, routes, weights=weights, residual=x)
        return y, (routes, xs, gate, up, h, ys, bad)

    def backward(self, dy, weights, kept):
        routes, _, gate, up, _, ys, _ = kept
        dys, dweights = q2k.moe_combine_backward(dy, ys, routes, weights)
        dh, _, dbias = q2k.linear_backward(dys, self.wd, self.inner, bias=True, routes=routes)
        dxs, dgate, dup = q2k.gated_ffn_backward(dh, gate, up, self.wg, self.wu, self.hidden,
                                                 routes=routes)
        dx = q2k.moe_sort_backward(dxs, routes)
        return dx, dweights, dbias, (dys, dh, dgate, dup, dxs)


def ok(got, ref, bound, what):
    err = np.abs(host(got) - ref)
    assert np.all(err <= bound + 1e-30), f"{what}: {np.max(err / np.maximum(bound, 1e-300)):.2f}"


@pytest.mark.parametrize("n_tokens,top_k,experts,hidden,inner,pad", [
    (1, 2, 8, 512, 256, 0), (5, 3, 4, 256, 512, 0.2), (70, 2, 6, 512, 768, 0.1),
    (150, 4, 5, 1024, 512, 0.3), (9, 2, 3, 256, 256, 1.0), (400, 2, 3, 1024, 256, 0)])
def test_layer(n_tokens, top_k, experts, hidden, inner, pad):
    rng = np.random.default_rng([1, n_tokens, hidden])
    layer = Layer(rng, experts, hidden, inner)
    ids = make_ids(rng, n_tokens, top_k, experts, pad)
    x, dy = bf16(rng, n_tokens, hidden), bf16(rng, n_tokens, hidden, scale=0.1)
    weights = dev(rng.random((n_tokens, top_k)).astype(np.float32))
    y, kept = layer.forward(x, dev(ids), weights)
    routes, xs, gate, up, h, ys, bad = kept
    dx, dweights, dbias, (dys, dh, dgate, dup, dxs) = layer.backward(dy, weights, kept)
    rows, order, offsets = reference_route(ids, experts)
    end, token = offsets[-1], order // top_k
    assert int(bad) == 0
    assert np.array_equal(host(xs)[:end], host(x)[token[:end]])
    for e in range(experts):
        s = slice(offsets[e], offsets[e + 1])
        if s.start == s.stop:
            continue
        wg, wu = decoded(layer.gate[e], inner, hidden)[0], decoded(layer.up[e], inner, hidden)[0]
        wd = decoded(layer.down[e], hidden, inner)[0]
        a, hv = host(xs)[s], host(h)[s]
        for got, w in ((gate, wg), (up, wu)):
            ref = a @ w.T
            ok(got[s], ref, 8e-3 * (np.abs(a) @ np.abs(w).T) + U16 * np.abs(ref) * 1.01, "projection")
        # h from the projections before they are rounded: two half steps and the slope's 1.13
        g, u = host(gate)[s], host(up)[s]
        ok(h[s], act(g, "silu") * u,
           U16 * (1.13 * np.abs(g * u) + 2.1 * np.abs(act(g, "silu") * u)) + 1e-6, "h")
        ref = hv @ wd.T + host(layer.bias)[e]
        ok(ys[s], ref, 8e-3 * (np.abs(hv) @ np.abs(wd).T) + U16 * np.abs(ref) * 1.01 + 1e-6, "ys")
        d = host(dys)[s]
        ref = d @ wd
        ok(dh[s], ref, 8e-3 * (np.abs(d) @ np.abs(wd)) + U16 * np.abs(ref) * 1.01, "dh")
        ok(dbias[e], d.sum(0), (len(d) + 1) * U * np.abs(d).sum(0), "dbias")
        dhv = host(dh)[s]
        ok(dgate[s], dhv * u * slope(g, "silu"),
           U16 * np.abs(dhv * u * slope(g, "silu")) + 1e-5 * np.abs(dhv * u), "dgate")
        ok(dup[s], dhv * act(g, "silu"), U16 * np.abs(dhv * act(g, "silu")) + 1e-5 * np.abs(dhv * g), "dup")
        dg, du = host(dgate)[s], host(dup)[s]
        ref = dg @ wg + du @ wu
        ok(dxs[s], ref, 8e-3 * (np.abs(dg) @ np.abs(wg) + np.abs(du) @ np.abs(wu))
           + U16 * np.abs(ref) * 1.01, "dxs")
    real = (rows < end)[..., None]
    w = np.where(real, host(weights)[..., None], 0)
    parts = np.where(real, host(ys)[rows], 0)
    ref = host(x) + (w * parts).sum(1)
    e = (top_k + 1) * U * (np.abs(host(x)) + np.abs(w * parts).sum(1))
    ok(y, ref, e + U16 * (np.abs(ref) + e), "y")
    products = parts * host(dy)[:, None]
    ok(dweights, products.sum(-1), (hidden + 1) * U * np.abs(products).sum(-1), "dweights")
    parts = np.where(real, host(dxs)[rows], 0)
    e = (top_k + 1) * U * np.abs(parts).sum(1)
    ok(dx, parts.sum(1), e + U16 * (np.abs(parts.sum(1)) + e), "dx")
    if pad == 1.0:
        assert torch.equal(y, x) and not bool(dx.any()) and not bool(dweights.any())


def finished(layer, out):
    """What a caller reads of a step: y, the gradients, and the rows that have an expert."""
    y, kept, back = out
    end = int(kept[0].offsets[-1])
    return [y, *kept[0], kept[1], *(t[:end] for t in kept[2:6]), *back[:3], *(t[:end] for t in back[3])]


def step(layer, x, ids, weights, dy):
    y, kept = layer.forward(x, ids, weights)
    return y, kept, layer.backward(dy, weights, kept)


def inputs(rng, layer, n_tokens, top_k, pad=0.1):
    return [bf16(rng, n_tokens, layer.hidden), dev(make_ids(rng, n_tokens, top_k, layer.experts, pad)),
            dev(rng.random((n_tokens, top_k)).astype(np.float32)),
            bf16(rng, n_tokens, layer.hidden, scale=0.1)]


@pytest.mark.parametrize("n_tokens,top_k,experts", [(2, 2, 16), (60, 3, 4), (300, 2, 2)])
def test_graph_replays_with_other_routes(n_tokens, top_k, experts):
    rng = np.random.default_rng([2, n_tokens])
    layer = Layer(rng, experts, 512, 512)
    args = inputs(rng, layer, n_tokens, top_k)
    step(layer, *args)
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(layer, *args)
    with torch.cuda.graph(other):
        held_too = step(layer, *args)
    for pad in (0.0, 0.5, 1.0):
        for a, b in zip(args, inputs(rng, layer, n_tokens, top_k, pad)):
            a.copy_(b)
        want = finished(layer, step(layer, *args))
        for _ in range(3):
            graph.replay()
            other.replay()
        torch.cuda.synchronize()
        for out in (held, held_too):
            assert all(torch.equal(p, q) for p, q in zip(finished(layer, out), want))


def test_threads_and_streams():
    rng = np.random.default_rng(3)
    layers = [Layer(rng, 4, 512, 256), Layer(rng, 3, 256, 768)]
    work = [(layer, inputs(rng, layer, n, k)) for layer, n, k in
            zip(layers * 3, (1, 7, 40, 90, 200, 300), (2, 1, 3, 2, 4, 2))]
    torch.cuda.synchronize()
    results, errors, start = [None] * 6, [], threading.Barrier(6)

    def worker(i):
        try:
            stream = torch.cuda.Stream()
            start.wait(30)
            with torch.cuda.stream(stream):
                for _ in range(10):
                    out = [step(layer, *args) for layer, args in work[i:] + work[:i]]
            stream.synchronize()
            results[i] = out
        except Exception as e:  # noqa: BLE001 (shown by the assertion below)
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors and all(r is not None for r in results)
    alone = [finished(layer, step(layer, *args)) for layer, args in work]
    for i, out in enumerate(results):
        for j, got in enumerate(out):
            at = (i + j) % len(work)
            assert all(torch.equal(p, q) for p, q in zip(finished(work[at][0], got), alone[at]))


def test_through_ctypes(monkeypatch):
    rng = np.random.default_rng(4)
    layer = Layer(rng, 3, 512, 256)
    args = inputs(rng, layer, 33, 2)
    assert q2k._quick()
    want = finished(layer, step(layer, *args))
    monkeypatch.setattr(q2k, "_quick_mod", False)
    got = finished(layer, step(layer, *args))
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    w = dev(blocks(rng, 40, 512))
    x, r = bf16(rng, 6, 512), bf16(rng, 6, 40)
    b = dev(rng.standard_normal(40).astype(np.float32))
    slow = q2k.linear(x, w, 40, bias=b, act="gelu", residual=r, save=True)
    back = q2k.linear_backward(r, w, 512, z=slow[1], act="gelu", bias=True)
    plain = q2k.linear_backward(r, w, 512)
    monkeypatch.undo()
    for p, q in zip(slow + back, q2k.linear(x, w, 40, bias=b, act="gelu", residual=r, save=True)
                    + q2k.linear_backward(r, w, 512, z=slow[1], act="gelu", bias=True)):
        assert torch.equal(p, q)
    again = q2k.linear_backward(r, w, 512)
    assert torch.equal(plain[0], again[0]) and plain[1] is r and again[1] is r and again[2] is None


@pytest.mark.parametrize("off", [4, 8, 12])
@pytest.mark.parametrize("k,n", [(1024, 40), (2304, 37)])
def test_weights_off_sixteen_bytes(k, n, off):
    rng = np.random.default_rng([5, off, k])
    lengths = [3, 0, 20, 50]
    offsets = dev(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32))
    routes = q2k.Routes(offsets[:0], offsets[:0], offsets)
    pool = np.concatenate([blocks(rng, n, k) for _ in lengths])
    hold = torch.zeros(pool.size + 64, dtype=torch.uint8, device="cuda:0")
    w = hold[off:off + pool.size]
    w.copy_(dev(pool))
    x, dy = bf16(rng, 73, k), bf16(rng, 73, n)
    for path in ("gemv", "tensor"):
        assert torch.equal(q2k.linear(x, w, n, path=path, routes=routes),
                           q2k.linear(x, w.clone(), n, path=path, routes=routes))
        for m in (1, 5, 30):
            assert torch.equal(q2k.linear(x[:m], w[:pool.size // 4], n, path=path),
                               q2k.linear(x[:m], w[:pool.size // 4].clone(), n, path=path))
    for a, b in zip(q2k.gated_ffn_backward(dy, dy, dy, w, w, k, routes=routes),
                    q2k.gated_ffn_backward(dy, dy, dy, w.clone(), w.clone(), k, routes=routes)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("path", ["gemv", "tensor"])
@pytest.mark.parametrize("k,n", [(1024, 40), (1280, 37), (4352, 133)])
def test_an_experts_nan_stays_its_own(path, k, n):
    """Weights of NaN and infinity in one expert, NaN in some tokens: the others' results
    are what they are without them."""
    rng = np.random.default_rng([6, k])
    lengths = [5, 40, 7, 70]
    offsets = dev(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32))
    routes = q2k.Routes(offsets[:0], offsets[:0], offsets)
    each = [blocks(rng, n, k) for _ in lengths]
    x, dy = bf16(rng, 122, k), bf16(rng, 122, n)
    clean = dev(np.concatenate(each))
    for bad in (1, 2):
        spoiled = each[bad].reshape(-1, 84).copy()
        spoiled[:, 80:82], spoiled[:, 82:84] = [0, 0x7E], [0, 0x7C]  # d NaN, dmin infinity
        w = dev(np.concatenate([*each[:bad], spoiled.reshape(-1), *each[bad + 1:]]))
        keep = np.ones(122, bool)
        keep[offsets[bad]:offsets[bad + 1]] = False
        xn, dn = x.clone(), dy.clone()
        xn[3], xn[60], dn[3], dn[60] = (float("nan"),) * 4
        for tensor in (xn, dn):
            tensor[offsets[bad]:offsets[bad + 1]] = float("inf")
        rows = dev(keep)
        rows[3] = rows[60] = False
        for name, call in (("linear", lambda a, ww: q2k.linear(a, ww, n, path=path, routes=routes)),
                           ("gated", lambda a, ww: q2k.gated_ffn(a, ww, ww, n, path=path, routes=routes))):
            got, want = call(xn, w), call(x, clean)
            assert torch.equal(got[rows], want[rows]), name
            assert bool(got[3].isnan().all()), name
        if path == "tensor":
            got = q2k.linear_backward(dn, w, k, bias=True, routes=routes)
            want = q2k.linear_backward(dy, clean, k, bias=True, routes=routes)
            assert torch.equal(got[0][rows], want[0][rows]) and bool(got[0][3].isnan().all())
            # (tokens 3 and 60 are experts 0's and 3's)
            assert torch.equal(got[2][3 - bad], want[2][3 - bad]) and bool(got[2][3].isnan().all())


@pytest.mark.parametrize("kind,down", [("gelu", 0.0), ("silu", 0.0)])
def test_backward_of_infinite_and_nan(kind, down):
    """act'(inf) = 1, act'(-inf) = 0; a NaN passes."""
    w = dev(blocks(np.random.default_rng(7), 8, 256))
    z = torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda:0")
    z[0, 0], z[0, 1], z[0, 2], z[0, 3], z[0, 4] = float("inf"), float("-inf"), float("nan"), 200.0, -200.0
    dy = torch.full_like(z, 3.0)
    _, dz, dbias = q2k.linear_backward(dy, w, 256, z=z, act=kind, bias=True)
    got = host(dz)
    assert got[0, 0] == 3 and got[0, 1] == down and np.isnan(got[0, 2])
    assert got[0, 3] == 3 and got[0, 4] == 0 and np.all(got[1] == 1.5)
    assert np.isnan(host(dbias)[2]) and host(dbias)[0] == 4.5


def test_infinities_in_a_projection():
    rng = np.random.default_rng(8)
    w = dev(blocks(rng, 12, 512))
    for m in (1, 3, 40):
        for dt in (torch.float32, torch.bfloat16):
            x = torch.randn(m, 512, device="cuda:0").to(dt)
            clean = q2k.linear(x, w, 12, act="gelu")
            x[0, 5] = float("nan")
            y = q2k.linear(x, w, 12, act="gelu")
            assert bool(y[0].isnan().all()) and torch.equal(y[1:], clean[1:])
            r = torch.zeros(m, 12, device="cuda:0").to(dt)
            r[0, 1] = float("-inf")
            x[0, 5] = 0
            y = q2k.linear(x, w, 12, residual=r)
            assert float(y[0, 1]) == float("-inf") and bool(y[0, 2:].isfinite().all())


def test_a_pool_past_4_gb():
    """4.8 GB of experts: the first and the last have weights and tokens."""
    rng = np.random.default_rng(9)
    experts, n, k = 500, 7168, 4096
    each = n * (k // 256) * 84
    pool = torch.zeros(experts * each, dtype=torch.uint8, device="cuda:0")
    first, last = (dev(blocks(rng, n, k)) for _ in range(2))
    pool[:each], pool[-each:] = first, last
    offsets = torch.full((experts + 1,), 3, dtype=torch.int32, device="cuda:0")
    offsets[0], offsets[-1] = 0, 43
    routes = q2k.Routes(offsets[:0], offsets[:0], offsets)
    x = bf16(rng, 43, k)
    whole = [q2k.dequantize(w).view(n, k).double() for w in (first, last)]
    where = (slice(0, 3), slice(3, 43))
    for path in ("gemv", "tensor"):
        y = q2k.linear(x, pool, n, path=path, routes=routes)
        h, gate, up = q2k.gated_ffn(x, pool, pool, n, save=True, path=path, routes=routes)
        assert torch.equal(gate, up) and bool(h.isfinite().all())
        for part, w, wf in zip(where, (first, last), whole):
            a = x[part].double()
            ref, bound = a @ wf.T, 8e-3 * (a.abs() @ wf.abs().T)
            if path == "gemv":  # the exact weights' bound, of the first and last rows
                bytes_of = 64 * (k // 256) * 84
                parts = [torch.from_numpy(decoded(v.cpu().numpy(), 64, k)[1]).to("cuda:0")
                         for v in (w[:bytes_of], w[-bytes_of:])]
                cols = torch.cat([torch.arange(64), torch.arange(n - 64, n)]).to("cuda:0")
                ref, bound = ref[:, cols], 1e-5 * (a.abs() @ torch.cat(parts).T)
            for got in (y, gate):
                got = got[part].double() if path == "tensor" else got[part][:, cols].double()
                assert bool(((got - ref).abs() <= bound + U16 * (ref.abs() + bound)).all())
    dy = bf16(rng, 43, n, scale=0.1)
    dx, _, dbias = q2k.linear_backward(dy, pool, k, bias=True, routes=routes)
    for part, wf, at in zip(where, whole, (0, experts - 1)):
        d = dy[part].double()
        ref, bound = d @ wf, 8e-3 * (d.abs() @ wf.abs())
        assert bool(((dx[part].double() - ref).abs() <= bound + U16 * (ref.abs() + bound)).all())
        assert bool(((dbias[at].double() - d.sum(0)).abs() <= 41 * U * d.abs().sum(0)).all())
    assert not bool(dbias[1:-1].any())


def test_rows_past_2_31():
    rng = np.random.default_rng(10)
    n_tokens, top_k, width = 50000, 6, 7168
    ids = dev(make_ids(rng, n_tokens, top_k, 9))
    routes = q2k.moe_route(ids, 9)
    x = torch.randn(n_tokens, width, dtype=torch.bfloat16, device="cuda:0")
    xs = q2k.moe_sort(x, routes)
    assert xs.numel() > 2 ** 31
    for at in (0, 149999, 299998, 299999):
        assert torch.equal(xs[at], x[int(routes.order[at]) // top_k])
    w = torch.rand(n_tokens, top_k, device="cuda:0")
    y = q2k.moe_combine(xs, routes, weights=w)
    dys, dw = q2k.moe_combine_backward(y, xs, routes, w)
    for t in (0, 31234, n_tokens - 1):
        ref = float(w[t].double().sum()) * x[t].double()
        assert bool(((y[t].double() - ref).abs() <= (U16 + 8 * U) * ref.abs()).all())
        ref = w[t, 2].double() * y[t].double()
        assert bool(((dys[routes.rows[t, 2]].double() - ref).abs() <= U16 * ref.abs()).all())
        ref = (y[t].double() * x[t].double()).sum()
        assert abs(float(dw[t, 5] - ref)) <= (width + 1) * U * float((y[t].double() * x[t].double()).abs().sum())


def test_results_past_2_31():
    """300000 rows of 7200 results, the last expert's checked."""
    rng = np.random.default_rng(11)
    m, n, k, experts = 300000, 7200, 256, 5
    w = [blocks(rng, 64, k) for _ in range(experts)]
    pool = dev(np.concatenate([np.resize(v.reshape(64, -1), (n, 84)).reshape(-1) for v in w]))
    offsets = dev(np.array([0, 100000, 100000, 200001, 299900, m - 7], np.int32))
    routes = q2k.Routes(offsets[:0], offsets[:0], offsets)
    x = torch.randn(m, k, dtype=torch.bfloat16, device="cuda:0")
    y = q2k.linear(x, pool, n, act="silu", routes=routes)
    assert y.numel() > 2 ** 31
    for e, part in ((0, slice(0, 3)), (2, slice(199990, 200001)), (3, slice(200001, 200010)), (4, slice(m - 20, m - 7))):
        a, wf = host(x[part]), decoded(w[e], 64, k)[0]
        z = a @ wf.T
        ez = 8e-3 * (np.abs(a) @ np.abs(wf).T)
        ref = act(z, "silu")
        for c in (0, 64 * 56, 64 * 112):
            got = host(y[part][:, c:c + 64])[:, :64]
            cols = got.shape[1]
            bound = (1.13 * ez + U16 * (np.abs(ref) + 1.13 * ez))[:, :cols]
            assert np.all(np.abs(got - ref[:, :cols]) <= bound + 1e-6)


def test_python_refuses():
    rng = np.random.default_rng(12)
    w, w3 = dev(blocks(rng, 8, 256)), dev(blocks(rng, 24, 256))
    x, r = bf16(rng, 20, 256), bf16(rng, 20, 8)
    b = torch.zeros(8, device="cuda:0")
    routes = q2k.moe_route(torch.zeros(10, 2, dtype=torch.int32, device="cuda:0"), 3)
    bad = [dict(bias=b.double()), dict(bias=b[:7]), dict(bias=b.bfloat16()), dict(residual=r.float()),
           dict(residual=r[:19]), dict(residual=r.t()), dict(out=r.float()), dict(routes=routes, bias=b),
           dict(act="relu"), dict(path="fast"), dict(workspace=r)]
    for kw in bad:
        with pytest.raises((TypeError, ValueError, KeyError)):
            q2k.linear(x, w3 if "routes" in kw else w, 8, **kw)
    with pytest.raises(q2k.InvalidArgument, match="w has"):
        q2k.linear(x, w, 8, routes=routes)
    with pytest.raises(q2k.InvalidArgument, match="w has"):
        q2k.linear(x, w3, 8)
    with pytest.raises(q2k.InvalidArgument, match="w_gate has"):
        q2k.gated_ffn(x, w, w, 8, routes=routes)
    with pytest.raises(q2k.InvalidArgument, match="alias"):
        q2k.linear(x, w, 8, residual=r, out=r)
    with pytest.raises(TypeError):
        q2k.linear(x.half(), w, 8)
    with pytest.raises(TypeError):
        q2k.linear_backward(r.float(), w, 256)
    with pytest.raises((TypeError, ValueError)):
        q2k.linear_backward(r, w, 256, act="gelu")
    with pytest.raises(ValueError):
        q2k.linear_backward(r, w, 256, z=r[:3], act="gelu")
    with pytest.raises(TypeError):
        q2k.linear(x, w3, 8, routes=q2k.Routes(routes.rows, routes.order, routes.offsets.long()))
    with pytest.raises(ValueError):
        q2k.linear(x, w3, 8, routes=q2k.Routes(routes.rows, routes.order, routes.offsets[:1]))
    assert q2k.linear(x, w, 8, out=torch.empty_like(r)).shape == (20, 8)
