"""The feed-forward operators on the GPU against their formulas in 64 bits.

Weights come from the oracle's decode (exact f32 values); products, activations
and gradients are then taken in float64.  Bounds, per output:

- a projection on the exact-weights path: 1e-5 T, T = sum_k |x| (dl q + ml).
  x is exact (bf16) or within 2^-22 (f32); a block's 17 tensor-core sums lose at
  most 2^-23 each of their absolute terms, the at most 56 blocks and 16 parts
  after them 2^-24 each: (4 + 34 + 72) 2^-24 = 6.6e-6.
- on the tensor path: 8e-3 S, S = sum_k |x w| (x and W rounded to bf16, 2 * 2^-8
  of each product, and f32 sums).
- h = act(g) u from errors eg, eu: 1.13 eg (|u| + eu) + |act(g)| eu (the
  activations' slopes are below 1.13) and 4 2^-24 |h| of its own arithmetic.
- an output in bf16 adds half a unit in its last place: 2^-8 of its magnitude.
- dx: dgate and dup rounded to bf16 and W as above: 8e-3 S over both products.
"""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
import oracle
import q2k_workloads as wl

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U16 = 2.0 ** -8
GELU_C, GELU_A = np.sqrt(2 / np.pi), 0.044715


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield
    assert q2k.device_error() == 0


def blocks(rng, n, k, scale=None):
    """n rows of Q2_K blocks; d and dmin such that projections are of order one."""
    w = wl.random_blocks(rng, n * (k // 256)).reshape(n, k // 256, 84)
    s = 1.5 / (0.43 * np.sqrt(k)) if scale is None else scale
    d = w[..., 80:].copy().view("<f2").astype(np.float64) * s
    w[..., 80:] = d.astype("<f2").view(np.uint8)
    return w.reshape(-1)


def decoded(w, n, k):
    """(W, |dl q| + |ml|) in float64."""
    wf = oracle.dequantize(w).astype(np.float64).reshape(n, k)
    b = w.reshape(n, k // 256, 84)
    dmin = b[..., 82:84].copy().view("<f2").astype(np.float64)
    ml = np.empty((n, k // 256, 256))
    for g in range(16):
        h, j, s = g >> 3, (g >> 1) & 3, g & 1
        at = 128 * h + 32 * j + 16 * s
        ml[..., at:at + 16] = (dmin[..., 0] * (b[..., g] >> 4))[..., None]
    ml = ml.reshape(n, k)
    return wf, np.abs(wf + ml) + np.abs(ml)


def act(g, kind):
    with np.errstate(over="ignore"):
        if kind == "silu":
            return g / (1 + np.exp(-g))
        return 0.5 * g * (1 + np.tanh(GELU_C * (g + GELU_A * g ** 3)))


def slope(g, kind):
    if kind == "silu":
        p = 1 / (1 + np.exp(-g))
        return p + g * p * (1 - p)
    t = np.tanh(GELU_C * (g + GELU_A * g ** 3))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * GELU_C * (1 + 3 * GELU_A * g * g)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.to(torch.float64).cpu().numpy()


def activations(rng, m, k, dtype, scale=1.0):
    """(device tensor, the same values in float64)."""
    t = dev((scale * rng.standard_normal((m, k))).astype(np.float32), dtype)
    return t, host(t)


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def projection(x, w, n, path):
    """(x W^T, its bound before any output rounding)."""
    k = x.shape[1]
    wf, parts = decoded(w, n, k)
    bound = 1e-5 * (np.abs(x) @ parts.T) if path == "gemv" else 8e-3 * (np.abs(x) @ np.abs(wf).T)
    return x @ wf.T, bound


def gated_reference(x, wg, wu, n, kind, path, dtype):
    g, eg = projection(x, wg, n, path)
    u, eu = projection(x, wu, n, path)
    r = U16 if dtype == "bf16" else 2.0 ** -24
    h = act(g, kind) * u
    eh = 1.13 * eg * (np.abs(u) + eu) + np.abs(act(g, kind)) * eu + 4 * 2.0 ** -24 * np.abs(h)
    return (h, eh + r * (np.abs(h) + eh)), (g, eg + r * (np.abs(g) + eg)), (u, eu + r * (np.abs(u) + eu))


def close(got, ref_bound, what):
    ref, bound = ref_bound
    err = np.abs(host(got) - ref)
    worst = np.max(err / np.maximum(bound, 1e-300))
    assert np.all(err <= bound + 1e-30), f"{what}: {worst:.2f} of the bound"


# m: one token, the paths' edges, ragged and whole tiles; n: one row, odd, off the
# tiles of 16 and 64 rows; k: one block, odd block counts (rows that start 4, 8 or
# 12 bytes off 16), whole TMA rows, more blocks than warps
GATED = [
    ("f32", 1, 1, 256, "silu"), ("f32", 1, 33, 1024, "gelu"), ("f32", 2, 97, 768, "silu"),
    ("f32", 5, 64, 2816, "silu"), ("f32", 8, 31, 4352, "gelu"),
    ("bf16", 1, 16, 256, "silu"), ("bf16", 3, 130, 1280, "gelu"), ("bf16", 8, 65, 14336, "silu"),
    ("bf16", 9, 48, 8192, "silu"), ("bf16", 16, 200, 4352, "gelu"),
    ("bf16", 17, 64, 1024, "silu"), ("bf16", 33, 63, 768, "gelu"), ("bf16", 64, 129, 2048, "silu"),
    ("bf16", 65, 1, 1024, "silu"), ("bf16", 128, 191, 2816, "gelu"), ("bf16", 129, 70, 256, "silu"),
    ("bf16", 256, 65, 1024, "silu"), ("bf16", 300, 257, 1280, "silu"), ("bf16", 515, 64, 512, "gelu"),
]


@pytest.mark.parametrize("dtype,m,n,k,kind", GATED)
def test_gated_matches_the_formula(dtype, m, n, k, kind):
    rng = np.random.default_rng([1, m, n, k])
    wg, wu = blocks(rng, n, k), blocks(rng, n, k)
    xt, x = activations(rng, m, k, DT[dtype])
    path = "gemv" if m <= (16 if dtype == "bf16" else 8) else "tensor"
    h, g, u = q2k.gated_ffn(xt, dev(wg), dev(wu), n, act=kind, save=True)
    rh, rg, ru = gated_reference(x, wg, wu, n, kind, path, dtype)
    close(g, rg, "gate")
    close(u, ru, "up")
    close(h, rh, "h")
    alone = q2k.gated_ffn(xt, dev(wg), dev(wu), n, act=kind)
    assert torch.equal(alone, h)


@pytest.mark.parametrize("dtype,m,path", [("f32", 20, "gemv"), ("f32", 20, "tensor"),
                                          ("f32", 3, "tensor"), ("bf16", 40, "gemv"),
                                          ("bf16", 2, "tensor")])
def test_gated_forced_paths(dtype, m, path):
    n, k = 77, 1536
    rng = np.random.default_rng([2, m])
    wg, wu = blocks(rng, n, k), blocks(rng, n, k)
    xt, x = activations(rng, m, k, DT[dtype])
    h = q2k.gated_ffn(xt, dev(wg), dev(wu), n, path=path)
    close(h, gated_reference(x, wg, wu, n, "silu", path, dtype)[0], "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gated_tokens_of_any_magnitude(dtype):
    """Tokens and blocks of a token far apart in magnitude keep their own precision."""
    n, k = 40, 1024
    rng = np.random.default_rng(3)
    wg, wu = blocks(rng, n, k), blocks(rng, n, k)
    x = rng.standard_normal((6, k)).astype(np.float32)
    x[0] *= 1e-15
    x[1] *= 1e15
    x[2, :256] *= 1e8
    x[3, 256:] = 0
    x[4] = 0
    x[5, 1::2] *= 1e-7
    xt = dev(x, DT[dtype])
    _, g, u = q2k.gated_ffn(xt, dev(wg), dev(wu), n, save=True)
    r = U16 if dtype == "bf16" else 2.0 ** -24
    for got, w in ((g, wg), (u, wu)):
        ref, bound = projection(host(xt), w, n, "gemv")
        close(got, (ref, bound + r * (np.abs(ref) + bound)), "projection")


@pytest.mark.parametrize("m", [4, 64])
def test_gated_keeps_tokens_apart(m):
    """A token that is not finite leaves every other token's bits alone."""
    n, k = 70, 1024
    rng = np.random.default_rng(4)
    wg, wu = dev(blocks(rng, n, k)), dev(blocks(rng, n, k))
    xt, _ = activations(rng, m, k, torch.bfloat16)
    clean = q2k.gated_ffn(xt, wg, wu, n)
    bad = xt.clone()
    bad[1, 7] = float("nan")
    bad[2, 500] = float("inf")
    h = q2k.gated_ffn(bad, wg, wu, n)
    keep = [i for i in range(m) if i not in (1, 2)]
    assert torch.equal(h[keep], clean[keep])
    assert not torch.isfinite(h[1]).any() and not torch.isfinite(h[2]).all()


@pytest.mark.parametrize("m", [1, 24, 300])
def test_gated_weights_off_sixteen_bytes(m):
    n, k = 50, 1024
    rng = np.random.default_rng([5, m])
    wg, wu = blocks(rng, n, k), blocks(rng, n, k)
    xt, x = activations(rng, m, k, torch.bfloat16)
    hold = torch.empty(2 * wg.size + 64, dtype=torch.uint8, device="cuda:0")
    a, b = hold[4:4 + wg.size], hold[wg.size + 12:2 * wg.size + 12]
    a.copy_(dev(wg))
    b.copy_(dev(wu))
    h = q2k.gated_ffn(xt, a, b, n)
    path = "gemv" if m <= 16 else "tensor"
    close(h, gated_reference(x, wg, wu, n, "silu", path, "bf16")[0], "h")


BACKWARD = [(1, 1, 256, "silu"), (1, 64, 1024, "gelu"), (2, 65, 768, "silu"), (7, 130, 256, "silu"),
            (16, 200, 1280, "gelu"), (33, 129, 1024, "silu"), (64, 64, 2816, "silu"),
            (65, 1, 512, "gelu"), (128, 300, 1024, "silu"), (129, 63, 768, "gelu"),
            (257, 513, 256, "silu"), (300, 1001, 1280, "silu")]


def backward_reference(dh, g, u, wg, wu, n, k, kind):
    dg, du = dh * u * slope(g, kind), dh * act(g, kind)
    wgf, wuf = decoded(wg, n, k)[0], decoded(wu, n, k)[0]
    dx = dg @ wgf + du @ wuf
    bx = 8e-3 * (np.abs(dg) @ np.abs(wgf) + np.abs(du) @ np.abs(wuf))
    # dg and du in f32: the logistic's error (4 units in its last place), scaled by
    # at most |g| z' <= 36 where the slope's terms cancel
    e = np.abs(dh) * (np.abs(u) * (1 + np.abs(g)) * 36 + np.abs(g)) * 8 * 2.0 ** -24
    return (dx, bx + U16 * np.abs(dx) + 8e-3 * bx), (dg, e + U16 * np.abs(dg)), (du, e + U16 * np.abs(du))


@pytest.mark.parametrize("m,n,k,kind", BACKWARD)
def test_gated_backward_matches_the_formula(m, n, k, kind):
    rng = np.random.default_rng([6, m, n, k])
    wg, wu = blocks(rng, n, k), blocks(rng, n, k)
    dht, dh = activations(rng, m, n, torch.bfloat16, 0.3)
    gt, g = activations(rng, m, n, torch.bfloat16, 2.0)
    ut, u = activations(rng, m, n, torch.bfloat16, 1.5)
    dx, dg, du = q2k.gated_ffn_backward(dht, gt, ut, dev(wg), dev(wu), k, act=kind)
    rx, rg, ru = backward_reference(dh, g, u, wg, wu, n, k, kind)
    close(dg, rg, "dgate")
    close(du, ru, "dup")
    close(dx, rx, "dx")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_backward_matches_differences(kind):
    """<dx, v> against central differences of the 64-bit forward pass along v."""
    m, n, k = 5, 90, 512
    rng = np.random.default_rng(7)
    wg, wu = blocks(rng, n, k), blocks(rng, n, k)
    xt, x = activations(rng, m, k, torch.bfloat16)
    dht, dh = activations(rng, m, n, torch.bfloat16)
    wgf, wuf = decoded(wg, n, k)[0], decoded(wu, n, k)[0]

    def loss(x):
        return np.sum(dh * act(x @ wgf.T, kind) * (x @ wuf.T))

    _, gt, ut = q2k.gated_ffn(xt, dev(wg), dev(wu), n, act=kind, save=True)
    dx = host(q2k.gated_ffn_backward(dht, gt, ut, dev(wg), dev(wu), k, act=kind)[0])
    # the saved projections carry bf16's 2^-8, the slopes vary by less than 1.2 per
    # unit, so dg and du are within 2^-8 (|dh| (|u| + |g u|) 1.2 + ...) of the formula's
    g, u = x @ wgf.T, x @ wuf.T
    eg = U16 * np.abs(dh) * np.abs(u) * (1.2 * np.abs(g) + np.abs(slope(g, kind)))
    eu = U16 * np.abs(dh) * 1.13 * np.abs(g)
    dg, du = dh * u * slope(g, kind), dh * act(g, kind)
    ex = (eg + 8e-3 * np.abs(dg)) @ np.abs(wgf) + (eu + 8e-3 * np.abs(du)) @ np.abs(wuf)
    ex += U16 * np.abs(dx)
    for _ in range(8):
        v = rng.standard_normal((m, k))
        t = 1e-4
        diff = (loss(x + t * v) - loss(x - t * v)) / (2 * t)
        assert abs(np.sum(dx * v) - diff) <= np.sum(ex * np.abs(v)) + 1e-5 * abs(diff)


def test_gated_backward_of_empty_gradients():
    """Rows of dh that are all zero get a gradient of exactly zero."""
    m, n, k = 40, 100, 512
    rng = np.random.default_rng(8)
    wg, wu = dev(blocks(rng, n, k)), dev(blocks(rng, n, k))
    dh, _ = activations(rng, m, n, torch.bfloat16)
    g, _ = activations(rng, m, n, torch.bfloat16, 100.0)  # both saturated ends
    u, _ = activations(rng, m, n, torch.bfloat16)
    dh[3:9] = 0
    dx, dg, du = q2k.gated_ffn_backward(dh, g, u, wg, wu, k, act="gelu")
    assert not dx[3:9].any() and not dg[3:9].any() and not du[3:9].any()
    assert torch.isfinite(dx.float()).all()


LORA = [("f32", 1, 1, 256, 8, 1), ("f32", 1, 64, 1024, 16, 3), ("f32", 4, 33, 2816, 8, 2),
        ("f32", 8, 100, 768, 64, 9), ("bf16", 1, 70, 1280, 16, 4), ("bf16", 5, 16, 14336, 24, 2),
        ("bf16", 16, 129, 4352, 16, 16), ("bf16", 17, 64, 512, 8, 5), ("bf16", 45, 203, 1792, 8, 5),
        ("bf16", 64, 65, 1024, 128, 2), ("bf16", 130, 97, 768, 256, 3), ("bf16", 300, 300, 1024, 40, 7)]


def lora_inputs(rng, dtype, m, n, k, r, na):
    w = blocks(rng, n, k)
    xt, x = activations(rng, m, k, DT[dtype])
    at, a = activations(rng, na * r, k, torch.bfloat16, 1 / np.sqrt(k))
    bt, b = activations(rng, na * n, r, torch.bfloat16, 1 / np.sqrt(r))
    s = rng.uniform(-2, 2, na).astype(np.float32)
    return w, xt, x, at.view(na, r, k), a.reshape(na, r, k), bt.view(na, n, r), b.reshape(na, n, r), s


def lora_reference(x, w, a, b, s, ids, n, path, dtype):
    y, e = projection(x, w, n, path)
    for i, d in enumerate(ids):
        if d >= 0:
            t, at = a[d] @ x[i], np.abs(a[d]) @ np.abs(x[i])
            y[i] += s[d] * (b[d] @ t)
            # both products in f32: (k / 32 + 32 + rank) roundings at most, plus the
            # split of x (f32) or of t (2^-16) on the way through the tensor cores
            c = (a.shape[2] / 32 + 64 + a.shape[1]) * 2.0 ** -24 + 2.0 ** -16
            if dtype == "f32":
                c = (a.shape[2] / 32 + 64 + a.shape[1]) * 2.0 ** -24
            e[i] += c * abs(s[d]) * (np.abs(b[d]) @ at)
    r = U16 if dtype == "bf16" else 2.0 ** -24
    return y, e + r * (np.abs(y) + e)


@pytest.mark.parametrize("dtype,m,n,k,r,na", LORA)
def test_lora_matches_the_formula(dtype, m, n, k, r, na):
    rng = np.random.default_rng([9, m, n, k])
    w, xt, x, at, a, bt, b, s = lora_inputs(rng, dtype, m, n, k, r, na)
    path = "gemv" if m <= (16 if dtype == "bf16" else 8) else "tensor"
    for ids in (rng.integers(-1, na, m), np.arange(m) * na // m, np.full(m, -1), np.full(m, na - 1)):
        y = q2k.matmul_lora(xt, dev(w), n, at, bt, dev(ids.astype(np.int32)), scales=dev(s))
        close(y, lora_reference(x, w, a, b, s, ids, n, path, dtype), "y")


@pytest.mark.parametrize("dtype,m", [("f32", 1), ("bf16", 9), ("bf16", 40)])
def test_lora_without_scales_and_bad_ids(dtype, m):
    n, k, r, na = 45, 768, 16, 4
    rng = np.random.default_rng([10, m])
    w, xt, x, at, a, bt, b, s = lora_inputs(rng, dtype, m, n, k, r, na)
    ids = rng.integers(-1, na, m).astype(np.int32)
    path = "gemv" if m <= 16 else "tensor"
    y = q2k.matmul_lora(xt, dev(w), n, at, bt, dev(ids))
    close(y, lora_reference(x, w, a, b, np.ones(na), ids, n, path, dtype), "y")
    bad = ids.copy()
    bad[0] = na
    bad[m // 2] = -2 if m > 1 else na
    with pytest.raises(q2k.InvalidArgument, match="outside"):
        q2k.matmul_lora(xt, dev(w), n, at, bt, dev(bad))
    z, count = q2k.matmul_lora(xt, dev(w), n, at, bt, dev(bad), check=False)
    rows = sorted({0, m // 2})
    assert int(count.item()) == len(rows)
    assert not z[rows].any()
    keep = [i for i in range(m) if i not in rows]
    assert torch.equal(z[keep], y[keep])


@pytest.mark.parametrize("m", [2, 40])
def test_lora_tokens_do_not_depend_on_the_batch(m):
    """An adapter's weights that are not finite reach only its own tokens."""
    n, k, r, na = 64, 1024, 8, 3
    rng = np.random.default_rng([11, m])
    w, xt, x, at, a, bt, b, s = lora_inputs(rng, "bf16", m, n, k, r, na)
    ids = np.full(m, 0, np.int32)
    ids[1] = 2
    y = q2k.matmul_lora(xt, dev(w), n, at, bt, dev(ids))
    at2, bt2 = at.clone(), bt.clone()
    at2[2] = float("nan")
    bt2[1] = float("inf")
    z = q2k.matmul_lora(xt, dev(w), n, at2, bt2, dev(ids))
    keep = [i for i in range(m) if i != 1]
    assert torch.equal(z[keep], y[keep])
    assert torch.isnan(z[1].float()).all()


@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_streams_repeats_and_capture(m):
    """The same bits on another stream, again, and replayed from a graph."""
    n, k, r, na = 96, 1024, 16, 3
    rng = np.random.default_rng([12, m])
    w, xt, x, at, a, bt, b, s = lora_inputs(rng, "bf16", m, n, k, r, na)
    w2 = dev(blocks(rng, n, k))
    wd, ids = dev(w), dev(rng.integers(-1, na, m).astype(np.int32))
    dh, _ = activations(rng, m, n, torch.bfloat16)

    def all_three():
        h, g, u = q2k.gated_ffn(xt, wd, w2, n, save=True, const_weights=True)
        back = q2k.gated_ffn_backward(dh, g, u, wd, w2, k)
        y, _bad = q2k.matmul_lora(xt, wd, n, at, bt, ids, check=False)
        return (h, g, u, *back, y)

    first = all_three()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = all_three()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = all_three()
    for t in third:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, third))
