"""The projection with bias, activation and residual, and the products over tokens in
segments (plain and gated, forward and backward), against their formulas in 64 bits.

A projection's bound is test_gpu_ffn's.  On top of it, per output:
- z: the bias' addition rounds once in f32;
- y = act(z) + residual from z's error e: 1.13 e (the activations' slopes), 8 2^-24
  (|z| + |y| + |residual|) of the arithmetic in f32, and the output's half step;
- dz = dy act'(z): the slope is within 1e-5 (its exponential and quotient are within
  2^-20 of theirs, which |g| p (1 - p) z', below 2, scales; 1 - p adds 2^-24 |g z'|, where
  p is not yet 1, |g z'| below 64): 1e-5 |dy|, and the half step;
- dbias: dz before its rounding, its sum over m tokens (m + 1) 2^-24 of the absolute
  terms;
- dx: 8e-3 sum |dz w| as test_gpu_ffn's, and 1e-5 sum |dy w| from dz's own error.
"""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import DT, U16, act, activations, blocks, decoded, dev, host, projection, slope

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
R = {"f32": U, "bf16": U16}


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield
    assert q2k.device_error() == 0


def close(got, ref, bound, what):
    err = np.abs(host(got) - ref)
    assert np.all(err <= bound + 1e-30), f"{what}: {np.max(err / np.maximum(bound, 1e-300)):.2f} of the bound"


def takes_rows(m, dtype, experts, path):
    if path != "auto":
        return path == "gemv"
    few, each = (16, 8) if dtype == "bf16" else (8, 4)
    return m <= few or (experts > 0 and m <= each * experts)


def linear_reference(x, w, n, kind, bias, residual, exact, dtype):
    """((y, its bound), (z, its bound))."""
    z, ez = projection(x, w, n, "gemv" if exact else "tensor")
    if bias is not None:
        z = z + bias
    ez = ez + U * np.abs(z)
    y = z if kind is None else act(z, kind)
    if residual is not None:
        y = y + residual
    ey = 1.13 * ez + 8 * U * (np.abs(z) + np.abs(y) + (0 if residual is None else np.abs(residual)))
    return (y, ey + R[dtype] * (np.abs(y) + ey)), (z, ez + R[dtype] * (np.abs(z) + ez))


FORWARD = [  # m, n, k, dtype, path, act, bias, residual, save
    (1, 8, 256, "f32", "auto", "gelu", True, False, False),
    (1, 1, 512, "bf16", "auto", None, False, True, True),
    (1, 513, 4096, "f32", "auto", "silu", True, True, True),
    (1, 96, 14336, "bf16", "auto", None, False, True, False),
    (1, 70, 4352, "f32", "auto", "gelu", True, True, False),
    (4, 33, 2304, "f32", "auto", None, True, False, True),
    (8, 100, 4096, "f32", "auto", "silu", False, True, False),
    (7, 64, 14336, "bf16", "auto", "gelu", True, True, True),
    (16, 131, 4096, "bf16", "auto", "silu", True, True, False),
    (16, 40, 1280, "bf16", "auto", None, True, True, True),
    (40, 40, 1280, "bf16", "gemv", "gelu", True, True, True),
    (9, 65, 768, "f32", "auto", "gelu", True, True, True),
    (100, 130, 1024, "f32", "auto", None, True, False, True),
    (300, 257, 2048, "f32", "auto", "silu", True, True, False),
    (3, 20, 1024, "bf16", "tensor", "gelu", True, True, True),
    (17, 1, 256, "bf16", "auto", "silu", True, True, True),
    (33, 128, 1024, "bf16", "auto", None, False, False, False),
    (77, 499, 2816, "bf16", "auto", "silu", True, True, False),
    (77, 496, 2816, "bf16", "auto", "gelu", True, True, True),
    (129, 1030, 4096, "bf16", "auto", "gelu", True, True, True),
    (256, 384, 2304, "bf16", "auto", None, True, True, False),
    (500, 2000, 1024, "bf16", "auto", "silu", False, True, True),
    (1000, 4100, 512, "bf16", "auto", "gelu", True, False, True),
]


@pytest.mark.parametrize("m,n,k,dtype,path,kind,bias,residual,save", FORWARD)
def test_linear(m, n, k, dtype, path, kind, bias, residual, save):
    rng = np.random.default_rng([1, m, n, k])
    w = blocks(rng, n, k)
    x, xv = activations(rng, m, k, DT[dtype])
    b = rng.standard_normal(n).astype(np.float32) if bias else None
    r, rv = activations(rng, m, n, DT[dtype]) if residual else (None, None)
    got = q2k.linear(x, dev(w), n, bias=dev(b) if bias else None, act=kind, residual=r, save=save,
                     path=path)
    y, z = linear_reference(xv, w, n, kind, b, rv, takes_rows(m, dtype, 0, path), dtype)
    if save:
        close(got[1], *z, "z")
        got = got[0]
    close(got, *y, "y")


def backward_reference(dy, z, w, n, kind):
    """((dx, bound), (dz, bound), (dbias, bound))."""
    wf, _ = decoded(w, n, len(w) // n // 84 * 256)
    dz = dy if kind is None else dy * slope(z, kind)
    e = np.zeros_like(dz) if kind is None else 1e-5 * np.abs(dy)
    return ((dz @ wf, 8e-3 * (np.abs(dz) @ np.abs(wf)) + e @ np.abs(wf) + U16 * np.abs(dz @ wf)),
            (dz, e + U16 * (np.abs(dz) + e)),
            (dz.sum(0), e.sum(0) + (len(dz) + 1) * U * np.abs(dz).sum(0)))


BACKWARD = [(1, 8, 256, "gelu", True), (5, 33, 512, None, True), (37, 1001, 1280, "gelu", True),
            (64, 136, 1024, None, False), (130, 72, 768, None, True), (200, 640, 2048, "silu", False),
            (512, 1000, 1024, "silu", True), (300, 4999, 256, "gelu", True), (513, 64, 2816, None, True),
            (1200, 2056, 4096, "silu", True), (70, 7, 4096, "silu", True)]


@pytest.mark.parametrize("m,n,k,kind,bias", BACKWARD)
def test_linear_backward(m, n, k, kind, bias):
    rng = np.random.default_rng([2, m, n, k])
    w = blocks(rng, n, k)
    dy, dyv = activations(rng, m, n, DT["bf16"], 0.1)
    z, zv = activations(rng, m, n, DT["bf16"], 2.0)
    got = q2k.linear_backward(dy, dev(w), k, z=z, act=kind, bias=bias)
    dx, dz, dbias = backward_reference(dyv, zv, w, n, kind)
    close(got[0], *dx, "dx")
    close(got[1], *dz, "dz")
    assert (got[1] is dy) == (kind is None)
    if bias:
        close(got[2], *dbias, "dbias")
    else:
        assert got[2] is None
    again = q2k.linear_backward(dy, dev(w), k, z=z, act=kind, bias=bias)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


def test_linear_gradients_against_differences():
    """<dy, y(x + h d) - y(x - h d)> / 2h against <dx, d>, and the same in the bias."""
    rng = np.random.default_rng(3)
    m, n, k, h = 24, 40, 512, 2.0 ** -5
    w = dev(blocks(rng, n, k))
    wf, _ = decoded(w.cpu().numpy(), n, k)
    x, xv = activations(rng, m, k, DT["bf16"])
    b = rng.standard_normal(n)
    _, z = q2k.linear(x, w, n, bias=dev(b.astype(np.float32)), act="gelu", save=True)
    dy, dyv = activations(rng, m, n, DT["bf16"])
    dx, dz, dbias = q2k.linear_backward(dy, w, k, z=z, act="gelu", bias=True)
    d, e = rng.standard_normal((m, k)), rng.standard_normal(n)

    def f(xx, bb):
        return float((dyv * act(xx @ wf.T + bb, "gelu")).sum())

    # the differences' own error is of order h^2 times third derivatives: 2 h^2 |dy| |d|^3
    # over the sums; z's and the product's rounding is 8e-3 of the absolute terms
    zs = d @ wf.T
    tol_x = 2 * h * h * float((np.abs(dyv) * np.abs(zs) ** 3).sum()) \
        + 2e-2 * float((np.abs(dyv) @ np.abs(wf) * np.abs(d)).sum())
    assert abs((f(xv + h * d, b) - f(xv - h * d, b)) / (2 * h) - float((host(dx) * d).sum())) < tol_x
    tol_b = 2 * h * h * float((np.abs(dyv) * np.abs(e) ** 3).sum()) \
        + 2e-2 * float((np.abs(dyv) * np.abs(e)).sum())
    assert abs((f(xv, b + h * e) - f(xv, b - h * e)) / (2 * h) - float((host(dbias) * e).sum())) < tol_b


SEGMENTS = [  # lengths of the experts' rows, rows before the first, rows behind the last
    ([1, 1, 1, 1, 1, 1, 1, 1] + [0] * 32, 0, 0),
    ([0, 5, 0, 1, 17, 3, 0], 0, 4),
    ([3], 2, 1),
    ([0, 0, 0], 0, 5),
    ([40, 1, 0, 9, 30], 3, 0),
    ([70, 64, 63, 65], 0, 6),
    ([130, 0, 3, 200, 127], 0, 0),
    ([300, 5, 520, 256], 1, 9),
]
SHAPES = [(40, 256), (130, 1024), (133, 2304), (64, 2816), (36, 4352)]


def routes_of(lengths, before):
    offsets = before + np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    empty = torch.empty(0, dtype=torch.int32, device="cuda:0")
    return q2k.Routes(empty, empty, dev(offsets.astype(np.int32))), offsets


def pool(rng, experts, n, k):
    each = [blocks(rng, n, k) for _ in range(experts)]
    return each, dev(np.concatenate(each))


def untouched(t, offsets, value):
    return bool((t[:offsets[0]] == value).all()) and bool((t[offsets[-1]:] == value).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("path", ["auto", "gemv", "tensor"])
@pytest.mark.parametrize("case", range(len(SEGMENTS)))
def test_segments_forward(case, path, dtype):
    lengths, before, behind = SEGMENTS[case]
    n, k = SHAPES[(case + (path == "tensor") + 2 * (dtype == "f32")) % len(SHAPES)]
    rng = np.random.default_rng([4, case, n, k])
    routes, offsets = routes_of(lengths, before)
    m, experts = int(offsets[-1]) + behind, len(lengths)
    each, w = pool(rng, experts, n, k)
    each2, w2 = pool(rng, experts, n, k)
    x, xv = activations(rng, m, k, DT[dtype])
    x[:before], x[offsets[-1]:] = float("nan"), float("nan")  # (never read)
    r, rv = activations(rng, m, n, DT[dtype])
    b = rng.standard_normal((experts, n)).astype(np.float32)
    y, h = (torch.full((m, n), 7.0, dtype=DT[dtype], device="cuda:0") for _ in range(2))
    _, z = q2k.linear(x, w, n, bias=dev(b), act="gelu", residual=r, save=True, out=y, path=path,
                      routes=routes)
    _, gate, up = q2k.gated_ffn(x, w, w2, n, save=True, out=h, path=path, routes=routes)
    assert untouched(y, offsets, 7) and untouched(h, offsets, 7)
    exact = takes_rows(m, dtype, experts, path)
    for e in range(experts):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        ref_y, ref_z = linear_reference(xv[lo:hi], each[e], n, "gelu", b[e], rv[lo:hi], exact, dtype)
        close(y[lo:hi], *ref_y, f"y of {e}")
        close(z[lo:hi], *ref_z, f"z of {e}")
        (g, eg), (u, eu) = (projection(xv[lo:hi], v[e], n, "gemv" if exact else "tensor")
                            for v in (each, each2))
        ref = act(g, "silu") * u
        eh = 1.13 * eg * (np.abs(u) + eu) + np.abs(act(g, "silu")) * eu + 4 * U * np.abs(ref)
        close(h[lo:hi], ref, eh + R[dtype] * (np.abs(ref) + eh), f"h of {e}")
        close(gate[lo:hi], g, eg + R[dtype] * (np.abs(g) + eg), f"gate of {e}")
        close(up[lo:hi], u, eu + R[dtype] * (np.abs(u) + eu), f"up of {e}")


@pytest.mark.parametrize("kind", [None, "silu"])
@pytest.mark.parametrize("case", range(len(SEGMENTS)))
def test_segments_backward(case, kind):
    lengths, before, behind = SEGMENTS[case]
    n, k = SHAPES[(case + (kind is None)) % len(SHAPES)]
    rng = np.random.default_rng([5, case, n, k])
    routes, offsets = routes_of(lengths, before)
    m, experts = int(offsets[-1]) + behind, len(lengths)
    each, w = pool(rng, experts, n, k)
    each2, w2 = pool(rng, experts, n, k)
    dy, dyv = activations(rng, m, n, DT["bf16"], 0.1)
    z, zv = activations(rng, m, n, DT["bf16"], 1.5)
    u, uv = activations(rng, m, n, DT["bf16"], 1.5)
    dx, dz, dbias = q2k.linear_backward(dy, w, k, z=z, act=kind, bias=True, routes=routes)
    gx, dg, du = q2k.gated_ffn_backward(dy, z, u, w, w2, k, act="gelu", routes=routes)
    assert dbias.shape == (experts, n)
    for e in range(experts):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            assert not bool(dbias[e].any())
            continue
        refs = backward_reference(dyv[lo:hi], zv[lo:hi], each[e], n, kind)
        for got, ref, what in zip((dx[lo:hi], dz[lo:hi], dbias[e]), refs, ("dx", "dz", "dbias")):
            close(got, *ref, f"{what} of {e}")
        a, c = dyv[lo:hi] * uv[lo:hi] * slope(zv[lo:hi], "gelu"), dyv[lo:hi] * act(zv[lo:hi], "gelu")
        w1, wu = decoded(each[e], n, k)[0], decoded(each2[e], n, k)[0]
        ea, ec = 1e-5 * np.abs(dyv[lo:hi] * uv[lo:hi]), 1e-5 * np.abs(dyv[lo:hi] * zv[lo:hi])
        close(dg[lo:hi], a, ea + U16 * (np.abs(a) + ea), f"dgate of {e}")
        close(du[lo:hi], c, ec + U16 * (np.abs(c) + ec), f"dup of {e}")
        ref = a @ w1 + c @ wu
        close(gx[lo:hi], ref, 8e-3 * (np.abs(a) @ np.abs(w1) + np.abs(c) @ np.abs(wu))
              + ea @ np.abs(w1) + ec @ np.abs(wu) + U16 * np.abs(ref), f"dx of {e}")


@pytest.mark.parametrize("n,k", [(40, 1024), (37, 1280), (132, 768)])
@pytest.mark.parametrize("before,lengths,behind", [(3, [5, 0, 40], 4), (2, [0, 0], 6), (0, [130, 7], 1)])
def test_segments_leave_other_rows(n, k, before, lengths, behind):
    """Through the C calls, every output prefilled: rows in no segment stay."""
    import ctypes
    lib, bf16 = q2k.load(), DT["bf16"]
    rng = np.random.default_rng([6, n, before])
    routes, offsets = routes_of(lengths, before)
    m, experts = int(offsets[-1]) + behind, len(lengths)
    _, w = pool(rng, experts, n, k)
    _, w2 = pool(rng, experts, n, k)
    dy, z, u = (activations(rng, m, n, bf16)[0] for _ in range(3))
    full = lambda cols: torch.full((m, cols), 7.0, dtype=bf16, device="cuda:0")  # noqa: E731
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda:0")
    dx, dz, gx, dg, du, px = full(k), full(n), full(k), full(n), full(n), full(k)
    stream = torch.cuda.current_stream().cuda_stream

    def linear(act, dxx, zz, dzz):
        p = q2k.LinearParams(m, n, k, 10, 1, act, experts, 0)
        return lib.q2k_linear_backward(dy.data_ptr(), m * n, zz, w.data_ptr(), w.numel(), dxx.data_ptr(),
                                       m * k, dzz, None, routes.offsets.data_ptr(), ctypes.byref(p),
                                       ws.data_ptr(), ws.numel(), stream)

    assert linear(1, dx, z.data_ptr(), dz.data_ptr()) == 0
    assert linear(2, px, None, None) == 0
    p = q2k.GatedFfnParams(m, n, k, 10, 1, 0)
    assert lib.q2k_gated_ffn_experts_backward(
        dy.data_ptr(), z.data_ptr(), u.data_ptr(), m * n, w.data_ptr(), w.numel(), w2.data_ptr(),
        w2.numel(), gx.data_ptr(), m * k, dg.data_ptr(), du.data_ptr(), routes.offsets.data_ptr(),
        experts, ctypes.byref(p), ws.data_ptr(), ws.numel(), stream) == 0
    for t in (dx, dz, gx, dg, du, px):
        assert untouched(t, offsets, 7)
    real = slice(int(offsets[0]), int(offsets[-1]))
    if sum(lengths):
        want = q2k.linear_backward(dy, w, k, z=z, act="gelu", routes=routes)
        assert torch.equal(dx[real], want[0][real]) and torch.equal(dz[real], want[1][real])
        assert torch.equal(px[real], q2k.linear_backward(dy, w, k, routes=routes)[0][real])
        want = q2k.gated_ffn_backward(dy, z, u, w, w2, k, routes=routes)
        assert all(torch.equal(a[real], b[real]) for a, b in zip((gx, dg, du), want))
