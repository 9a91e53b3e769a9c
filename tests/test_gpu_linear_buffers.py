"""The C calls of the projection, of tokens in segments and of a routed layer's moves with
buffers of exactly the stated sizes: nothing around the outputs and the workspace is
written, and what lies behind an input (NaN here) reaches nothing, the workspace's own
padding included."""

import ctypes

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import DT, _device, activations, blocks, dev
from test_gpu_ffn_buffers import Guarded, code, stream
from test_gpu_linear import routes_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]

BF16 = torch.bfloat16


def among_nan(t):
    """A copy of t with bytes 0xFF (NaN) before and behind it."""
    g = Guarded(t.numel(), t.dtype)
    g.hold.fill_(0xFF)
    out = g.tensor(t.dtype, *t.shape)
    out.copy_(t)
    return out


def weights(rng, n, k):
    return dev(blocks(rng, min(n, 64), k)).repeat(-(-n // 64))[:n * (k // 256) * 84].clone()


def ptr(t):
    return None if t is None else t.data_ptr()


BACKWARD = [  # m, n, k: rows of 4 mod 8 values, of 8, of 2, and odd ones
    (1, 4, 256), (5, 12, 256), (64, 36, 1024), (33, 132, 768), (130, 1004, 1280), (300, 68, 512),
    (40, 124, 512), (64, 136, 768), (17, 1002, 1280), (37, 1001, 1280), (600, 5004, 4096)]


@pytest.mark.parametrize("act", [q2k.ACT_SILU, q2k.ACT_GELU, q2k.ACT_NONE])
@pytest.mark.parametrize("segments", [False, True])
@pytest.mark.parametrize("m,n,k", BACKWARD)
def test_linear_backward(m, n, k, segments, act):
    lib = q2k.load()
    rng = np.random.default_rng([301, m, n])
    experts = 3 if segments else 0
    before = 1 if segments and m > 4 else 0
    lengths = [m - before - m // 2, 0, m // 2]  # (the last segment ends with the last row)
    routes = routes_of(lengths, before)[0] if segments else None
    w = torch.cat([weights(rng, n, k) for _ in range(max(experts, 1))])
    dy = among_nan(activations(rng, m, n, BF16, 0.1)[0])
    z = None if act == q2k.ACT_NONE else among_nan(activations(rng, m, n, BF16, 1.5)[0])
    name = {q2k.ACT_SILU: "silu", q2k.ACT_GELU: "gelu", q2k.ACT_NONE: None}[act]
    expected = q2k.linear_backward(dy.clone(), w, k, z=None if z is None else z.clone(), act=name, bias=True,
                                   routes=routes)
    p = q2k.LinearParams(m, n, k, q2k.GGML_TYPE_Q2_K, q2k.DTYPE_BF16, act, experts, 0)
    real = slice(before, m)
    for with_dz, with_bias in ((True, True), (False, True), (False, False), (True, False)):
        if with_dz and act == q2k.ACT_NONE:
            continue
        need = lib.q2k_linear_backward_workspace_bytes(ctypes.byref(p))
        ws, dx = Guarded(need, torch.uint8), Guarded(m * k, BF16)
        dz, db = Guarded(m * n, BF16), Guarded(max(experts, 1) * n, torch.float32)
        ws.inside.fill_(0xFF)
        assert lib.q2k_linear_backward(
            dy.data_ptr(), m * n, ptr(z), w.data_ptr(), w.numel(), dx.ptr, m * k, dz.ptr if with_dz else None,
            db.ptr if with_bias else None, ptr(routes.offsets if segments else None), ctypes.byref(p),
            ws.ptr if need else None, need, stream()) == 0
        torch.cuda.synchronize()
        assert all(g.untouched() for g in (ws, dx, dz, db))
        assert torch.equal(dx.tensor(BF16, m, k)[real], expected[0][real])
        if with_dz:
            assert torch.equal(dz.tensor(BF16, m, n)[real], expected[1][real])
        if with_bias:
            assert torch.equal(db.tensor(torch.float32, *expected[2].shape), expected[2])
        # where the caller's rows are not whole 16 bytes, dz in rows that are is the
        # workspace's last part: columns past n are zeros, not another row's values or
        # what lies behind the inputs
        if n % 8 != 0:
            pitch = (n + 7) // 8 * 8
            rows = ws.inside[need - (m * pitch * 2 + 255) // 256 * 256:][:m * pitch * 2]
            rows = rows.view(torch.int16).view(m, pitch)
            assert not bool(rows[real, n:].any())
            assert bool((rows[:before] == -1).all())
            assert torch.equal(rows[real, :n], expected[1].view(torch.int16)[real])


@pytest.mark.parametrize("dtype,m,n,k", [("f32", 1, 12, 256), ("f32", 1, 45, 4352), ("f32", 7, 36, 2304),
                                         ("f32", 70, 132, 1280), ("bf16", 1, 1, 256), ("bf16", 16, 33, 4096),
                                         ("bf16", 40, 12, 1024), ("bf16", 150, 130, 1280),
                                         ("bf16", 300, 1001, 1280)])
@pytest.mark.parametrize("segments", [False, True])
def test_linear(dtype, m, n, k, segments):
    lib = q2k.load()
    rng = np.random.default_rng([302, m, n])
    experts = 3 if segments else 0
    lengths = [m - m // 2, 0, m // 2]
    routes = routes_of(lengths, 0)[0] if segments else None
    w = torch.cat([weights(rng, n, k) for _ in range(max(experts, 1))])
    x, residual = (among_nan(activations(rng, m, c, DT[dtype])[0]) for c in (k, n))
    bias = among_nan(dev(rng.standard_normal((experts, n) if segments else n).astype(np.float32)))
    expected = q2k.linear(x.clone(), w, n, bias=bias.clone(), act="gelu", residual=residual.clone(), save=True,
                          routes=routes)
    p = q2k.LinearParams(m, n, k, q2k.GGML_TYPE_Q2_K, code(dtype), q2k.ACT_GELU, experts, 0)
    need = lib.q2k_linear_workspace_bytes(0, ctypes.byref(p))
    for save in (True, False):
        ws, y, z = Guarded(need, torch.uint8), Guarded(m * n, DT[dtype]), Guarded(m * n, DT[dtype])
        ws.inside.fill_(0xFF)
        assert lib.q2k_linear(0, 0, x.data_ptr(), m * k, w.data_ptr(), w.numel(), bias.data_ptr(),
                              residual.data_ptr(), y.ptr, m * n, z.ptr if save else None,
                              ptr(routes.offsets if segments else None), ctypes.byref(p),
                              ws.ptr if need else None, need, stream()) == 0
        torch.cuda.synchronize()
        assert all(g.untouched() for g in (ws, y, z))
        assert torch.equal(y.tensor(DT[dtype], m, n), expected[0])
        if save:
            assert torch.equal(z.tensor(DT[dtype], m, n), expected[1])
        else:
            assert bool((z.inside == 0xA5).all())


@pytest.mark.parametrize("dtype,m,n,k", [("f32", 3, 12, 2304), ("f32", 60, 36, 1280), ("bf16", 5, 132, 4352),
                                         ("bf16", 130, 1001, 1280), ("bf16", 300, 68, 1024)])
def test_gated_experts(dtype, m, n, k):
    lib = q2k.load()
    rng = np.random.default_rng([303, m, n])
    experts = 4
    routes, offsets = routes_of([m // 3, 0, m - m // 3], 0)
    routes = routes._replace(offsets=torch.cat([routes.offsets, routes.offsets[-1:]]))
    wg, wu = (torch.cat([weights(rng, n, k) for _ in range(experts)]) for _ in range(2))
    x = among_nan(activations(rng, m, k, DT[dtype])[0])
    expected = q2k.gated_ffn(x.clone(), wg, wu, n, save=True, routes=routes)
    p = q2k.GatedFfnParams(m, n, k, q2k.GGML_TYPE_Q2_K, code(dtype), q2k.ACT_SILU)
    need = lib.q2k_gated_ffn_experts_workspace_bytes(0, ctypes.byref(p), experts)
    ws, out = Guarded(need, torch.uint8), [Guarded(m * n, DT[dtype]) for _ in range(3)]
    ws.inside.fill_(0xFF)
    assert lib.q2k_gated_ffn_experts(0, 0, x.data_ptr(), m * k, wg.data_ptr(), wg.numel(), wu.data_ptr(),
                                     wu.numel(), out[0].ptr, m * n, out[1].ptr, out[2].ptr,
                                     routes.offsets.data_ptr(), experts, ctypes.byref(p), ws.ptr, need,
                                     stream()) == 0
    torch.cuda.synchronize()
    assert ws.untouched() and all(o.untouched() for o in out)
    assert all(torch.equal(o.tensor(DT[dtype], m, n), e) for o, e in zip(out, expected))
    if dtype == "f32":
        return
    dh, gate, up = (among_nan(activations(rng, m, n, BF16)[0]) for _ in range(3))
    expected = q2k.gated_ffn_backward(dh.clone(), gate.clone(), up.clone(), wg, wu, k, routes=routes)
    need = lib.q2k_gated_ffn_experts_backward_workspace_bytes(ctypes.byref(p), experts)
    ws, out = Guarded(need, torch.uint8), [Guarded(m * c, BF16) for c in (k, n, n)]
    ws.inside.fill_(0xFF)
    assert lib.q2k_gated_ffn_experts_backward(
        dh.data_ptr(), gate.data_ptr(), up.data_ptr(), m * n, wg.data_ptr(), wg.numel(), wu.data_ptr(), wu.numel(),
        out[0].ptr, m * k, out[1].ptr, out[2].ptr, routes.offsets.data_ptr(), experts, ctypes.byref(p), ws.ptr,
        need, stream()) == 0
    torch.cuda.synchronize()
    assert ws.untouched() and all(o.untouched() for o in out)
    assert all(torch.equal(o.tensor(BF16, m, c), e) for o, c, e in zip(out, (k, n, n), expected))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,top_k,width", [(1, 1, 1), (7, 2, 12), (33, 8, 257), (70, 3, 1028), (5, 9, 4100)])
def test_moves(tokens, top_k, width, dtype):
    lib, experts = q2k.load(), 6
    rng = np.random.default_rng([304, tokens, width])
    ids = dev(rng.integers(-1, experts, (tokens, top_k)).astype(np.int32))
    x, dy, residual = (among_nan(activations(rng, tokens, width, DT[dtype])[0]) for _ in range(3))
    ys = among_nan(activations(rng, tokens * top_k, width, DT[dtype])[0])
    weight = among_nan(dev(rng.random((tokens, top_k)).astype(np.float32)))
    p = q2k.MoeParams(tokens, top_k, experts, width, code(dtype), 0)
    r = tokens * top_k
    rows, order, bad = Guarded(r, torch.int32), Guarded(r, torch.int32), Guarded(1, torch.int32)
    offsets = Guarded(experts + 1, torch.int32)
    assert lib.q2k_moe_route(ids.data_ptr(), r, rows.ptr, order.ptr, offsets.ptr, ctypes.byref(p), bad.ptr,
                             stream()) == 0
    xs, dxs, y, dys = (Guarded(c * width, DT[dtype]) for c in (r, tokens, tokens, r))
    dw = Guarded(r, torch.float32)
    where = (rows.ptr, offsets.ptr)
    assert lib.q2k_moe_sort(x.data_ptr(), x.numel(), *where, xs.ptr, r * width, ctypes.byref(p), stream()) == 0
    assert lib.q2k_moe_sort_backward(ys.data_ptr(), ys.numel(), *where, dxs.ptr, tokens * width, ctypes.byref(p),
                                     stream()) == 0
    assert lib.q2k_moe_combine(ys.data_ptr(), ys.numel(), *where, weight.data_ptr(), residual.data_ptr(), y.ptr,
                               tokens * width, ctypes.byref(p), stream()) == 0
    assert lib.q2k_moe_combine_backward(dy.data_ptr(), dy.numel(), ys.data_ptr(), ys.numel(), *where,
                                        weight.data_ptr(), dys.ptr, dw.ptr, ctypes.byref(p), stream()) == 0
    torch.cuda.synchronize()
    assert all(g.untouched() for g in (rows, order, bad, offsets, xs, dxs, y, dys, dw))
    routes = q2k.moe_route(ids, experts)
    assert torch.equal(rows.tensor(torch.int32, tokens, top_k), routes.rows)
    assert torch.equal(order.tensor(torch.int32, r), routes.order)
    assert torch.equal(offsets.tensor(torch.int32, experts + 1), routes.offsets)
    assert torch.equal(xs.tensor(DT[dtype], r, width), q2k.moe_sort(x.clone(), routes))
    assert torch.equal(dxs.tensor(DT[dtype], tokens, width), q2k.moe_sort_backward(ys.clone(), routes))
    want = q2k.moe_combine(ys.clone(), routes, weights=weight.clone(), residual=residual.clone())
    assert torch.equal(y.tensor(DT[dtype], tokens, width), want)
    want = q2k.moe_combine_backward(dy.clone(), ys.clone(), routes, weight.clone())
    assert torch.equal(dys.tensor(DT[dtype], r, width), want[0])
    assert torch.equal(dw.tensor(torch.float32, tokens, top_k), want[1])
