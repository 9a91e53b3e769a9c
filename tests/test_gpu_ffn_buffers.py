"""The C calls with buffers of exactly the stated sizes: nothing around them is written,
nothing inside is left unwritten, and the optional pointers may be null."""

import ctypes

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import DT, _device, activations, blocks, dev, lora_inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]

GUARD = 4096
G, L = q2k.GatedFfnParams, q2k.LoraParams


class Guarded:
    """`count` elements in the middle of a buffer of 0xA5 bytes."""

    def __init__(self, count, dtype):
        size = count * torch.empty(0, dtype=dtype).element_size()
        self.hold = torch.full((size + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda:0")
        self.size = size
        # (views start 16 bytes off a larger alignment)
        self.inside = self.hold[GUARD - 16:GUARD - 16 + size]
        self.ptr = self.inside.data_ptr()

    def untouched(self):
        return bool((self.hold[:GUARD - 16] == 0xA5).all()) and \
            bool((self.hold[GUARD - 16 + self.size:] == 0xA5).all())

    def tensor(self, dtype, *shape):
        return self.inside.view(dtype).view(shape)


def stream():
    return torch.cuda.current_stream().cuda_stream


def code(dtype):
    return q2k.DTYPE_F32 if dtype == "f32" else q2k.DTYPE_BF16


SHAPES = [("f32", 1, 45, 2304), ("f32", 3, 17, 768), ("f32", 20, 65, 1024), ("f32", 300, 65, 1280),
          ("bf16", 1, 1, 256), ("bf16", 16, 33, 4096), ("bf16", 40, 63, 768), ("bf16", 150, 129, 1024),
          ("bf16", 300, 1001, 1280), ("bf16", 100, 12000, 16384), ("f32", 40, 12000, 16384)]


@pytest.mark.parametrize("dtype,m,n,k", SHAPES)
def test_gated(dtype, m, n, k):
    lib = q2k.load()
    rng = np.random.default_rng([101, m])
    wg = dev(blocks(rng, min(n, 64), k)).repeat(-(-n // 64))[:n * (k // 256) * 84].clone()
    wu = wg.view(n, -1).roll(3, 0).reshape(-1).contiguous()
    x, _ = activations(rng, m, k, DT[dtype])
    p = G(m, n, k, q2k.GGML_TYPE_Q2_K, code(dtype), q2k.ACT_SILU)
    need = lib.q2k_gated_ffn_workspace_bytes(0, ctypes.byref(p))
    ws, out = Guarded(need, torch.uint8), [Guarded(m * n, DT[dtype]) for _ in range(3)]
    expected = q2k.gated_ffn(x, wg, wu, n, save=True)
    for save in (True, False):
        for o in out:
            o.inside.fill_(0xA5)
        assert lib.q2k_gated_ffn(0, 0, x.data_ptr(), x.numel(), wg.data_ptr(), wg.numel(), wu.data_ptr(),
                                 wu.numel(), out[0].ptr, m * n, out[1].ptr if save else None,
                                 out[2].ptr if save else None, ctypes.byref(p), ws.ptr if need else None,
                                 need, stream()) == 0
        torch.cuda.synchronize()
        assert ws.untouched() and all(o.untouched() for o in out)
        for o, e in zip(out[:3 if save else 1], expected):
            assert torch.equal(o.tensor(DT[dtype], m, n), e)
    assert all(bool((o.inside == 0xA5).all()) for o in out[1:])


@pytest.mark.parametrize("m,n,k", [(1, 1, 256), (7, 130, 512), (37, 1001, 1280), (130, 300, 1024),
                                   (600, 5000, 4096), (601, 5003, 4096), (300, 14336, 4096)])
def test_backward(m, n, k):
    lib = q2k.load()
    rng = np.random.default_rng([102, m])
    wg = dev(blocks(rng, min(n, 64), k)).repeat(-(-n // 64))[:n * (k // 256) * 84].clone()
    wu = wg.view(n, -1).roll(5, 0).reshape(-1).contiguous()
    dh, g, u = (activations(rng, m, n, torch.bfloat16)[0] for _ in range(3))
    expected = q2k.gated_ffn_backward(dh, g, u, wg, wu, k)
    p = G(m, n, k, q2k.GGML_TYPE_Q2_K, q2k.DTYPE_BF16, q2k.ACT_SILU)
    need = lib.q2k_gated_ffn_backward_workspace_bytes(ctypes.byref(p))
    ws = Guarded(need, torch.uint8)
    out = [Guarded(m * k, torch.bfloat16), Guarded(m * n, torch.bfloat16), Guarded(m * n, torch.bfloat16)]
    for both in (True, False):
        ws.inside.fill_(0xFF)  # (NaN, whatever it is read as)
        out[0].inside.fill_(0xA5)
        assert lib.q2k_gated_ffn_backward(
            dh.data_ptr(), g.data_ptr(), u.data_ptr(), m * n, wg.data_ptr(), wg.numel(), wu.data_ptr(), wu.numel(),
            out[0].ptr, m * k, out[1].ptr if both else None, out[2].ptr if both else None, ctypes.byref(p),
            ws.ptr if need else None, need, stream()) == 0
        torch.cuda.synchronize()
        assert ws.untouched() and all(o.untouched() for o in out)
        assert torch.equal(out[0].tensor(torch.bfloat16, m, k), expected[0])
        if both:
            for o, e in zip(out[1:], expected[1:]):
                assert torch.equal(o.tensor(torch.bfloat16, m, n), e)


@pytest.mark.parametrize("dtype,m,n,k,r", [("f32", 1, 45, 2304, 8), ("f32", 5, 100, 768, 24),
                                           ("f32", 70, 65, 1024, 16), ("bf16", 1, 1, 256, 8),
                                           ("bf16", 16, 129, 4352, 64), ("bf16", 45, 203, 1792, 256),
                                           ("bf16", 300, 300, 1024, 40)])
def test_adapters(dtype, m, n, k, r):
    lib = q2k.load()
    na = 4
    rng = np.random.default_rng([103, m])
    w, x, _, a, _, b, _, s = lora_inputs(rng, dtype, m, n, k, r, na)
    w, s = dev(w), dev(s)
    ids = dev(rng.integers(-1, na, m).astype(np.int32))
    expected = q2k.matmul_lora(x, w, n, a, b, ids, scales=s)
    p = L(m, n, k, q2k.GGML_TYPE_Q2_K, code(dtype), r, na, 0)
    need = lib.q2k_matmul_lora_workspace_bytes(0, ctypes.byref(p))
    ws, y, bad = Guarded(need, torch.uint8), Guarded(m * n, DT[dtype]), Guarded(1, torch.int32)

    def call(ids, count):
        ws.inside.fill_(0xFF)
        y.inside.fill_(0xA5)
        return lib.q2k_matmul_lora(0, 0, x.data_ptr(), x.numel(), w.data_ptr(), w.numel(), a.data_ptr(),
                                   a.numel(), b.data_ptr(), b.numel(), s.data_ptr(), ids.data_ptr(), y.ptr,
                                   m * n, ctypes.byref(p), count, ws.ptr, need, stream())

    for count in (bad.ptr, None):
        assert call(ids, count) == 0
        torch.cuda.synchronize()
        assert ws.untouched() and y.untouched() and bad.untouched()
        assert torch.equal(y.tensor(DT[dtype], m, n), expected)
    assert int(bad.tensor(torch.int32, 1)) == 0
    # without a counter the call waits and says which ids were out of range
    wrong = ids.clone()
    wrong[-1] = na
    assert call(wrong, None) != 0
    assert b"1" in lib.q2k_last_error()
    assert not y.tensor(DT[dtype], m, n)[-1].any()
    assert call(wrong, bad.ptr) == 0
    torch.cuda.synchronize()
    assert int(bad.tensor(torch.int32, 1)) == 1
