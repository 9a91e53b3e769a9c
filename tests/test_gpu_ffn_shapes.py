"""The feed-forward operators where their work is divided: several units, tiles or
parts of K for a worker, and the same bits whenever a call is repeated.  Bounds as in
test_gpu_ffn; the terms of the exact path's bound hold for any number of blocks up
to 160 (K 40960): (4 + 34 + 160 + 16) 2^-24 is 1.3e-5, of T / 2 = |dl q| or |ml| at
most for every product but the last rounding, so 2e-5 T is used above 56 blocks.
"""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import (DT, _device, activations, blocks, close, decoded, dev, gated_reference,
                          lora_inputs, lora_reference)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device", "decoded"]

# one, few and a pass's most tokens; 9, 11, 16 blocks (a CTA each), 20, 24, 56, 128
# (clusters of two to eight), 18 and 132 (neither); n: less than a tile, and units
# for some workers and not for others
FEW = [("f32", 1, 2500, 2304), ("bf16", 1, 2433, 2816), ("f32", 1, 5000, 4096),
       ("f32", 1, 700, 5120), ("bf16", 1, 1201, 6144), ("f32", 1, 1300, 14336), ("f32", 1, 3, 32768),
       ("f32", 1, 40, 4608), ("bf16", 1, 33, 33792),
       ("f32", 4, 2450, 2304), ("bf16", 8, 2600, 4096), ("bf16", 3, 900, 5120), ("f32", 2, 1250, 14336),
       ("f32", 8, 2481, 2816), ("bf16", 16, 5001, 4096), ("bf16", 9, 650, 6144), ("bf16", 16, 1290, 14336),
       ("bf16", 16, 17, 32768), ("f32", 5, 100, 33792)]


def few_path(ref, k):
    """Twice the bound above 56 blocks."""
    return tuple((r, b * (2 if k > 14336 else 1)) for r, b in ref)


@pytest.mark.parametrize("dtype,m,n,k", FEW)
def test_gated_few_tokens(dtype, m, n, k):
    rng = np.random.default_rng([21, m, n, k])
    wg, wu = blocks(rng, n, k), blocks(rng, n, k)
    xt, x = activations(rng, m, k, DT[dtype])
    h, g, u = q2k.gated_ffn(xt, dev(wg), dev(wu), n, save=True)
    rh, rg, ru = few_path(gated_reference(x, wg, wu, n, "silu", "gemv", dtype), k)
    close(g, rg, "gate")
    close(u, ru, "up")
    close(h, rh, "h")


@pytest.mark.parametrize("dtype,m,n,k", [("f32", 1, 5100, 2816), ("bf16", 1, 2561, 5120),
                                         ("f32", 3, 2500, 6144), ("bf16", 16, 2700, 14336),
                                         ("bf16", 12, 5200, 4096)])
def test_lora_few_tokens(dtype, m, n, k):
    rng = np.random.default_rng([22, m, n, k])
    r, na = 16, 5
    w, xt, x, at, a, bt, b, s = lora_inputs(rng, dtype, m, n, k, r, na)
    ids = rng.integers(-1, na, m)
    y = q2k.matmul_lora(xt, dev(w), n, at, bt, dev(ids.astype(np.int32)), scales=dev(s))
    close(y, lora_reference(x, w, a, b, s, ids, n, "gemv", dtype), "y")


@pytest.mark.parametrize("m,n,k", [(20, 12000, 512), (100, 11000, 256), (200, 10100, 512),
                                   (400, 9000, 256), (70, 300, 4096), (256, 130, 6144),
                                   (20, 3, 768), (40, 6, 1280), (33, 129, 2816), (300, 515, 2816),
                                   (150, 10103, 768)])
def test_gated_many_tokens(m, n, k):
    """More tiles than workers, whole and cut, few tiles in parts of K, and rows that
    start off 16 bytes with one to three past the last four."""
    rng = np.random.default_rng([23, m, n, k])
    wg, wu = blocks(rng, n, k), blocks(rng, n, k)
    xt, x = activations(rng, m, k, torch.bfloat16)
    h = q2k.gated_ffn(xt, dev(wg), dev(wu), n)
    close(h, gated_reference(x, wg, wu, n, "silu", "tensor", "bf16")[0], "h")


REPEATS = [(1, 14336, 4096), (1, 4096, 14336), (4, 14336, 4096), (16, 14336, 4096), (16, 4096, 14336),
           (32, 14336, 4096), (64, 14336, 4096), (128, 14336, 4096), (256, 14336, 4096),
           (512, 14336, 4096), (1024, 4096, 4096)]


@pytest.mark.parametrize("m,n,k", REPEATS)
def test_repeats_at_size(m, n, k):
    """Forty calls of each operator on full-size weights give the same bits."""
    gen = torch.Generator(device="cuda:0").manual_seed(m + n)
    wg = dev(blocks(np.random.default_rng(24), 64, k)).repeat(n // 64)
    wu = wg.roll(84 * 7)
    x = torch.randn(m, k, device="cuda:0", generator=gen).bfloat16()
    dh = torch.randn(m, n, device="cuda:0", generator=gen).bfloat16()
    a = torch.randn(6, 16, k, device="cuda:0", generator=gen).bfloat16()
    b = torch.randn(6, n, 16, device="cuda:0", generator=gen).bfloat16()
    ids = torch.randint(-1, 6, (m,), device="cuda:0", generator=gen, dtype=torch.int32)

    def run():
        h, g, u = q2k.gated_ffn(x, wg, wu, n, save=True, const_weights=True)
        back = q2k.gated_ffn_backward(dh, g, u, wg, wu, k)
        y, _bad = q2k.matmul_lora(x, wg, n, a, b, ids, const_weights=True, check=False)
        return (h, g, u, *back, y)

    first = run()
    for _ in range(40):
        assert all(torch.equal(p, q) for p, q in zip(first, run()))


@pytest.mark.parametrize("m", [1, 16, 40])
def test_explicit_buffers_give_the_same_bits(m):
    """The compiled module's way and the one with the caller's own buffers."""
    assert q2k._quick()
    n, k, r, na = 96, 1024, 16, 3
    rng = np.random.default_rng([25, m])
    w, xt, x, at, a, bt, b, s = lora_inputs(rng, "bf16", m, n, k, r, na)
    wd, w2 = dev(w), dev(blocks(rng, n, k))
    ids, sd = dev(rng.integers(-1, na, m).astype(np.int32)), dev(s)
    dh, _ = activations(rng, m, n, torch.bfloat16)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda:0")
    h = q2k.gated_ffn(xt, wd, w2, n, act="gelu")
    out = torch.empty_like(h)
    assert q2k.gated_ffn(xt, wd, w2, n, act="gelu", out=out, workspace=ws) is out
    assert torch.equal(h, out)
    h, g, u = q2k.gated_ffn(xt, wd, w2, n, save=True)
    for p, q in zip((h, g, u), q2k.gated_ffn(xt, wd, w2, n, save=True, workspace=ws)):
        assert torch.equal(p, q)
    for p, q in zip(q2k.gated_ffn_backward(dh, g, u, wd, w2, k),
                    q2k.gated_ffn_backward(dh, g, u, wd, w2, k, workspace=ws)):
        assert torch.equal(p, q)
    y = q2k.matmul_lora(xt, wd, n, at, bt, ids, scales=sd)
    assert torch.equal(y, q2k.matmul_lora(xt, wd, n, at, bt, ids, scales=sd, out=out, workspace=ws))


def test_refusals_with_device_tensors():
    """What the compiled module does not take is refused by name."""
    n, k = 32, 512
    rng = np.random.default_rng(26)
    w = dev(blocks(rng, n, k))
    x, _ = activations(rng, 4, k, torch.bfloat16)
    with pytest.raises(ValueError, match="contiguous"):
        q2k.gated_ffn(activations(rng, 4, 2 * k, torch.bfloat16)[0][:, ::2], w, w, n)
    with pytest.raises(TypeError, match="w_up"):
        q2k.gated_ffn(x, w, w.float(), n)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        q2k.gated_ffn(x.half(), w, w, n)
    with pytest.raises(q2k.InvalidArgument):
        q2k.gated_ffn(x, w, w[:-84], n)
    with pytest.raises(q2k.InvalidArgument):
        q2k.gated_ffn(x[:0], w, w, n)
    with pytest.raises(KeyError):
        q2k.gated_ffn(x, w, w, n, act="relu")
    with pytest.raises(ValueError, match="gate"):
        q2k.gated_ffn_backward(x[:, :n].contiguous(), x, x, w, w, k)
    a, b = torch.zeros(2, 16, k, device="cuda:0").bfloat16(), torch.zeros(2, n, 16, device="cuda:0").bfloat16()
    ids = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    for bad in (ids.long(), ids[:3], ids.cpu()):
        with pytest.raises((TypeError, ValueError), match="ids"):
            q2k.matmul_lora(x, w, n, a, b, bad)
    with pytest.raises(ValueError, match="lora_b"):
        q2k.matmul_lora(x, w, n, a, b[:, :-1].contiguous(), ids)
    with pytest.raises(ValueError, match="scales"):
        q2k.matmul_lora(x, w, n, a, b, ids, scales=torch.ones(3, device="cuda:0"))
