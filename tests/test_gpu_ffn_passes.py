"""Few-token kernels asked for many tokens: passes over them within a launch, and
more passes than a launch holds (65535).  Bounds as in test_gpu_ffn."""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import (DT, U16, _device, activations, blocks, close, decoded, dev, gated_reference,
                          lora_inputs, lora_reference)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]


@pytest.mark.parametrize("dtype,m", [("f32", 9), ("f32", 29), ("bf16", 17), ("bf16", 70)])
@pytest.mark.parametrize("n,k", [(700, 2304), (5001, 4096), (70, 4608), (130, 5120), (650, 14336)])
def test_passes_of_a_launch(dtype, m, n, k):
    rng = np.random.default_rng([61, m, k])
    r, na = 16, 3
    w, xt, x, at, a, bt, b, s = lora_inputs(rng, dtype, m, n, k, r, na)
    w2 = blocks(rng, n, k)
    out = q2k.gated_ffn(xt, dev(w), dev(w2), n, save=True, path="gemv")
    for got, ref, what in zip(out, gated_reference(x, w, w2, n, "silu", "gemv", dtype), ("h", "gate", "up")):
        close(got, ref, what)
    ids = rng.integers(-1, na, m)
    y = q2k.matmul_lora(xt, dev(w), n, at, bt, dev(ids.astype(np.int32)), scales=dev(s), path="gemv")
    close(y, lora_reference(x, w, a, b, s, ids, n, "gemv", dtype), "y")


def worst_of_bound(xt, got, w, n, k, dtype, rows=1 << 16):
    """The largest error of a projection in units of its bound, in float64 on the GPU."""
    wf, parts = (torch.from_numpy(v).to("cuda:0") for v in decoded(w, n, k))
    worst = 0.0
    for i in range(0, len(xt), rows):
        x = xt[i:i + rows].double()
        ref, bound = x @ wf.T, 1e-5 * (x.abs() @ parts.T)
        bound += (U16 if dtype == "bf16" else 2.0 ** -24) * (ref.abs() + bound)
        worst = max(worst, float(((got[i:i + rows].double() - ref).abs() / bound).max()))
    return worst


@pytest.mark.parametrize("dtype,m,n,k", [("f32", 8 * 65535 + 1, 3, 256), ("f32", 1 << 20, 3, 256),
                                         ("bf16", 16 * 65535 + 9, 3, 256), ("f32", 8 * 65535 + 13, 20, 2304)])
def test_more_passes_than_a_launch_holds(dtype, m, n, k):
    rng = np.random.default_rng([62, k])
    w, w2 = blocks(rng, n, k), blocks(rng, n, k)
    gen = torch.Generator(device="cuda:0").manual_seed(m)
    xt = torch.randn(m, k, device="cuda:0", generator=gen).to(DT[dtype])
    h, g, u = q2k.gated_ffn(xt, dev(w), dev(w2), n, save=True, path="gemv")
    assert worst_of_bound(xt, g, w, n, k, dtype) <= 1
    assert worst_of_bound(xt, u, w2, n, k, dtype) <= 1
    # every adapter is worth a multiple of one column
    a = torch.zeros(2, 8, k, device="cuda:0").bfloat16()
    a[:, 0, 0] = 1
    b = torch.zeros(2, n, 8, device="cuda:0").bfloat16()
    b[0, :, 0], b[1, :, 0] = 1, -2
    ids = torch.randint(-1, 2, (m,), device="cuda:0", generator=gen, dtype=torch.int32)
    y = q2k.matmul_lora(xt, dev(w), n, a, b, ids, path="gemv")
    plain = q2k.matmul_lora(xt, dev(w), n, a, b, torch.full_like(ids, -1), path="gemv")
    assert torch.equal(plain, g)
    factor = torch.where(ids < 0, 0, torch.where(ids == 0, 1, -2))
    ref = g.double() + (factor * xt[:, 0].double())[:, None]
    # one f32 addition, and in bf16 the roundings of both results
    unit = 2 * U16 if dtype == "bf16" else 2.0 ** -22
    assert bool(((y.double() - ref).abs() <= unit * (ref.abs() + g.double().abs()) + 1e-30).all())
