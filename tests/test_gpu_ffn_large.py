"""Offsets past 32 bits: activations, weights and adapters of more than 2^31 elements or
2^32 bytes, sampled at both ends against 64 bits.  Bounds as in test_gpu_ffn."""

import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import _device
from test_gpu_ffn_divided import ROWS, Matrix, randn, silu, within

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]


@pytest.fixture(autouse=True)
def _memory():
    free, _ = torch.cuda.mem_get_info()
    if free < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


def ends(m, count=40):
    """Tokens at both ends and in the middle."""
    at = list(range(count)) + list(range(m // 2, m // 2 + count)) + list(range(m - count, m))
    return torch.tensor(at, device="cuda:0")


def test_activations():
    m, n, k = 140_003, 16_384, 256  # 2.29e9 of h, gate, up
    gen = torch.Generator(device="cuda:0").manual_seed(1)
    a, b = Matrix(n, k, 1), Matrix(n, k, 2)
    x = randn(gen, m, k).bfloat16()
    h, g, u = q2k.gated_ffn(x, a.w, b.w, n, save=True)
    at = ends(m)
    (rg, sg), (ru, su) = a.times(x[at].double()), b.times(x[at].double())
    eg, eu = 8e-3 * sg, 8e-3 * su
    within(g[at], rg, eg, "bf16", "gate")
    within(u[at], ru, eu, "bf16", "up")
    eh = 1.13 * eg * (ru.abs() + eu) + silu(rg).abs() * eu
    within(h[at], silu(rg) * ru, eh + 4 * 2.0 ** -24 * (silu(rg) * ru).abs(), "bf16", "h")
    dx, dg, du = q2k.gated_ffn_backward(h, g, u, a.w, b.w, k)
    (r1, s1), (r2, s2) = a.under(dg[at].double()), b.under(du[at].double())
    within(dx[at], r1 + r2, 8e-3 * (s1 + s2), "bf16", "dx")
    gd, hd = g[at].double(), h[at].double()
    within(du[at], hd * gd * torch.sigmoid(gd), 1e-6 * hd.abs() * gd.abs(), "bf16", "dup")


@pytest.mark.parametrize("dtype,m", [("f32", 1), ("bf16", 5), ("bf16", 20), ("f32", 20)])
def test_weights(dtype, m):
    n, k = 1 << 20, 16_384  # 5.6e9 bytes of each matrix
    gen = torch.Generator(device="cuda:0").manual_seed(2)
    a = Matrix(n, k, 1)
    b = a.w.view(-1, ROWS, k // 256 * 84).roll(-9, 1).reshape(-1)  # (Wu: Wg's rows, nine on)
    x = randn(gen, m, k).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    h, g, u = q2k.gated_ffn(x, a.w, b, n, save=True)
    ref, total = a.times(x.double())
    # (the tensor path's bound for both: what is looked for is rows read elsewhere)
    within(g, ref, 8e-3 * total, dtype, "gate")
    at = (torch.arange(n, device="cuda:0") + 9) % ROWS
    within(u, ref[:, at], 8e-3 * total[:, at], dtype, "up")
    within(h, silu(g.double()) * u.double(), 2.0 ** -20 * (g.double() * u.double()).abs()
           + (2.0 ** -6 * (g.double() * u.double()).abs() if dtype == "bf16" else 0), dtype, "h")
    y = q2k.matmul_lora(x, a.w, n, torch.zeros(1, 8, k, device="cuda:0").bfloat16(),
                        torch.zeros(1, n, 8, device="cuda:0").bfloat16(),
                        torch.zeros(m, dtype=torch.int32, device="cuda:0"))
    within(y, ref, 8e-3 * total, dtype, "y")


@pytest.mark.parametrize("m", [1, 12, 50])
def test_adapters(m):
    n, k, r, na = 16_384, 256, 256, 700  # 2.9e9 of b
    gen = torch.Generator(device="cuda:0").manual_seed(3)
    w = Matrix(n, k, 1)
    x = randn(gen, m, k).bfloat16()
    a = randn(gen, na, r, k, scale=k ** -0.5).bfloat16()
    b = torch.randn((na, n, r), device="cuda:0", generator=gen, dtype=torch.bfloat16) * r ** -0.5
    ids = (na - 1 - 37 * torch.arange(m, device="cuda:0") % na).int()
    y = q2k.matmul_lora(x, w.w, n, a, b, ids)
    ref, total = w.times(x.double())
    bound = 8e-3 * total
    for i in range(m):
        t, tt = a[ids[i]].double() @ x[i].double(), a[ids[i]].double().abs() @ x[i].double().abs()
        ref[i] += b[ids[i]].double() @ t
        bound[i] += ((k / 32 + 64 + r) * 2.0 ** -24 + 2.0 ** -16) * (b[ids[i]].double().abs() @ tt)
    within(y, ref, bound, "bf16", "y")
