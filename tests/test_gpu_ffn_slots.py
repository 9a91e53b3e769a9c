"""The tensor kernel's raw weight slots, refilled by copies while decoders read them:
full-size products in every tile width and every way that weights arrive (maps of
single rows, maps of four rows together, by the word) give the same bits again and
again, and sampled columns agree with 64 bits.  Bounds as in test_gpu_ffn."""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import U16, _device, act, blocks, decoded, dev, host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]

ROWS = 64  # different weight rows; the matrices repeat them


def matrices(n, k, off):
    """Two matrices of n rows (Wu's are Wg's, nine rows on) `off` bytes past a
    16-byte boundary, and their decoded ROWS rows."""
    w = blocks(np.random.default_rng([31, k]), ROWS, k)
    out = []
    for shift in (0, 9):
        rows = np.roll(w.reshape(ROWS, -1), -shift, axis=0)
        hold = torch.empty(n * rows.shape[1] + 64, dtype=torch.uint8, device="cuda:0")
        m = hold[off:off + n * rows.shape[1]]
        m.copy_(dev(np.resize(rows, (n, rows.shape[1])).reshape(-1)))
        out.append((m, decoded(rows.reshape(-1), ROWS, k)[0]))
    return out


FORMS = [(14336, 4096, 0), (9001, 2816, 0), (6001, 2816, 4)]


@pytest.mark.parametrize("m", [32, 64, 128, 300, 512])
@pytest.mark.parametrize("n,k,off", FORMS)
def test_gated(m, n, k, off):
    (wg, fg), (wu, fu) = matrices(n, k, off)
    gen = torch.Generator(device="cuda:0").manual_seed(m)
    x = torch.randn(m, k, device="cuda:0", generator=gen).bfloat16()
    first = q2k.gated_ffn(x, wg, wu, n, save=True)
    xf = host(x)
    for got, f in zip(first[1:], (fg, fu)):
        ref, bound = xf @ f.T, 8e-3 * (np.abs(xf) @ np.abs(f).T)
        whole = host(got)
        for at in range(0, n, ROWS):  # every column of the matrix against its row
            part = whole[:, at:at + ROWS]
            r, b = ref[:, :part.shape[1]], bound[:, :part.shape[1]]
            assert np.all(np.abs(part - r) <= b + U16 * (np.abs(r) + b))
    for _ in range(60):
        again = q2k.gated_ffn(x, wg, wu, n, save=True)
        assert all(torch.equal(p, q) for p, q in zip(first, again))


@pytest.mark.parametrize("m", [32, 64, 128, 300, 512])
@pytest.mark.parametrize("n,k,off", FORMS)
def test_backward(m, n, k, off):
    (wg, fg), (wu, fu) = matrices(n, k, off)
    gen = torch.Generator(device="cuda:0").manual_seed(m)
    dh, g, u = (torch.randn(m, n, device="cuda:0", generator=gen).bfloat16() for _ in range(3))
    first = q2k.gated_ffn_backward(dh, g, u, wg, wu, k)
    # dx from the dgate and dup that the call returned (rows 64 apart meet the same weights)
    dg, du = host(first[1]), host(first[2])
    pad = -n % ROWS

    def folded(v):
        return np.pad(v, ((0, 0), (0, pad))).reshape(m, -1, ROWS).sum(axis=1)

    ref = folded(dg) @ fg + folded(du) @ fu
    bound = 8e-3 * (folded(np.abs(dg)) @ np.abs(fg) + folded(np.abs(du)) @ np.abs(fu))
    assert np.all(np.abs(host(first[0]) - ref) <= bound + U16 * (np.abs(ref) + bound))
    assert np.all(np.abs(du - host(dh) * act(host(g), "silu")) <= 2 * U16 * np.abs(du) + 1e-6)
    for _ in range(60):
        again = q2k.gated_ffn_backward(dh, g, u, wg, wu, k)
        assert all(torch.equal(p, q) for p, q in zip(first, again))


@pytest.mark.parametrize("m", [32, 128, 300, 512])
@pytest.mark.parametrize("n,k,off", FORMS)
def test_adapters(m, n, k, off):
    """Adapters of zeros: the projection's own bits, again and again."""
    (w, f), _ = matrices(n, k, off)
    gen = torch.Generator(device="cuda:0").manual_seed(m)
    x = torch.randn(m, k, device="cuda:0", generator=gen).bfloat16()
    a = torch.randn(5, 16, k, device="cuda:0", generator=gen).bfloat16()
    b = torch.zeros(5, n, 16, device="cuda:0").bfloat16()
    ids = torch.randint(-1, 5, (m,), device="cuda:0", generator=gen, dtype=torch.int32)
    first = q2k.matmul_lora(x, w, n, a, b, ids)
    xf = host(x)
    ref, bound = xf @ f.T, 8e-3 * (np.abs(xf) @ np.abs(f).T)
    whole = host(first)
    for at in range(0, n, ROWS):
        part = whole[:, at:at + ROWS]
        r, e = ref[:, :part.shape[1]], bound[:, :part.shape[1]]
        assert np.all(np.abs(part - r) <= e + U16 * (np.abs(r) + e))
    for _ in range(60):
        assert torch.equal(first, q2k.matmul_lora(x, w, n, a, b, ids))
