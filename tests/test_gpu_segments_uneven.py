"""Products over segments of very uneven lengths: all rows or half of them at one of many
experts, at the first or the last one, and few rows of thousands of experts.  The bounds
are test_gpu_linear's."""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import DT, U16, _device, act, activations, blocks, decoded, dev, projection, slope
from test_gpu_linear import R, U, backward_reference, close, linear_reference, routes_of, takes_rows

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]


def uneven(experts, lengths):
    """Lengths of all experts from {expert: rows}."""
    out = [0] * experts
    for e, c in lengths.items():
        out[e] = c
    return out


CASES = [  # lengths, n, k
    (uneven(64, {37: 300}), 136, 1024),
    (uneven(64, {0: 700}), 36, 512),
    (uneven(64, {63: 290}), 132, 2304),
    ([150] + [3, 0, 2, 1] * 16, 64, 1280),
    (uneven(4096, {0: 1, 17: 9, 2048: 1, 4095: 20}), 12, 256),
    (uneven(4096, {4095: 1}), 20, 2560),
    (uneven(300, {299: 2, 5: 1}), 33, 4352),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("path", ["auto", "gemv", "tensor"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward(case, path, dtype):
    lengths, n, k = CASES[case]
    rng = np.random.default_rng([501, case])
    routes, offsets = routes_of(lengths, 0)
    m, experts, mat = int(offsets[-1]), len(lengths), n * (k // 256) * 84
    w, w2 = (blocks(rng, experts * n, k) for _ in range(2))
    x, xv = activations(rng, m, k, DT[dtype])
    r, rv = activations(rng, m, n, DT[dtype])
    b = rng.standard_normal((experts, n)).astype(np.float32)
    y, z = q2k.linear(x, dev(w), n, bias=dev(b), act="silu", residual=r, save=True, path=path, routes=routes)
    h = q2k.gated_ffn(x, dev(w), dev(w2), n, path=path, routes=routes)
    exact = takes_rows(m, dtype, experts, path)
    for e in np.flatnonzero(lengths):
        lo, hi, at = offsets[e], offsets[e + 1], slice(e * mat, (e + 1) * mat)
        ref_y, ref_z = linear_reference(xv[lo:hi], w[at], n, "silu", b[e], rv[lo:hi], exact, dtype)
        close(y[lo:hi], *ref_y, f"y of {e}")
        close(z[lo:hi], *ref_z, f"z of {e}")
        (g, eg), (u, eu) = (projection(xv[lo:hi], v[at], n, "gemv" if exact else "tensor") for v in (w, w2))
        ref = act(g, "silu") * u
        eh = 1.13 * eg * (np.abs(u) + eu) + np.abs(act(g, "silu")) * eu + 4 * U * np.abs(ref)
        close(h[lo:hi], ref, eh + R[dtype] * (np.abs(ref) + eh), f"h of {e}")


@pytest.mark.parametrize("case", range(len(CASES)))
def test_backward(case):
    lengths, n, k = CASES[case]
    rng = np.random.default_rng([502, case])
    routes, offsets = routes_of(lengths, 0)
    m, experts, mat = int(offsets[-1]), len(lengths), n * (k // 256) * 84
    w, w2 = (blocks(rng, experts * n, k) for _ in range(2))
    dy, dyv = activations(rng, m, n, DT["bf16"], 0.1)
    z, zv = activations(rng, m, n, DT["bf16"], 1.5)
    u, uv = activations(rng, m, n, DT["bf16"], 1.5)
    got = q2k.linear_backward(dy, dev(w), k, z=z, act="gelu", bias=True, routes=routes)
    gx, dg, du = q2k.gated_ffn_backward(dy, z, u, dev(w), dev(w2), k, act="gelu", routes=routes)
    empty = np.flatnonzero(np.array(lengths) == 0)
    assert not bool(got[2][dev(empty)].any())
    for e in np.flatnonzero(lengths):
        lo, hi, at = offsets[e], offsets[e + 1], slice(e * mat, (e + 1) * mat)
        refs = backward_reference(dyv[lo:hi], zv[lo:hi], w[at], n, "gelu")
        for t, ref, what in zip((got[0][lo:hi], got[1][lo:hi], got[2][e]), refs, ("dx", "dz", "dbias")):
            close(t, *ref, f"{what} of {e}")
        # as test_gpu_linear's test of segments
        a, c = dyv[lo:hi] * uv[lo:hi] * slope(zv[lo:hi], "gelu"), dyv[lo:hi] * act(zv[lo:hi], "gelu")
        w1, wu = decoded(w[at], n, k)[0], decoded(w2[at], n, k)[0]
        ea, ec = 1e-5 * np.abs(dyv[lo:hi] * uv[lo:hi]), 1e-5 * np.abs(dyv[lo:hi] * zv[lo:hi])
        close(dg[lo:hi], a, ea + U16 * (np.abs(a) + ea), f"dgate of {e}")
        close(du[lo:hi], c, ec + U16 * (np.abs(c) + ec), f"dup of {e}")
        ref = a @ w1 + c @ wu
        close(gx[lo:hi], ref, 8e-3 * (np.abs(a) @ np.abs(w1) + np.abs(c) @ np.abs(wu))
              + ea @ np.abs(w1) + ec @ np.abs(wu) + U16 * np.abs(ref), f"dx of {e}")
    again = q2k.linear_backward(dy, dev(w), k, z=z, act="gelu", bias=True, routes=routes)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
