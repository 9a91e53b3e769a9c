"""A token that holds an infinity or a NaN has no finite result, however few of its
values those are and whichever kernel takes the call; and where the formula gives an
infinity, so does the call."""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import DT, _device, act, activations, blocks, decoded, dev, host, lora_inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]

# one block of K a warp, and K divided over clusters of two and four; up to 8 blocks
# and odd divisions go to the other kernel
KS = [1024, 2304, 4096, 4608, 5120, 14336]
# what is put where: one value first and last, a NaN of the smallest payload, nothing else
BAD = {"nan": (float("nan"), [700]), "nan last": (float("nan"), [-1]), "inf": (float("inf"), [3]),
       "-inf": (float("-inf"), [-2]), "all nan": (float("nan"), slice(None)),
       "both": (None, [5, 261])}


def spoiled(x, what):
    value, at = BAD[what]
    bad = x.clone()
    bad[-1, at] = value if value is not None else torch.tensor([float("nan"), float("inf")],
                                                               device=x.device, dtype=x.dtype)
    return bad


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", BAD)
@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("m", [1, 3])
def test_nothing_finite_comes_out(m, k, what, dtype):
    n, r, na = 45, 8, 2
    rng = np.random.default_rng([41, k])
    w, xt, _, at, _, bt, _, s = lora_inputs(rng, dtype, m, n, k, r, na)
    w2 = blocks(rng, n, k)
    bad = spoiled(xt, what)
    out = q2k.gated_ffn(bad, dev(w), dev(w2), n, save=True)
    clean = q2k.gated_ffn(xt, dev(w), dev(w2), n, save=True)
    for a, b in zip(out, clean):
        assert not torch.isfinite(a[-1]).any()
        assert torch.equal(a[:-1], b[:-1])
    for token in (-1, 1):  # without and with an adapter
        ids = torch.full((m,), token, dtype=torch.int32, device="cuda:0")
        y = q2k.matmul_lora(bad, dev(w), n, at, bt, ids, scales=dev(s))
        assert not torch.isfinite(y[-1]).any()


@pytest.mark.parametrize("k", [2304, 4096])
def test_nan_of_any_payload(k):
    n = 40
    rng = np.random.default_rng([42, k])
    w = dev(blocks(rng, n, k))
    x, _ = activations(rng, 1, k, DT["f32"])
    for bits in (0x7F800001, 0x7FFFFFFF, 0xFF800001 - (1 << 32), 0xFFC00000 - (1 << 32)):
        bad = x.clone()
        bad.view(torch.int32)[0, 9] = bits
        assert torch.isnan(q2k.gated_ffn(bad, w, w, n)).all()


def times(x, f):
    """x f^T term by term: zero times an infinity is NaN, whatever a library does."""
    with np.errstate(invalid="ignore"):
        return np.stack([(row * f).sum(1) for row in x])


def same_kind(got, ref, what):
    got = host(got)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), what
    assert np.isfinite(got[np.isfinite(ref)]).all(), what


WHERE = {"one": [(3, np.inf)], "minus": [(-2, -np.inf)], "two": [(700, np.inf), (-1, np.inf)],
         "against": [(0, np.inf), (-1, -np.inf)], "with nan": [(9, -np.inf), (300, np.nan)],
         "beside large": [(5, np.inf), (6, 1e30), (7, -1e30)]}


@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("dtype,m,k", [("f32", 1, 1024), ("f32", 1, 2304), ("bf16", 1, 4096), ("f32", 1, 5120),
                                       ("f32", 3, 1024), ("f32", 8, 4096), ("bf16", 5, 2304), ("bf16", 16, 5120),
                                       ("bf16", 12, 1280), ("bf16", 40, 1024), ("f32", 40, 1280),
                                       ("bf16", 300, 1024), ("f32", 300, 1024), ("bf16", 70, 2816)])
def test_infinities_are_the_formulas(dtype, m, k, where):
    n, r, na = 83, 8, 2
    rng = np.random.default_rng([43, m, k])
    w, w2 = blocks(rng, n, k), blocks(rng, n, k)
    x = rng.standard_normal((m, k))
    for at, v in WHERE[where]:
        x[m // 2, at] = v
    xt = dev(x.astype(np.float32), DT[dtype])
    x = host(xt)
    h, g, u = q2k.gated_ffn(xt, dev(w), dev(w2), n, save=True)
    rg, ru = times(x, decoded(w, n, k)[0]), times(x, decoded(w2, n, k)[0])
    assert np.isinf(rg[m // 2]).any() or where in ("against", "with nan")
    with np.errstate(invalid="ignore"):
        rh = act(rg, "silu") * ru
    for got, ref, what in ((g, rg, "gate"), (u, ru, "up"), (h, rh, "h")):
        same_kind(got, ref, what)
    # adapters whose entries have one sign, so that their infinities stay
    a = np.abs(rng.standard_normal((na, r, k))) + 0.1
    b = np.abs(rng.standard_normal((na, n, r))) + 0.1
    at, bt = dev(a.astype(np.float32), torch.bfloat16), dev(b.astype(np.float32), torch.bfloat16)
    for token in (-1, 1):
        ids = torch.full((m,), token, dtype=torch.int32, device="cuda:0")
        y = q2k.matmul_lora(xt, dev(w), n, at, bt, ids)
        ref = rg
        if token == 1:
            with np.errstate(invalid="ignore"):
                ref = rg + times(times(x, host(at[1])), host(bt[1]))
        same_kind(y, ref, f"y, id {token}")


def largest_weights(n, k):
    """Rows of 45 everywhere: d 1, every scale 15 and code 3, no minima."""
    b = np.zeros((n, k // 256, 84), dtype=np.uint8)
    b[..., :16], b[..., 16:80] = 0x0F, 0xFF
    b[..., 80:] = np.array([1.0, 0.0], dtype="<f2").view(np.uint8)
    return b.reshape(-1)


@pytest.mark.parametrize("k", [1024, 2304, 5120])
@pytest.mark.parametrize("dtype,m", [("f32", 1), ("f32", 4), ("f32", 8), ("bf16", 1), ("bf16", 16)])
def test_sums_that_overflow_are_infinite(dtype, m, k):
    n = 30
    w = dev(largest_weights(n, k))
    for value in (3e38, -1.7e38):
        x = torch.full((m, k), value, device="cuda:0").to(DT[dtype])
        x[0, ::2] *= -0.5  # (parts of both signs)
        _, g, u = q2k.gated_ffn(x, w, w, n, save=True)
        for got in (g, u):
            assert torch.isinf(got).all() and bool(((got > 0) == (value > 0)).all())


@pytest.mark.parametrize("m", [1, 4])
def test_weights_that_are_not_finite(m):
    """A block's d that is infinite or NaN makes its row's results not finite, no others."""
    n, k = 40, 2304
    rng = np.random.default_rng([45])
    w = blocks(rng, n, k).reshape(n, -1, 84)
    x, _ = activations(rng, m, k, DT["f32"])
    clean = q2k.gated_ffn(x, dev(w.reshape(-1)), dev(w.reshape(-1)), n, save=True)[1]
    w[7, 3, 80:82] = np.array([np.inf], dtype="<f2").view(np.uint8)
    w[9, 8, 82:84] = np.array([np.nan], dtype="<f2").view(np.uint8)
    g = q2k.gated_ffn(x, dev(w.reshape(-1)), dev(w.reshape(-1)), n, save=True)[1]
    keep = [i for i in range(n) if i not in (7, 9)]
    assert torch.equal(g[:, keep], clean[:, keep])
    assert not torch.isfinite(g[:, [7, 9]]).any()


@pytest.mark.parametrize("m", [1, 3, 8])
@pytest.mark.parametrize("k", [1024, 2304, 4096, 5120])
def test_rows_past_the_last_leave_the_others_alone(m, k):
    """What shared memory held before (here weights that are not finite) stands in the
    place of rows past N: no row's bits depend on it."""
    n, r = 20, 8
    rng = np.random.default_rng([46, k])
    w, w2 = dev(blocks(rng, n, k)), dev(blocks(rng, n, k))
    wide = dev(blocks(rng, 152 * 64, k)).view(-1, 84)
    x, _ = activations(rng, m, k, DT["f32"])
    a, b = torch.zeros(1, r, k, device="cuda:0").bfloat16(), torch.zeros(1, n, r, device="cuda:0").bfloat16()
    b_wide = torch.zeros(1, 152 * 64, r, device="cuda:0").bfloat16()
    ids = torch.full((m,), -1, dtype=torch.int32, device="cuda:0")
    results = []
    for d in (0.0, float("inf"), float("nan"), 1.0):
        wide[:, 80:] = torch.tensor([d, d], dtype=torch.float16).view(torch.uint8).to("cuda:0")
        for _ in range(3):
            q2k.gated_ffn(x, wide.view(-1), wide.view(-1), 152 * 64)
            results.append(q2k.gated_ffn(x, w, w2, n, save=True)[1])
            q2k.matmul_lora(x, wide.view(-1), 152 * 64, a, b_wide, ids)
            results.append(q2k.matmul_lora(x, w, n, a, b, ids))
    assert all(torch.equal(results[0], v) for v in results)
