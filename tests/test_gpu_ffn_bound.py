"""The stated error of the few-token kernels for x whose values lie far apart.

Per output, with w = dl q + ml and T = sum_k |x| w (see include/q2k.h):
    c T + r * sum over blocks of 256 of (max |x| sum w),
c = max(1e-5, k 2^-31): the roundings of a block's sums and of k / 256 blocks' after
them, (54 + k / 256) 2^-24 of T; r the rounding of x beside its block's largest: half a
unit of 2^(e-21), e the largest's exponent, for one token in integers, 2^-22 of the half
left after that (2^-43 in all) where more than a quarter of the block is below 2^-9
of the largest; 2^-25 / 2^10 for two f16 parts of an x scaled to 2^10 and above.
Outputs are f32, or bf16 with half a unit in their last place."""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import DT, U16, _device, blocks, close, decoded, dev, host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]


def zero_group(w, n, k, groups):
    """The same rows with the scale bytes of `groups` of every block zero: their
    weights and minima are zero."""
    b = w.reshape(n, k // 256, 84).copy()
    b[..., groups] = 0
    return b.reshape(-1)


def stated(x, parts, dtype, ref):
    m, k = x.shape
    xb, wb = np.abs(x).reshape(m, -1, 256), parts.reshape(len(parts), -1, 256)
    top = np.maximum(xb.max(-1), 2.0 ** -100)
    r = np.full(top.shape, 2.0 ** -34)
    if m == 1:
        e = np.floor(np.log2(top))[..., None]
        wide = ((xb > 0) & (xb < 2.0 ** (e - 9))).sum(-1) > 64
        r = np.where(wide, 2.0 ** -43, 2.0 ** -22)
    bound = max(1e-5, k * 2.0 ** -31) * (np.abs(x) @ parts.T) + (r * top) @ wb.sum(-1).T
    return bound + (U16 if dtype == "bf16" else 2.0 ** -24) * (np.abs(ref) + bound)


def check(x, dtype, n, wg, wu, bound_of=stated):
    k = x.shape[1]
    xt = dev(np.asarray(x, dtype=np.float32), DT[dtype])
    _, g, u = q2k.gated_ffn(xt, dev(wg), dev(wu), n, save=True)
    y = q2k.matmul_lora(xt, dev(wg), n, torch.zeros(1, 8, k, device="cuda:0").bfloat16(),
                        torch.zeros(1, n, 8, device="cuda:0").bfloat16(),
                        torch.full((len(x),), -1, dtype=torch.int32, device="cuda:0"))
    xh = host(xt)
    for got, w, what in ((g, wg, "gate"), (u, wu, "up"), (y, wg, "y")):
        wf, parts = decoded(w, n, k)
        ref = xh @ wf.T
        close(got, (ref, bound_of(xh, parts, dtype, ref)), what)


def without_rest(x, parts, dtype, ref):
    """The bound without its second term."""
    bound = 1e-5 * (np.abs(x) @ parts.T)
    return bound + (U16 if dtype == "bf16" else 2.0 ** -24) * (np.abs(ref) + bound)


KS = [2304, 4096, 5120, 14336]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
# (two tokens and more: two f16 parts hold 2^-34 of the largest)
@pytest.mark.parametrize("m,outlier,rest", [(1, 1024.0, 1.0002), (1, 2.0 ** 23, 1.0), (1, 3e4, -0.37),
                                            (1, 1e20, 1.5), (2, 1024.0, 1.0002), (2, 3e4, -0.37)])
@pytest.mark.parametrize("k", KS)
def test_small_values_beside_an_outlier_without_weight(m, outlier, rest, k, dtype):
    """A value far above its block's others, on weights of zero, takes nothing from
    them: with it left out, the formula's bound is 1e-5 T."""
    n = 50
    rng = np.random.default_rng([51, k])
    wg, wu = (zero_group(blocks(rng, n, k), n, k, [5]) for _ in range(2))
    x = np.full((m, k), rest)
    x *= rng.uniform(1, 1.9, x.shape)
    x[:, 256 * (k // 512) + 32 * 2 + 16 + 3] = outlier  # (group 5: shift 2, segment 1)
    if outlier == 1e20:  # 22 + 22 bits below the largest: 1e20 2^-43 is 1.1e7
        x *= np.where(np.abs(x) < 1e10, 1e13, 1)
    check(x, dtype, n, wg, wu, without_rest)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("span", [2, 8, 12, 18, 30, 60])
@pytest.mark.parametrize("m,k", [(1, k) for k in KS] + [(1, 1024), (3, 2304), (4, 14336), (8, 1024)])
def test_values_over_many_magnitudes(m, k, span, dtype):
    """x = +-2^-u, u over `span` octaves, every block's largest on weights of zero."""
    n = 50
    rng = np.random.default_rng([52, k, span])
    wg, wu = (zero_group(blocks(rng, n, k), n, k, [0, 1, 6]) for _ in range(2))
    x = 2.0 ** -rng.uniform(0, span, (m, k)) * rng.choice([-1, 1], (m, k))
    x[rng.random(x.shape) < 0.1] = 0
    check(x, dtype, n, wg, wu)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", KS)
def test_one_token_of_any_magnitude(k, dtype):
    n = 40
    rng = np.random.default_rng([53, k])
    wg, wu = blocks(rng, n, k), blocks(rng, n, k)
    for change in (lambda v: v * 1e-15, lambda v: v * 1e15, lambda v: v * 1e-31, lambda v: v * 0,
                   lambda v: np.where(np.arange(k) < 256, v * 1e8, v),
                   lambda v: np.where(np.arange(k) < 256, v, 0),
                   lambda v: np.where(np.arange(k) % 2, v * 1e-7, v),
                   lambda v: np.where(np.arange(k) % 256, 0, v)):
        check(change(rng.standard_normal((1, k))), dtype, n, wg, wu)


@pytest.mark.parametrize("dtype,m", [("f32", 1), ("bf16", 1), ("f32", 3), ("bf16", 5)])
def test_long_sums(dtype, m):
    n, k = 5, 1 << 18
    rng = np.random.default_rng([54, m])
    wg, wu = blocks(rng, n, k), blocks(rng, n, k)
    check(rng.standard_normal((m, k)), dtype, n, wg, wu)
