"""A token that holds an infinity or a NaN has no finite result, however few of its
values those are and whichever kernel takes the call."""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import DT, _device, activations, blocks, dev, lora_inputs

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
