"""The feed-forward example runs, its tuning makes progress, and a prompt's rows are
those of the same tokens served one request at a time, up to the paths' roundings."""

import importlib.util
import os

import pytest

import ggml_q2_quantized_gb300 as q2k

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ff = load()
    losses, y = ff.main(512, 1280, 96, 20)
    assert losses[-1] < losses[0]
    assert torch.isfinite(y.float()).all()
    layer = ff.FeedForward(512, 1280)
    gen = torch.Generator(device="cuda:0").manual_seed(2)
    x = torch.randn(40, 512, device="cuda:0", generator=gen).bfloat16()
    ids = (torch.arange(40, device="cuda:0") % 4).int()
    whole = layer(x, ids).float()
    for i in range(0, 40, 8):
        part = layer(x[i:i + 8].contiguous(), ids[i:i + 8].contiguous()).float()
        # (h and y are rounded to bf16, x and W on the prompt's path: a few 2^-8 of
        # values whose sums have hundreds of terms)
        assert (part - whole[i:i + 8]).abs().max() < 0.05 * whole.abs().max()
    assert q2k.device_error() == 0
