"""The compiled module in front of the feed-forward calls, without a GPU: it takes
only ordinary CUDA tensors and leaves everything else to the Python layer."""

import pytest

import ggml_q2_quantized_gb300 as q2k

torch = pytest.importorskip("torch")


def test_it_is_built():
    assert q2k._quick()


@pytest.mark.parametrize("x", [None, 3, "x", [1.0], torch.zeros(2, 256), torch.zeros(2, 256).half(),
                               torch.zeros(2, 256).bfloat16()])
def test_other_tensors_are_declined(x):
    quick = q2k._quick()
    w = torch.zeros(84, dtype=torch.uint8)
    assert quick.gated(x, w, w, 1, "silu", False, "auto", True) is None
    assert quick.backward(x, x, x, w, w, 256, "silu") is None
    assert quick.lora(x, w, 1, x, x, x, None, "auto", True) is None


@pytest.mark.parametrize("args", [(), (1,), tuple(range(7)), tuple(range(12))])
def test_other_counts_are_declined(args):
    quick = q2k._quick()
    for f, n in ((quick.gated, 8), (quick.backward, 7), (quick.lora, 9)):
        assert f(*(args if len(args) != n else ())) is None


def test_bind_wants_six_addresses():
    quick = q2k._quick()
    with pytest.raises(TypeError):
        quick.bind(1, 2)
    with pytest.raises(ValueError):
        quick.bind(1, 2, 3, 4, 5, 0)
