"""Tensors whose memory may not be written are read, and one whose memory cannot be had
at all is an error, not the end of the process."""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import _device, activations, blocks, dev, lora_inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]


def test_inputs_that_share_memory_until_written_keep_it():
    """Lazy clones stay lazy: a call reads its inputs and makes no copies of them."""
    m, n, k = 4, 40, 512
    rng = np.random.default_rng([81])
    w, xt, _, at, _, bt, _, s = lora_inputs(rng, "bf16", m, n, k, 8, 2)
    w, w2, s = dev(w), dev(blocks(rng, n, k)), dev(s)
    ids = torch.tensor([0, 1, -1, 1], dtype=torch.int32, device="cuda:0")
    dh, _ = activations(rng, m, n, torch.bfloat16)

    def run(f):
        h, g, u = q2k.gated_ffn(f(xt), f(w), f(w2), n, save=True)
        back = q2k.gated_ffn_backward(f(dh), f(g), f(u), f(w), f(w2), k)
        return (h, g, u, *back, q2k.matmul_lora(f(xt), f(w), n, f(at), f(bt), f(ids), scales=f(s)))

    clones = []

    def lazy(t):
        clones.append(torch._lazy_clone(t))
        return clones[-1]

    plain, shared = run(lambda t: t), run(lazy)
    assert all(torch.equal(p, q) for p, q in zip(plain, shared))
    assert all(torch._C._is_cow_tensor(t) for t in clones)


def test_memory_that_may_not_be_written_is_read():
    m, n, k = 4, 40, 512
    rng = np.random.default_rng([82])
    w, w2 = dev(blocks(rng, n, k)), dev(blocks(rng, n, k))
    x, _ = activations(rng, m, k, torch.bfloat16)
    h = q2k.gated_ffn(x, w, w2, n)
    fixed = x.clone()
    torch._C._set_throw_on_mutable_data_ptr(fixed)  # (a writer's pointer raises)
    assert torch.equal(q2k.gated_ffn(fixed, w, w2, n), h)


def test_tensors_without_memory_are_refused():
    """(the pointer of such a tensor is null, or raises)"""
    from torch._subclasses.fake_tensor import FakeTensorMode

    assert q2k._quick()
    torch.cuda.current_device()
    with FakeTensorMode():
        x = torch.zeros(4, 256, device="cuda:0")
        w = torch.zeros(84 * 8, dtype=torch.uint8, device="cuda:0")
        with pytest.raises((q2k.InvalidArgument, RuntimeError)):
            q2k.gated_ffn(x, w, w, 8)


def test_unknown_names_are_said():
    n, k = 8, 256
    w = dev(blocks(np.random.default_rng(83), n, k))
    x = torch.zeros(2, k, device="cuda:0")
    a, b = torch.zeros(1, 8, k, device="cuda:0").bfloat16(), torch.zeros(1, n, 8, device="cuda:0").bfloat16()
    dh = torch.zeros(2, n, device="cuda:0").bfloat16()
    with pytest.raises(KeyError, match="act must be one of 'silu', 'gelu', got 'relu'"):
        q2k.gated_ffn(x, w, w, n, act="relu")
    with pytest.raises(KeyError, match="act must be"):
        q2k.gated_ffn_backward(dh, dh, dh, w, w, k, act="Gelu")
    for call in (lambda: q2k.gated_ffn(x, w, w, n, path="fast"),
                 lambda: q2k.matmul_lora(x, w, n, a, b, torch.zeros(2, dtype=torch.int32, device="cuda:0"),
                                         path="fast")):
        with pytest.raises(KeyError, match="path must be one of"):
            call()
