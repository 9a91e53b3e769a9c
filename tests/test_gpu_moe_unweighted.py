"""Rows combined without weights: their gradient is the sort of y's, as the documentation
says, and the same as that of weights of one."""

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import DT, _device, activations, dev, host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,top_k,width", [(1, 1, 8), (30, 2, 65), (17, 8, 256)])
def test_gradient_without_weights(tokens, top_k, width, dtype):
    rng = np.random.default_rng([401, tokens])
    ids = dev(rng.integers(-1, 5, (tokens, top_k)).astype(np.int32))
    routes = q2k.moe_route(ids, 5)
    dy, dyv = activations(rng, tokens, width, DT[dtype])
    dys = q2k.moe_sort(dy, routes)
    # y = sum over the choices with an expert: row p's gradient is its token's (a copy:
    # exact), and nothing reaches the rows behind the last expert's
    order, end = routes.order.cpu().numpy(), int(routes.offsets[-1])
    ref = np.where(np.arange(tokens * top_k)[:, None] < end, dyv[order // top_k], 0)
    assert np.array_equal(host(dys), ref)
    ys = activations(rng, tokens * top_k, width, DT[dtype])[0]
    assert torch.equal(q2k.moe_combine(ys, routes),
                       q2k.moe_combine(ys, routes, weights=torch.ones(tokens, top_k, device="cuda:0")))
    again, _ = q2k.moe_combine_backward(dy, ys, routes, torch.ones(tokens, top_k, device="cuda:0"))
    assert torch.equal(again, dys)
    with pytest.raises(TypeError, match="weights"):
        q2k.moe_combine_backward(dy, ys, routes, None)
