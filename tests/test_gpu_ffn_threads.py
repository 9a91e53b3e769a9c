"""Feed-forward calls from several host threads at once, each on its own stream, from
the first call on: the same bits as one after another."""

import threading

import numpy as np
import pytest

import ggml_q2_quantized_gb300 as q2k
from test_gpu_ffn import _device, activations, blocks, dev, lora_inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

__all__ = ["_device"]

SHAPES = [(1, 70, 2304), (3, 70, 1024), (16, 70, 5120), (40, 200, 1024), (150, 200, 1280), (300, 200, 1024)]


def test_threads():
    work = []
    for m, n, k in SHAPES:
        rng = np.random.default_rng([71, m])
        w, xt, _, at, _, bt, _, s = lora_inputs(rng, "bf16", m, n, k, 16, 3)
        dh, _ = activations(rng, m, n, torch.bfloat16)
        work.append((xt, dev(w), dev(blocks(rng, n, k)), n, k, dh, at, bt,
                     dev(rng.integers(-1, 3, m).astype(np.int32)), dev(s)))

    def run(x, w, w2, n, k, dh, a, b, ids, s):
        h, g, u = q2k.gated_ffn(x, w, w2, n, save=True)
        back = q2k.gated_ffn_backward(dh, g, u, w, w2, k)
        return (h, g, u, *back, q2k.matmul_lora(x, w, n, a, b, ids, scales=s, check=False)[0])

    torch.cuda.synchronize()
    results, errors = [None] * 8, []
    start = threading.Barrier(len(results))

    def worker(i):
        try:
            stream = torch.cuda.Stream()
            start.wait(30)
            with torch.cuda.stream(stream):
                for _ in range(20):
                    out = [run(*work[(i + j) % len(work)]) for j in range(len(work))]
            stream.synchronize()
            results[i] = out
        except Exception as e:  # noqa: BLE001 (shown by the assertion below)
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(results))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors and all(r is not None for r in results)
    alone = [run(*w) for w in work]
    for i, out in enumerate(results):
        for j, got in enumerate(out):
            assert all(torch.equal(p, q) for p, q in zip(got, alone[(i + j) % len(work)]))
