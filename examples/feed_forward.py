"""A feed-forward layer with frozen Q2_K weights: tuned, prompted and served.

The layer is ``y_i = Wd h_i + s_a B_a (A_a h_i)`` with ``h = act(x Wg^T) * (x Wu^T)``
and an adapter ``a`` for each request.  Three steps use it as a program would:

1. tune: a soft prompt (trainable input vectors) is fitted to a target h through the
   frozen gated block, by its backward pass;
2. prompt: the requests' prompts go through the layer in one batch;
3. serve: one token of each request at a time, the step captured in a CUDA graph.

    python examples/feed_forward.py [hidden inner]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ggml_q2_quantized_gb300 as q2k  # noqa: E402


def random_q2_k(n, k, gen):
    """n rows of Q2_K blocks whose products with unit-variance x are of order one."""
    b = torch.randint(0, 256, (n * (k // 256), 84), device=gen.device, generator=gen, dtype=torch.uint8)
    scale = 1 / (14 * k ** 0.5)  # d; q sc - 1.5 m has a deviation of about 14
    b[:, 80:] = torch.tensor([scale, 1.5 * scale], dtype=torch.float16).view(torch.uint8).to(b.device)
    return b.view(-1)


class FeedForward:
    """Frozen Q2_K projections and the down projection's adapters."""

    def __init__(self, hidden, inner, adapters=4, rank=16, device="cuda:0", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.hidden, self.inner = hidden, inner
        self.gate, self.up = random_q2_k(inner, hidden, gen), random_q2_k(inner, hidden, gen)
        self.down = random_q2_k(hidden, inner, gen)
        self.a = (torch.randn(adapters, rank, inner, device=device, generator=gen) / inner ** 0.5).bfloat16()
        self.b = (torch.randn(adapters, hidden, rank, device=device, generator=gen) / rank ** 0.5).bfloat16()
        self.scales = torch.ones(adapters, device=device)

    def __call__(self, x, ids):
        h = q2k.gated_ffn(x, self.gate, self.up, self.inner, const_weights=True)
        y, _bad = q2k.matmul_lora(h, self.down, self.hidden, self.a, self.b, ids, scales=self.scales,
                                  const_weights=True, check=False)
        return y


class GatedBlock(torch.autograd.Function):
    """The gated block for autograd, its weights frozen."""

    @staticmethod
    def forward(ctx, x, layer):
        h, g, u = q2k.gated_ffn(x, layer.gate, layer.up, layer.inner, save=True)
        ctx.save_for_backward(g, u)
        ctx.layer = layer
        return h

    @staticmethod
    def backward(ctx, dh):
        g, u = ctx.saved_tensors
        layer = ctx.layer
        return q2k.gated_ffn_backward(dh.contiguous(), g, u, layer.gate, layer.up, layer.hidden)[0], None


def tune(layer, tokens, steps, gen):
    """Fit a soft prompt to the h of another input; returns the losses."""
    like = torch.randn(tokens, layer.hidden, device=gen.device, generator=gen).bfloat16()
    target = q2k.gated_ffn(like, layer.gate, layer.up, layer.inner).float()
    x = (like + 0.5 * torch.randn(like.shape, device=gen.device, generator=gen)).float().requires_grad_()
    opt = torch.optim.Adam([x], lr=3e-2)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = (GatedBlock.apply(x.bfloat16(), layer).float() - target).square().mean()
        loss.backward()
        opt.step()
        losses.append(loss.detach().item())
    return losses


def serve(layer, requests, steps, gen):
    """`steps` tokens of each request, one CUDA graph replayed; returns the last y
    and the time of a step in microseconds."""
    x = torch.randn(requests, layer.hidden, device=gen.device, generator=gen).bfloat16()
    ids = (torch.arange(requests, device=gen.device) % layer.a.shape[0]).int()
    layer(x, ids)  # (a kernel's first call sets it up)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, ids)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(steps):
        graph.replay()  # (x would be the step's tokens, copied in)
    end.record()
    end.synchronize()
    return y, 1e3 * start.elapsed_time(end) / steps


def main(hidden=4096, inner=14336, tokens=512, steps=20):
    gen = torch.Generator(device="cuda:0").manual_seed(1)
    layer = FeedForward(hidden, inner)
    losses = tune(layer, tokens // 4, steps, gen)
    print(f"tune: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    x = torch.randn(tokens, hidden, device="cuda:0", generator=gen).bfloat16()
    ids = (torch.arange(tokens, device="cuda:0") * 4 // tokens).int()
    y = layer(x, ids)
    print(f"prompt: {tokens} tokens of 4 requests -> {list(y.shape)}, rms {float(y.float().square().mean()) ** 0.5:.3f}")
    for requests in (1, 4, 16):
        _, us = serve(layer, requests, 50, gen)
        print(f"serve: {requests} requests, {us:.1f} us a step")
    assert q2k.device_error() == 0
    return losses, y


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:3]))
