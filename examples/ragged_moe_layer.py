"""A mixture-of-experts layer on the operators for experts with any number of
rows: bf16 training (router, expert SwiGLU MLPs, weighted join, and all their
gradients), then serving with 8-bit integer or floating-point experts, prompts and
single tokens; and blocks of such layers in a residual stream, with the norms
around them.

    python examples/ragged_moe_layer.py [--steps 60]
"""

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_grouped_group_amd as mx  # noqa: E402


@dataclass
class Layer:
    """Master weights fp32: router [E, H], w1 [E, 2F, H] (gate | up), w2 [E, H, F]."""
    router: torch.Tensor
    w1: torch.Tensor
    w2: torch.Tensor
    top_k: int

    @staticmethod
    def random(experts, hidden, ffn, top_k, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        draw = lambda *s: torch.randn(s, generator=gen, device="cuda") / s[-1] ** 0.5  # noqa: E731
        return Layer(draw(experts, hidden), draw(experts, 2 * ffn, hidden), draw(experts, hidden, ffn),
                     top_k)

    def bf16(self):
        return Layer(self.router.bfloat16(), self.w1.bfloat16(), self.w2.bfloat16(), self.top_k)


def _all(rows):
    """m_splits of a product with one expert that owns every row."""
    return torch.full((1,), rows, dtype=torch.int64, device="cuda")


def forward(layer, x, token_mask=None):
    """x [T, H] bf16 -> out [T, H] bf16, and what the backward pass needs."""
    logits = mx.ragged_gemm("NT", x, layer.router[None], _all(len(x)), out_dtype=torch.float32)
    route = mx.moe_route(logits, layer.top_k, token_mask=token_mask)
    h, a = mx.ragged_gemm_swiglu(x, layer.w1, route.m_splits, row_index=route.row_token)
    y = mx.ragged_gemm("NT", a, layer.w2, route.m_splits)
    return mx.moe_combine(y, route.row_pos, route.weights), (x, logits, route, h, y)


def backward(layer, saved, dout):
    """Gradients of x (bf16) and of the weights (fp32)."""
    x, logits, route, h, y = saved
    f32 = torch.float32
    dy, dweights = mx.moe_combine_bwd(dout, y, route.row_pos, route.weights)
    dh, a = mx.ragged_gemm_swiglu_bwd(dy, layer.w2, h, route.m_splits)   # the activation anew
    dw2 = mx.ragged_gemm("TN", dy, a, route.m_splits, out_dtype=f32)
    dw1 = mx.ragged_gemm("TN", dh, x, route.m_splits, row_index=route.row_token, out_dtype=f32)
    dx_rows = mx.ragged_gemm("NN", dh, layer.w1, route.m_splits)
    dlogits = mx.moe_route_bwd(logits, route, dweights).bfloat16()
    drouter = mx.ragged_gemm("TN", dlogits, x, _all(len(x)), out_dtype=f32)[0]
    # a token's gradient: its rows' and the router's
    dx = mx.moe_combine(dx_rows, route.row_pos)
    dx += mx.ragged_gemm("NN", dlogits, layer.router[None], _all(len(x)))
    return dx, Layer(drouter, dw1, dw2, layer.top_k)


@dataclass
class Block:
    """A layer in a residual stream, fp32 weights [H]: `post` normalizes the layer's output
    before it joins the stream (scaled by `scale`), `next` the stream for the next block."""
    layer: Layer
    post: torch.Tensor
    next: torch.Tensor
    scale: float = 1.0


def blocks_forward(blocks, first, x, token_mask=None):
    """x [T, H] bf16, first [H] the norm before the first block -> the last block's normalized
    stream, and what the backward pass needs."""
    stream, y = mx.residual_norm(x, pre_weight=first)
    kept = [stream]
    for b in blocks:
        out, saved = forward(b.layer, y, token_mask)
        stream, y = mx.residual_norm(stream, out, residual_scale=b.scale, post_weight=b.post, pre_weight=b.next)
        kept.append((saved, stream, out))
    return y, kept


def blocks_backward(blocks, first, kept, dy):
    """Gradients of x, of `first` and of each block (as Block, norms fp32)."""
    dstream, grads = None, []
    for b, (saved, stream, out) in zip(blocks[::-1], kept[:0:-1]):
        around = mx.residual_norm_bwd(dy, dstream, stream, out, residual_scale=b.scale, post_weight=b.post,
                                      pre_weight=b.next)
        dy, grad = backward(b.layer, saved, around.f)
        dstream = around.x
        grads.append(Block(grad, around.post_weight, around.pre_weight, b.scale))
    around = mx.residual_norm_bwd(dy, dstream, kept[0], pre_weight=first)
    return around.x, around.pre_weight, grads[::-1]


@dataclass
class Int8Layer:
    """Serving weights, laid out once: codes and the scale of each output channel."""
    router: torch.Tensor
    w1: torch.Tensor
    s1: torch.Tensor
    w2: torch.Tensor
    s2: torch.Tensor
    top_k: int

    @staticmethod
    def of(layer):
        def codes(w):
            q, s = mx.quantize_int8(w.reshape(-1, w.shape[-1]))
            return q.view(w.shape), s.view(w.shape[:2])
        return Int8Layer(layer.router, *codes(layer.w1), *codes(layer.w2), layer.top_k)


def serve(layer, x, token_mask=None):
    """The forward pass with 8-bit integer experts; the router stays bf16."""
    logits = mx.ragged_gemm("NT", x, layer.router[None], _all(len(x)), out_dtype=torch.float32)
    route = mx.moe_route(logits, layer.top_k, token_mask=token_mask)
    q, s = mx.quantize_int8(x)
    h = mx.ragged_gemm_int8(q, s, layer.w1, layer.s1, route.m_splits, row_index=route.row_token)
    q, s = mx.quantize_int8(mx.swiglu_fwd(h))
    y = mx.ragged_gemm_int8(q, s, layer.w2, layer.s2, route.m_splits)
    return mx.moe_combine(y, route.row_pos, route.weights)


@dataclass
class Fp8Layer:
    """The same in 8-bit floating point, a scale for each block of 128 x 128."""
    router: torch.Tensor
    w1: torch.Tensor
    s1: torch.Tensor
    w2: torch.Tensor
    s2: torch.Tensor
    top_k: int

    @staticmethod
    def of(layer):
        return Fp8Layer(layer.router, *mx.quantize_fp8_weight(layer.w1), *mx.quantize_fp8_weight(layer.w2),
                        layer.top_k)


def serve_fp8(layer, x, token_mask=None):
    """The forward pass with 8-bit floating-point experts; the router stays bf16."""
    logits = mx.ragged_gemm("NT", x, layer.router[None], _all(len(x)), out_dtype=torch.float32)
    route = mx.moe_route(logits, layer.top_k, token_mask=token_mask)
    q, s = mx.quantize_fp8(x)
    h = mx.ragged_gemm_fp8(q, s, layer.w1, layer.s1, route.m_splits, row_index=route.row_token)
    q, s = mx.quantize_fp8(mx.swiglu_fwd(h))
    y = mx.ragged_gemm_fp8(q, s, layer.w2, layer.s2, route.m_splits)
    return mx.moe_combine(y, route.row_pos, route.weights)


def train(steps, tokens=1500, experts=16, hidden=512, ffn=768, top_k=2, rate=1.0):
    """Fits a layer to another one's outputs; returns the layer and the losses."""
    teacher = Layer.random(experts, hidden, ffn, top_k, seed=1).bf16()
    layer = Layer.random(experts, hidden, ffn, top_k, seed=2)
    gen = torch.Generator("cuda").manual_seed(3)
    losses = []
    for _ in range(steps):
        x = torch.randn((tokens, hidden), generator=gen, device="cuda").bfloat16()
        want = forward(teacher, x)[0].float()
        low = layer.bf16()
        out, saved = forward(low, x)
        off = out.float() - want
        losses.append(float(off.square().mean()))
        _, grad = backward(low, saved, (off / tokens).bfloat16())
        for name in ("router", "w1", "w2"):
            getattr(layer, name).sub_(getattr(grad, name), alpha=rate)
    return layer, losses


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    steps = ap.parse_args().steps
    layer, losses = train(steps)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    low = layer.bf16()
    served, served_fp8 = Int8Layer.of(low), Fp8Layer.of(low)
    for tokens in (777, 1):
        x = torch.randn((tokens, low.router.shape[1]), device="cuda").bfloat16()
        a = forward(low, x)[0].float()
        for name, b in (("integer", serve(served, x)), ("floating-point", serve_fp8(served_fp8, x))):
            print(f"serving {tokens} token(s): 8-bit {name} output differs from bf16 by "
                  f"{float((a - b.float()).norm() / a.norm()):.4f} of its norm")


if __name__ == "__main__":
    main()
