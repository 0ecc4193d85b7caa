"""A mixture-of-experts layer around a compressed all-to-all, forward and backward.

    router logits -> route -> dispatch (with the segment table) -> batched
    compression -> [the wire] -> decompression -> the experts' two block-scaled
    e4m3 products -> combine

The exchange stands for the all-to-all: with one GPU every expert is local, so
the streams that would be sent are decoded in place of the received ones.  The
wire carries each expert's static part (its first `capacity` rows) and the rest
as streams of their own; the sizes are read by the host, as an all-to-all's
are, and nothing else of a step visits it.

    python examples/moe_layer.py [--tokens 4096 --hidden 2048 --inner 1024 --experts 64 --top-k 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_bf16_exponent_split_gb300 as z  # noqa: E402


class MoeLayer:
    """silu(rows W_up^T) W_down^T of the chosen experts, weighted by the router."""

    def __init__(self, experts, top_k, hidden, inner, *, capacity, sigma=1.0, seed=0, **route):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5

        self.capacity = capacity
        self.moe = z.Moe(experts, top_k, **route)
        self.fp8 = z.BlockFp8()
        self.codec = z.Codec()
        self.lut = z.zccl_lut_from_sigma(sigma)
        self.router = weight(experts, hidden).bfloat16()
        self.bias = torch.zeros(experts, device="cuda")
        self.w_up, self.w_down = weight(experts, inner, hidden), weight(experts, hidden, inner)
        self.up = self.fp8.quantize_weight(self.w_up, backward=True)
        self.down = self.fp8.quantize_weight(self.w_down, backward=True)
        self.wire_bytes = self.payload_bytes = 0

    def exchange(self, d):
        """The dispatch's rows after the wire, bit for bit."""
        segments = 2 * self.moe.experts
        hidden = d.rows.shape[1]
        sizes = self.codec.compress_batched([None] * segments, self.lut, total_n=d.rows.numel(), table=d.table)
        table = d.table.cpu().numpy().view(z.codec.SEGMENT_DTYPE)
        sizes = sizes.tolist()
        received = torch.zeros_like(d.rows)
        flat, row = received.view(torch.int16).flatten(), 0
        for (_, n, out, _), size in zip(table.tolist(), sizes):
            if n:
                first = out - d.streams.data_ptr()
                self.codec.decompress(d.streams[first:first + size], size, n, out=flat[row * hidden:row * hidden + n])
                row += n // hidden
        self.wire_bytes, self.payload_bytes = sum(sizes), 2 * row * hidden
        return received

    def forward(self, x):
        logits = x @ self.router.t()
        idx, weights = self.moe.route(logits, self.bias)
        d = self.moe.dispatch(x, idx, capacity=self.capacity)
        rows = self.exchange(d)
        h = self.fp8.linear(rows, self.up, d.offsets)
        a = torch.nn.functional.silu(h)
        y = self.fp8.linear(a, self.down, d.offsets)
        self.kept = x, logits, idx, weights, d, rows, h, a, y
        return self.moe.combine(y, d.pos, weights)

    def backward(self, grad):
        """Gradients of (x, router, up, down) from the gradient of forward's output."""
        x, logits, idx, weights, d, rows, h, a, y = self.kept
        grad_y, grad_weights = self.moe.combine_backward(grad, y, d.pos, weights, d.offsets)
        grad_a, grad_down = self.fp8.linear_backward(grad_y, a, self.down, d.offsets)
        s = torch.sigmoid(h.float())
        grad_h = (grad_a.float() * s * (1 + h.float() * (1 - s))).bfloat16()
        grad_rows, grad_up = self.fp8.linear_backward(grad_h, rows, self.up, d.offsets)
        grad_logits = self.moe.route_backward(logits, idx, grad_weights)
        grad_x = self.moe.combine(grad_rows, d.pos) + grad_logits @ self.router
        return grad_x, grad_logits.t() @ x, grad_up, grad_down

    def check_status(self):
        for part in (self.moe, self.fp8, self.codec):
            part.check_status("moe layer")


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inner", 1024), ("experts", 64), ("top-k", 8)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    layer = MoeLayer(a.experts, a.top_k, a.hidden, a.inner, capacity=a.tokens * a.top_k // a.experts, score="sigmoid")
    for tokens in (a.tokens, 1):  # a training step, a serving step
        x = torch.randn(tokens, a.hidden, device="cuda").bfloat16()
        out = layer.forward(x)
        layer.check_status()
        print(f"{tokens} tokens: output {tuple(out.shape)}, {layer.wire_bytes} bytes sent for {layer.payload_bytes}")
        if tokens > 1:
            grads = layer.backward(torch.randn_like(out))
            layer.check_status()
            print("gradients: " + ", ".join(f"{n} {tuple(g.shape)}" for n, g in zip(("x", "router", "up", "down"), grads)))


if __name__ == "__main__":
    main()
