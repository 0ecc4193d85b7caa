"""A mixture-of-experts layer around a compressed all-to-all, and the block of a model
that it is, forward and backward.

    router logits -> route -> dispatch (with the segment table) -> batched
    compression -> [the wire] -> decompression -> the experts' two block-scaled
    e4m3 products -> combine

The block norms the residual for the layer, norms the layer's output, joins it with
the residual (with dropout), norms that for the next block, and has a loss that keeps
the experts balanced.

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

    def __init__(self, experts, top_k, hidden, inner, *, capacity, sigma=1.0, seed=0, dropout=0.0, **route):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5

        self.capacity = capacity
        self.moe = z.Moe(experts, top_k, **route)
        self.fp8 = z.BlockFp8()
        self.codec = z.Codec()
        self.dropout = z.Dropout(dropout, seed=seed) if dropout else None
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

    def forward(self, x, step=0, train=True):
        """step: another one for each call has another dropout mask; train: False for an evaluation, without one."""
        logits = x @ self.router.t()
        idx, weights = self.moe.route(logits, self.bias)
        d = self.moe.dispatch(x, idx, capacity=self.capacity)
        rows = self.exchange(d)
        h = self.fp8.linear(rows, self.up, d.offsets)
        a = torch.nn.functional.silu(h)
        self.drops = self.dropout if train else None
        if self.drops:
            a = self.drops.apply(a, offset=step)
        y = self.fp8.linear(a, self.down, d.offsets)
        self.kept, self.step = (x, logits, idx, weights, d, rows, h, a, y), step
        return self.moe.combine(y, d.pos, weights)

    def backward(self, grad, balance=None, sequences=None, coefficient=1.0):
        """Gradients of (x, router, up, down) from the gradient of forward's output, and
        of the balance loss where that is given (Moe.balance's)."""
        x, logits, idx, weights, d, rows, h, a, y = self.kept
        grad_y, grad_weights = self.moe.combine_backward(grad, y, d.pos, weights, d.offsets)
        grad_a, grad_down = self.fp8.linear_backward(grad_y, a, self.down, d.offsets)
        if self.drops:
            grad_a = self.drops.apply(grad_a, offset=self.step)
        s = torch.sigmoid(h.float())
        grad_h = (grad_a.float() * s * (1 + h.float() * (1 - s))).bfloat16()
        grad_rows, grad_up = self.fp8.linear_backward(grad_h, rows, self.up, d.offsets)
        grad_logits = self.moe.route_backward(logits, idx, grad_weights)
        if balance is not None:
            self.moe.balance_backward(logits, idx, balance, sequences, coefficient, out=grad_logits)
        grad_x = self.moe.combine(grad_rows, d.pos) + grad_logits @ self.router
        return grad_x, grad_logits.t() @ x, grad_up, grad_down

    def check_status(self):
        for part in (self.moe, self.fp8, self.codec):
            part.check_status("moe layer")


class MoeBlock:
    """h = N(x), r = x + scale * drop(N(layer(h))), and N(r) for the next block.  A handle's
    dropout is its own: evaluations have a second one without."""

    def __init__(self, experts, top_k, hidden, inner, *, scale=1.0, dropout=0.0, balance=0.01, seed=0, **layer):
        self.layer = MoeLayer(experts, top_k, hidden, inner, seed=seed, dropout=dropout, **layer)
        self.norm = z.ResidualNorm(hidden, post=True, scale=scale, dropout=dropout, seed=seed + 1)
        self.plain = z.ResidualNorm(hidden, post=True, scale=scale)
        self.weight, self.post_weight, self.next_weight = (torch.ones(hidden, device="cuda") for _ in range(3))
        self.coefficient = balance

    def forward(self, x, step=0, sequences=None, train=True):
        """(the residual behind the block, the next block's input, the balance loss);
        sequences: where each sequence of the batch begins, and where the last ends;
        train: False for an evaluation, where nothing is dropped."""
        norm = self.norm if train else self.plain
        h = norm.norm(x, self.weight)
        y = self.layer.forward(h, step, train)
        _, logits, idx, *_ = self.layer.kept
        balance = self.layer.moe.balance(logits, idx, sequences, self.coefficient)
        r, h_next = norm.add(x, y, self.next_weight, post_weight=self.post_weight, offset=step)
        self.kept = norm, x, y, r, balance, sequences, step
        return r, h_next, balance.loss

    def backward(self, grad_r, grad_h):
        """Gradients of (x, weight, post_weight, next_weight, router, up, down) from those of
        the residual behind the block and the next block's input, and of the balance loss."""
        norm, x, y, r, balance, sequences, step = self.kept
        g = norm.add_backward(grad_r, grad_h, r, y, self.next_weight, post_weight=self.post_weight, offset=step)
        grad_in, *grads = self.layer.backward(g.y, balance, sequences, self.coefficient)
        grad_x, grad_weight = norm.norm_backward(grad_in, x, self.weight, residual=g.x)
        return grad_x, grad_weight, g.post_weight, g.weight, *grads

    def check_status(self):
        self.layer.check_status()
        for norm in (self.norm, self.plain):
            norm.check_status("moe block")


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inner", 1024), ("experts", 64), ("top-k", 8)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    block = MoeBlock(a.experts, a.top_k, a.hidden, a.inner, capacity=a.tokens * a.top_k // a.experts, score="sigmoid",
                     dropout=0.1)
    layer = block.layer
    names = ("x", "weight", "post weight", "next weight", "router", "up", "down")
    for step, tokens in enumerate((a.tokens, 1)):  # a training step, a serving step
        x = torch.randn(tokens, a.hidden, device="cuda").bfloat16()
        r, h, loss = block.forward(x, step, train=tokens > 1)
        block.check_status()
        print(f"{tokens} tokens: output {tuple(r.shape)}, {layer.wire_bytes} bytes sent for {layer.payload_bytes}, "
              f"balance loss {loss.item():.4f}")
        if tokens > 1:
            grads = block.backward(torch.randn_like(r), torch.randn_like(h))
            block.check_status()
            print("gradients: " + ", ".join(f"{n} {tuple(g.shape)}" for n, g in zip(names, grads)))


if __name__ == "__main__":
    main()
