"""GPU: the norms, the residual join, dropout and the balance loss run together, around
the mixture-of-experts layer and in a CUDA graph.

The block is compared with the same block in float64, with the router's choice taken
from the kernels and the dropout's masks from the generator's plain form.  The layer's
output is off by at most 0.114 in the mean square, and its gradients by 0.161 (e4m3
products, as in the layer's own test); dividing a row by its size keeps a relative
error up to second order (0.114^2 = 0.013), so the joined residual and its norm are
off by less than 0.13.  The gradients of the two weights behind the layer are sums of
products with one such factor: the same.  That of the layer's output takes its norm's
direction from an output that is 0.114 off, of which the projection keeps a part of
order 1 / sqrt(hidden); what reaches the layer's own gradients is 0.161 and the
e4m3 products' 0.114 in the rows they are taken with, sqrt(0.161^2 + 0.114^2) = 0.197."""
import pytest
import torch

import norm_ref as ref
from gpu_util import load_lib, require_gpu
from test_gpu_moe_layer import example, off  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
OUT_BOUND, GRAD_BOUND = 0.13, 0.2


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inner,dropout,bounds,route", [
    (300, 8, 2, 256, 128, 0.0, None, dict()),
    (257, 8, 2, 264, 136, 0.25, [0, 100, 100, 200], dict(score="sigmoid")),
    (1, 4, 2, 256, 128, 0.1, None, dict()),
])
def test_block_forward_and_backward(example, tokens, experts, top_k, hidden, inner, dropout, bounds, route):  # noqa: F811
    block = example.MoeBlock(experts, top_k, hidden, inner, capacity=20, scale=0.7, dropout=dropout, balance=50.0, seed=3, **route)
    gen = torch.Generator(device="cuda").manual_seed(tokens)

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    for w in (block.weight, block.post_weight, block.next_weight):
        w.copy_(1 + 0.2 * randn(hidden))
    x, grad_r, grad_h = (randn(tokens, hidden).bfloat16() for _ in range(3))
    seq = None if bounds is None else torch.tensor(bounds, dtype=torch.int32, device="cuda")
    r, h, loss = block.forward(x, step=5, sequences=seq)
    got = block.backward(grad_r, grad_h)
    block.check_status()
    layer = block.layer
    _, logits, idx, _, d, *_ = layer.kept

    leaves = [t.double().requires_grad_() for t in (x, block.weight, block.post_weight, block.next_weight, layer.router, layer.w_up, layer.w_down)]
    xd, w1, w2, w3, router, up, down = leaves

    def unit(v, w):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w

    hd = unit(xd, w1)
    ld = hd @ router.t()
    p = torch.softmax(ld, 1) if route.get("score", "softmax") == "softmax" else torch.sigmoid(ld)
    w = p.gather(1, idx.long())
    w = w / w.sum(1, keepdim=True)
    yd = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    rows = d.pos.long()
    keep = ref.kept(tokens * top_k, inner, dropout, 3, 5).cuda() if dropout else None
    for e in range(experts):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        a = torch.nn.functional.silu(hd[t] @ up[e].t())
        if dropout:
            a = torch.where(keep[rows[t, k]], a * ref.gain(dropout), 0.0)
        yd = yd.index_add(0, t, (a @ down[e].t()) * w[t, k, None])
    b = unit(yd, w2) * 0.7
    if dropout:
        b = torch.where(ref.kept(tokens, hidden, dropout, 4, 5).cuda(), b * ref.gain(dropout), 0.0)
    rd = xd + b
    q = p / p.sum(1, keepdim=True)
    losses = []
    for lo, hi in zip((bounds or [0, tokens])[:-1], (bounds or [0, tokens])[1:]):
        if hi > lo:
            f = torch.bincount(idx[lo:hi].flatten().long(), minlength=experts).double()
            losses.append(experts * (f / f.sum() * q[lo:hi].mean(0)).sum())
    balance = 50.0 * sum(losses) / len(losses)
    ((rd * grad_r.double()).sum() + (unit(rd, w3) * grad_h.double()).sum() + balance).backward()
    assert off(r, rd.detach()) < OUT_BOUND and off(h, unit(rd, w3).detach()) < OUT_BOUND
    # the logits are BF16 (2^-8 of values up to 5): shares are off by less than 2 %
    balance = float(balance.detach())
    assert abs(float(loss) - balance) < 0.02 * balance
    for name, g, leaf in zip(("x", "weight", "post_weight", "next_weight", "router", "up", "down"), got, leaves):
        assert g.shape == leaf.shape
        assert off(g, leaf.grad) < GRAD_BOUND, name


def test_calls_in_a_graph(z):
    """A training step's calls without the exchange, captured twice and replayed on other inputs with other masks, beside
    eager calls on another stream."""
    tokens, experts, top_k, hidden = 90, 16, 4, 512
    moe, norm, drop = z.Moe(experts, top_k), z.ResidualNorm(hidden, post=True, dropout=0.2, seed=1), z.Dropout(0.2, seed=2)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16()
    logits = torch.randn(tokens, experts, generator=gen, device="cuda")
    w = torch.randn(hidden, generator=gen, device="cuda")
    gate = torch.randn(2, hidden, generator=gen, device="cuda").bfloat16()
    offset = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step(offset):
        h = norm.norm(x, w)
        idx, weights = moe.route(logits)
        b = moe.balance(logits, idx)
        d = moe.dispatch(h, idx)
        rows = drop.apply(d.rows, offset)
        y = moe.combine(rows, d.pos, weights)
        r, h2 = norm.add(x, y, w, post_weight=w, gate=gate, offset=offset)
        g = norm.add_backward(r, h2, r, y, w, post_weight=w, gate=gate, offset=offset)
        grad_rows, grad_weights = moe.combine_backward(g.y, rows, d.pos, weights, d.offsets)
        grad_h = moe.combine(drop.apply(grad_rows, offset), d.pos)
        grad_logits = moe.balance_backward(logits, idx, b, out=moe.route_backward(logits, idx, grad_weights))
        return [r, h2, b.loss, b.counts, g.weight, g.post_weight, g.gate, grad_logits, *norm.norm_backward(grad_h, x, w, residual=g.x)]

    step(offset)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(offset)
            offset += 1
        graphs.append((g, out))
    offset.zero_()
    other = torch.cuda.Stream()
    for i, (g, out) in enumerate(reversed(graphs * 2)):
        x.copy_(torch.randn(tokens, hidden, generator=gen, device="cuda"))
        logits.copy_(torch.randn(tokens, experts, generator=gen, device="cuda"))
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(other):
            want = step(i)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    moe.check_status()
    norm.check_status()


def test_residual_gradient_of_a_norm_alone(z):
    norm = z.ResidualNorm(200)
    x, grad, up = (torch.randn(7, 200, device="cuda") for _ in range(3))
    gx, _ = norm.norm_backward(grad, x)
    both, _ = norm.norm_backward(grad, x, residual=up)
    # one addition, the terms of up to 4 in size
    assert float((both - (gx + up)).abs().max()) <= 4 * 2.0 ** -22
    with pytest.raises(ValueError):
        norm.norm_backward(grad, x, residual=up.bfloat16())
