"""GPU: the mixture-of-experts calls run together, as a layer and in a CUDA graph.

The layer is compared with the same layer in float64, with the router's choice
taken from the kernels.  Its bounds (in the Frobenius norm) follow from the
products' rounding to e4m3: a value keeps 4 significant bits, so its relative
error is at most 2^-4, at most 2^-4 / sqrt(3) = 0.036 in the mean square, and a
product of two such factors is off by sqrt(2) * 0.036 = 0.051.  silu changes a
relative error of its argument at most twofold here (slope at most 1.1, norm of
the result at least 0.55 of the argument's): the second product's error is at
most sqrt(0.102^2 + 2 * 0.036^2) = 0.114, and a gradient that passes another
product and silu' at most sqrt(0.114^2 + 0.102^2 + 2 * 0.036^2) = 0.161."""
import importlib.util
import os

import pytest
import torch

from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu
OUT_BOUND, GRAD_BOUND = 0.12, 0.17


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


@pytest.fixture(scope="module")
def example(z):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inner,capacity,route", [
    (300, 8, 2, 256, 128, 40, dict()),
    (129, 16, 4, 200, 72, 0, dict(score="sigmoid", groups=4, top_groups=2, scale=2.5)),
    (1, 8, 2, 256, 128, 1, dict(score="sigmoid")),
    (700, 4, 1, 136, 264, 1 << 20, dict(renormalize=False)),
])
def test_layer_forward_and_backward(example, tokens, experts, top_k, hidden, inner, capacity, route):
    layer = example.MoeLayer(experts, top_k, hidden, inner, capacity=capacity, seed=3, **route)
    gen = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16()
    grad = torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16()
    out = layer.forward(x)
    got = (out, *layer.backward(grad))
    _, logits, idx, weights, d, rows, *_ = layer.kept
    layer.check_status()
    assert torch.equal(rows, d.rows)  # the wire is lossless
    assert int(d.offsets[-1]) == tokens * top_k and layer.payload_bytes == 2 * tokens * top_k * hidden

    leaves = [t.double().requires_grad_() for t in (x, layer.router, layer.w_up, layer.w_down)]
    xd, router, up, down = leaves
    ld = xd @ router.t()
    p = torch.softmax(ld, 1) if route.get("score", "softmax") == "softmax" else torch.sigmoid(ld)
    w = p.gather(1, idx.long())
    if route.get("renormalize", True):
        w = w / w.sum(1, keepdim=True)
    w = w * route.get("scale", 1.0)
    want = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    for e in range(experts):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        y = torch.nn.functional.silu(xd[t] @ up[e].t()) @ down[e].t()
        want = want.index_add(0, t, y * w[t, k, None])
    want.backward(grad.double())
    assert off(out, want.detach()) < OUT_BOUND
    for g, leaf in zip(got[1:], leaves):
        if float(leaf.grad.norm()) < 1e-9 * float(leaf.detach().norm()):  # one expert, renormalised: no gradient at all
            continue
        assert off(g, leaf.grad) < GRAD_BOUND


def test_calls_in_a_graph(z):
    """One capture, replayed on other inputs, with calls outside the graph in between."""
    tokens, experts, top_k, hidden, n = 40, 8, 2, 256, 128
    moe, fp8 = z.Moe(experts, top_k), z.BlockFp8()
    gen = torch.Generator(device="cuda").manual_seed(5)
    weight = fp8.quantize_weight(torch.randn(experts, n, hidden, generator=gen, device="cuda").bfloat16())
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros(tokens, experts, device="cuda")

    def step():
        idx, w = moe.route(logits)
        d = moe.dispatch(x, idx)
        return moe.combine(fp8.linear(d.rows, weight, d.offsets), d.pos, w)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for g, out in reversed(graphs):  # the second capture must not lean on the first
        x.copy_(torch.randn(tokens, hidden, generator=gen, device="cuda"))
        logits.copy_(torch.randn(tokens, experts, generator=gen, device="cuda"))
        g.replay()
        got = out.clone()
        assert torch.equal(got, step())
        g.replay()
        assert torch.equal(out, got)
    moe.check_status()
    fp8.check_status()
