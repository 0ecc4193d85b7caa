"""CPU: the references of the norm, dropout and balance tests against published
vectors, differences and automatic differentiation."""
import numpy as np
import pytest
import torch

import norm_ref as ref


def test_generator_known_answers():
    # known-answer vectors of Philox4x32-10, published with the method
    for c, k, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        assert tuple(int(v) for v in ref.philox(c, k)) == want


def test_share_that_is_kept():
    rows, cols, p = 400, 1001, 0.3
    k = ref.kept(rows, cols, p, 12345, 678)
    n = rows * cols
    m = ref.dropped_of(p) / 65536
    assert abs(float((~k).sum()) - n * m) < 6 * np.sqrt(n * m * (1 - m))  # six standard deviations
    assert not torch.equal(k, ref.kept(rows, cols, p, 12345, 679))
    assert torch.equal(k[:7, :100], ref.kept(7, 100, p, 12345, 678))  # a function of row and column


def total(r, grad_r, grad_h):
    got = r.r()[0]
    out = 0.0
    if grad_r is not None:
        out = out + (got * grad_r).sum()
    if grad_h is not None:
        out = out + (got * ref.inverse_rms(got, r.eps) * r.w * grad_h).sum()
    return out


@pytest.mark.parametrize("post,gates,p,gr,gh", [(True, 1, 0.0, True, True), (False, 3, 0.2, True, True),
                                                (True, 6, 0.4, False, True), (True, 0, 0.0, True, False)])
def test_gradients_against_differences(post, gates, p, gr, gh):
    g = torch.Generator().manual_seed(1)
    rows, hidden = 6, 11

    def randn(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    leaves = dict(x=randn(rows, hidden), y=randn(rows, hidden), weight=randn(hidden))
    if post:
        leaves["post_weight"] = randn(hidden)
    if gates:
        leaves["gate"] = randn(gates, hidden)
    more = dict(post=post, scale=0.5, dropout=p, seed=9, offset=3)
    grad_r, grad_h = (randn(rows, hidden) if t else None for t in (gr, gh))
    if grad_h is None:
        leaves.pop("weight")
    at = ref.Ref(**leaves, **more)
    got = at.backward(grad_r, grad_h, at.r()[0])
    for name, leaf in leaves.items():
        step = randn(*leaf.shape)
        ends = [total(ref.Ref(**dict(leaves, **{name: leaf + s * 1e-6 * step}), **more), grad_r, grad_h) for s in (1, -1)]
        want = float((got[name][0] * step).sum())
        # differences over 1e-6: 2^-53 * the total's terms / 1e-6 of rounding, and 1e-12 * third derivatives
        assert abs(float(ends[0] - ends[1]) / 2e-6 - want) < 1e-6 * (1 + abs(want))
        assert bool((got[name][0].abs() <= got[name][1] * (1 + 1e-12)).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    g = torch.Generator().manual_seed(2)
    l = torch.randn(13, 6, generator=g, dtype=torch.float64)
    l[3, 2] = -float("inf")
    idx = torch.randint(-1, 6, (13, 2), generator=g)
    idx[5] = -1
    bounds = [0, 4, 4, 9, 12]
    _, counts, tokens, grad, _ = ref.balance(l, idx, bounds, score)
    assert int(tokens[-1]) == 3 and int(counts.sum()) == int((idx[:12] >= 0).sum())
    step = torch.randn(13, 6, generator=g, dtype=torch.float64)
    ends = [ref.balance(l + s * 1e-6 * step, idx, bounds, score)[0] for s in (1, -1)]
    assert abs((ends[0] - ends[1]) / 2e-6 - float((grad * step).sum())) < 1e-8
    even = ref.balance(torch.zeros(12, 6), torch.arange(12)[:, None] % 6, [0, 12], score)[0]
    assert abs(even - 1.0) < 1e-12
