"""GPU: rows of more than 16384 values, several of them for each CTA: sums over rows that
go on, gate rows within a CTA's rows, over the border of two and over many.

Bounds as in test_gpu_norm.py: a row's sum has at most 16 tiles of 4 pairs a lane and 11 halvings
(139 roundings with the last addition of two), twice for y's gradient; a CTA's rows are at most 4, and the
CTAs' sums at most 303, of which a thread adds 303 / 128 and up, 32 by halves: under 512 in all."""
import pytest
import torch

import norm_ref as ref
from test_gpu_norm import B, F, close, inputs, z  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

CASES = [  # rows, hidden, residual, block, weight, post, gates, scale, dropout
    (700, 16392, B, B, F, True, 0, 1.0, 0.0),
    (700, 16392, B, B, F, True, 7, 0.5, 0.1),      # a gate row over many CTAs
    (700, 16385, F, B, F, True, 350, 1.0, 0.0),    # more gate rows than CTAs, some over a border
    (700, 16385, B, B, B, False, 1, 1.0, 0.1),
    (700, 16392, F, F, F, True, 700, 1.0, 0.1),
    (300, 65536, B, F, F, True, 150, 1.0, 0.1),    # four rows a CTA, with two gate rows
    (300, 65535, F, B, None, False, 100, 0.5, 0.0),
    (301, 40001, B, B, F, True, 43, 1.0, 0.2),
]


@pytest.mark.parametrize("case", CASES)
def test_forward_and_gradients_of_several_rows_a_cta(z, case):  # noqa: F811
    rows, hidden, residual, block, weight, post, gates, scale, dropout = case
    n, x, y, w, more, grad_r, grad_h = inputs(z, *case)
    r, h = n.add(x, y, w, offset=7, **more)
    at = ref.Ref(x=x, y=y, weight=w, post=post, eps=1e-5, scale=scale, dropout=dropout, seed=0xFEDCBA9876543210, offset=7, **more)
    close(r, *at.r(), "r")
    want = at.h(r)
    close(h, want, want.abs(), "h")
    got = n.add_backward(grad_r, grad_h, r, y, w, offset=7, **more)
    wanted = at.backward(grad_r, grad_h, r)
    for name, have in got._asdict().items():
        if have is not None:
            close(have, *wanted[name], name)
    assert (got.gate is None) == (gates == 0) and (got.weight is None) == (weight is None)
    again = n.add_backward(grad_r, grad_h, r, y, w, offset=7, **more)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))
    n.check_status()
