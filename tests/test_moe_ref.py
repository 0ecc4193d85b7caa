"""The numpy reference of the routing itself: its gradient formulas against
central differences, and hand-worked choices."""
import numpy as np
import pytest

import moe_ref as ref


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_formulas_match_differences(kind, renorm):
    rng = np.random.default_rng(3)
    l = rng.normal(size=(5, 9)) * 2
    l[1, 3] = -np.inf
    idx, w, _ = ref.route(l, None, kind, 4, renorm=renorm, scale=1.7)
    gw = rng.normal(size=w.shape)
    got = ref.route_grad(l, idx, gw, kind, renorm, 1.7)
    h = 1e-6
    for r in range(l.shape[0]):
        for e in range(l.shape[1]):
            if np.isneginf(l[r, e]):
                assert got[r, e] == 0
                continue
            up, dn = l[r].copy(), l[r].copy()
            up[e] += h
            dn[e] -= h
            chosen = list(idx[r])
            num = ((ref.weights(up, chosen, kind, renorm, 1.7) - ref.weights(dn, chosen, kind, renorm, 1.7)) * gw[r]).sum()
            # central differences: h^2 truncation and 2^-53 / h rounding
            assert abs(num / (2 * h) - got[r, e]) < 1e-8


def test_choices_worked_by_hand():
    l = np.array([[0.0, 2.0, 1.0, 2.0]])
    idx, w, _ = ref.route(l, None, "softmax", 2)
    assert idx.tolist() == [[1, 3]] and np.allclose(w, 0.5)
    # groups {0, 1} and {2, 3}: sums of sigmoids 0.5 + 0.88 against 0.73 + 0.88: the second
    idx, w, _ = ref.route(l, None, "sigmoid", 2, groups=2, top_groups=1)
    assert idx.tolist() == [[3, 2]]
    # one expert left: the other slot is empty
    idx, w, _ = ref.route(np.array([[-np.inf, -np.inf, 3.0, -np.inf]]), None, "softmax", 2)
    assert idx.tolist() == [[2, -1]] and w.tolist() == [[1.0, 0.0]]
    idx, w, _ = ref.route(np.full((1, 4), -np.inf), None, "sigmoid", 2)
    assert idx.tolist() == [[-1, -1]] and w.tolist() == [[0.0, 0.0]]


def test_places_worked_by_hand():
    pos, counts, offsets, order = ref.places(np.array([[1, 0], [-1, 1], [0, 9]]), 2)
    assert pos.tolist() == [[2, 0], [-1, 3], [1, -1]]
    assert counts.tolist() == [2, 2] and offsets.tolist() == [0, 2, 4]
