"""GPU: the router on more than 4096 tokens, where several tokens share a warp:
against 64-bit numpy, and bit for bit against the same rows in smaller calls,
which a whole warp a token takes."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu

WEIGHT_RTOL = 64 * 2.0 ** -24  # as for the smaller calls: under 64 roundings of 2^-24
CHUNK = 1500


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


def in_chunks(moe, l, bias):
    parts = [moe.route(l[i:i + CHUNK], bias) for i in range(0, l.shape[0], CHUNK)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def bits(t):
    return t.view(torch.int32)


CASES = [(t, e, k) for t, e in ((4097, 5), (5003, 16), (4099, 17), (4098, 32), (5003, 33), (4099, 64)) for k in (1, 3, 8) if k <= e]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("t,e,k", CASES)
def test_many_tokens(z, t, e, k, score, renorm, dtype, bias):
    rng = np.random.default_rng(100 * t + e)
    values = rng.normal(size=(t, e)) * 2
    half = rng.random(t) < 0.25
    values[half] = np.round(values[half])  # rows with many ties
    masked = rng.random((t, e)) < 0.1
    masked[rng.random(t) < 0.05] = True    # and rows that leave nothing
    l = torch.from_numpy(np.where(masked, -np.inf, values).astype(np.float32)).to(dtype)
    b = (rng.integers(-100, 101, e) / 1000).astype(np.float32) if bias else None
    bd = None if b is None else torch.from_numpy(b).cuda()
    moe = z.Moe(e, k, score=score, renormalize=renorm, scale=1.25)
    idx, w = moe.route(l.cuda(), bd)
    small_idx, small_w = in_chunks(moe, l.cuda(), bd)
    assert torch.equal(idx, small_idx) and torch.equal(bits(w), bits(small_w))
    assert moe.read_status() == z.OK
    some = np.r_[0:70, t - 70:t]
    want_idx, want_w, margin = ref.route(l.double().numpy()[some], b, score, k, renorm=renorm, scale=1.25)
    clear = margin > 1e-5  # ten times the error of a value in 32 bits
    assert clear.mean() > 0.7
    assert np.array_equal(idx.cpu().numpy()[some][clear], want_idx[clear])
    np.testing.assert_allclose(w.cpu().numpy()[some][clear], want_w[clear], rtol=WEIGHT_RTOL, atol=1e-30)


@pytest.mark.parametrize("e", [9, 24, 64])
def test_ties_go_to_the_lowest_index(z, e):
    """Whole-number logits from a few values: the choice is a stable sort, whatever lane holds an expert."""
    rng = np.random.default_rng(e)
    l = rng.integers(0, 3, (4500, e)).astype(np.float32)
    idx, _ = z.Moe(e, 8).route(torch.from_numpy(l).cuda())
    assert np.array_equal(idx.cpu().numpy(), np.argsort(-l, axis=1, kind="stable")[:, :8])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_bad_row_leaves_its_warp_s_other_rows_alone(z, score):
    gen = torch.Generator(device="cuda").manual_seed(4)
    l = torch.randn(4203, 64, generator=gen, device="cuda")
    moe = z.Moe(64, 8, score=score)
    idx, w = moe.route(l)
    assert moe.read_status() == z.OK
    bad = [0, 5, 10, 15, 18, 19, 2000, 4202]  # each place of a warp's four rows, two of one warp, the last row
    spoilt = l.clone()
    for i, r in enumerate(bad):
        spoilt[r, (9 * i) % 64] = float("nan")
    got_idx, got_w = moe.route(spoilt)
    assert moe.read_status() == z.INVALID_ARG
    good = torch.ones(4203, dtype=torch.bool, device="cuda")
    good[bad] = False
    assert torch.equal(got_idx[good], idx[good]) and torch.equal(bits(got_w[good]), bits(w[good]))
    assert (got_idx[bad] == -1).all() and not got_w[bad].any()


def test_strided_rows_and_a_row_for_every_token(z):
    gen = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn(4500, 90, generator=gen, device="cuda")
    moe = z.Moe(61, 8)
    view = wide[:, 3:64]
    a, b = moe.route(view), moe.route(view.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(bits(a[1]), bits(b[1]))
    one = view[:1].expand(4500, 61)
    got = moe.route(one)
    assert torch.equal(got[0], a[0][:1].expand(4500, 8)) and torch.equal(bits(got[1]), bits(a[1][:1].expand(4500, 8).contiguous()))
