"""GPU: routing, dispatch and combine against plain 64-bit numpy, at the sizes
and masks where they can go wrong, and the dispatch's segment table through the
batched compression."""
import numpy as np
import pytest
import torch

import moe_ref as ref
import oracle
from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu

# Roundings of a weight in 32 bits: the difference l - max (|l - max| <= 40 units of 2^-24), the exponential (2), a
# sum by halves of at most 512 (9), a quotient and a product: under 64 units of 2^-24.
WEIGHT_RTOL = 64 * 2.0 ** -24


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


def logits_of(rng, t, e, dtype, masked=0.05):
    l = torch.from_numpy((rng.normal(size=(t, e)) * 2).astype(np.float32)).to(dtype)
    m = rng.random((t, e)) < masked
    m[rng.random(t) < masked] = True
    l[torch.from_numpy(m)] = -float("inf")
    return l


ROUTES = [  # tokens, experts, top_k, groups, top_groups, score, renorm, bias, dtype
    (1, 64, 8, 1, 1, "softmax", True, False, torch.float32),
    (1, 1, 1, 1, 1, "sigmoid", False, False, torch.float32),
    (67, 5, 5, 1, 1, "softmax", False, False, torch.bfloat16),
    (129, 60, 4, 1, 1, "softmax", False, True, torch.float32),
    (33, 256, 8, 8, 4, "sigmoid", True, True, torch.float32),
    (40, 160, 6, 8, 3, "softmax", True, False, torch.bfloat16),
    (17, 512, 32, 32, 7, "sigmoid", False, True, torch.float32),
    (23, 96, 7, 3, 2, "sigmoid", True, False, torch.float32),
    (31, 12, 3, 12, 5, "softmax", True, True, torch.float32),
    (2100, 33, 2, 1, 1, "sigmoid", True, True, torch.float32),
]


@pytest.mark.parametrize("t,e,k,g,tg,score,renorm,bias,dtype", ROUTES)
def test_route_and_gradient(z, t, e, k, g, tg, score, renorm, bias, dtype):
    rng = np.random.default_rng(t * 1000 + e)
    l = logits_of(rng, t, e, dtype)
    b = rng.integers(-100, 101, e).astype(np.float32) / 1000 if bias else None
    moe = z.Moe(e, k, score=score, groups=g, top_groups=tg, renormalize=renorm, scale=1.25)
    ld = l.cuda()
    idx, w = moe.route(ld, None if b is None else torch.from_numpy(b).cuda())
    l64 = l.double().numpy()
    want_idx, want_w, margin = ref.route(l64, b, score, k, g, tg, renorm, 1.25)
    clear = margin > 1e-5  # ten times the error of a value in 32 bits
    assert clear.mean() > 0.7
    assert np.array_equal(idx.cpu().numpy()[clear], want_idx[clear])
    np.testing.assert_allclose(w.cpu().numpy()[clear], want_w[clear], rtol=WEIGHT_RTOL, atol=1e-30)
    assert moe.read_status() == z.OK

    gw = rng.normal(size=(t, k)).astype(np.float32)
    got = moe.route_backward(ld, idx, torch.from_numpy(gw).cuda()).float().cpu().numpy()
    want = ref.route_grad(l64, idx.cpu().numpy(), gw, score, renorm, 1.25)
    # an entry is a difference of terms up to scale * max|gw|, each within the weights' error (and K of them added)
    atol = 1.25 * np.abs(gw).max() * (WEIGHT_RTOL + k * 2.0 ** -24)
    np.testing.assert_allclose(got, want, rtol=2.0 ** -8 if dtype == torch.bfloat16 else WEIGHT_RTOL, atol=atol)


def test_route_ties_go_to_the_lowest_index(z):
    l = torch.zeros(3, 70, device="cuda")
    l[1, 40:] = 1.0
    idx, w = z.Moe(70, 4).route(l)
    assert idx.cpu().tolist() == [[0, 1, 2, 3], [40, 41, 42, 43], [0, 1, 2, 3]]
    assert torch.equal(w.cpu(), torch.full((3, 4), 0.25))
    # groups of equal value: the lowest groups
    idx, _ = z.Moe(64, 3, groups=8, top_groups=2, score="sigmoid").route(torch.zeros(2, 64, device="cuda"))
    assert idx.cpu().tolist() == [[0, 1, 2]] * 2


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_lowest_values_do_not_underflow(z, score):
    """Logits at the type's lowest value and far below the others stay finite; renormalised weights add up to one."""
    low = torch.finfo(torch.float32).min
    l = torch.tensor([[low, low, low, low], [-200.0, -201.0, -202.0, low], [300.0, -300.0, 2.0, 1.0]], device="cuda")
    moe = z.Moe(4, 3, score=score)
    idx, w = moe.route(l)
    assert moe.read_status() == z.OK
    w = w.double().cpu().numpy()
    assert np.isfinite(w).all()
    np.testing.assert_allclose(w.sum(1), 1.0, rtol=1e-6)
    if score == "sigmoid":
        want = np.exp([0.0, -1.0, -2.0])
        np.testing.assert_allclose(w[1][np.argsort(idx[1].cpu().numpy())], want / want.sum(), rtol=200 * 2.0 ** -23)
    grad = moe.route_backward(l, idx, torch.ones(3, 3, device="cuda"))
    assert torch.isfinite(grad).all()


def test_route_masked_rows_and_bad_values(z):
    inf, nan = float("inf"), float("nan")
    l = torch.tensor([[-inf] * 4, [-inf, 1.0, -inf, -inf], [nan, 1.0, 2.0, 3.0], [1.0, 2.0, 3.0, 4.0]], device="cuda")
    moe = z.Moe(4, 2)
    idx, w = moe.route(l[[0, 1, 3]].contiguous())
    assert idx.cpu().tolist() == [[-1, -1], [1, -1], [3, 2]]
    assert w[0].tolist() == [0.0, 0.0] and w[1].tolist() == [1.0, 0.0]
    assert moe.read_status() == z.OK
    g = moe.route_backward(l[:2].contiguous(), idx[:2].contiguous(), torch.ones(2, 2, device="cuda"))
    assert torch.equal(g.cpu(), torch.zeros(2, 4))
    idx, w = moe.route(l)
    assert idx[2].tolist() == [-1, -1] and w[2].tolist() == [0.0, 0.0] and idx[3].tolist() == [3, 2]
    assert moe.read_status() == z.INVALID_ARG
    with pytest.raises(z.ZcclError):
        moe.check_status()
    moe.reset_status()
    # +inf: no softmax; a sigmoid of 1
    l = torch.tensor([[inf, 0.0, 1.0, 2.0]], device="cuda")
    assert moe.route(l)[0].tolist() == [[-1, -1]] and moe.read_status() == z.INVALID_ARG
    sig = z.Moe(4, 2, score="sigmoid", renormalize=False)
    idx, w = sig.route(l)
    assert idx.tolist() == [[0, 3]] and w[0, 0].item() == 1.0 and sig.read_status() == z.OK
    # a bias of -inf takes its expert away
    idx, _ = sig.route(torch.zeros(1, 4, device="cuda"), torch.tensor([0.0, -inf, 0.0, 0.0], device="cuda"))
    assert idx.tolist() == [[0, 2]]


def test_route_strided_rows_and_no_tokens(z):
    rng = np.random.default_rng(5)
    wide = torch.from_numpy(rng.normal(size=(19, 131)).astype(np.float32)).cuda()
    view = wide[:, 3:67]
    moe = z.Moe(64, 6)
    a, b = moe.route(view), moe.route(view.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    gw = torch.ones(19, 6, device="cuda")
    assert torch.equal(moe.route_backward(view, a[0], gw), moe.route_backward(view.contiguous(), a[0], gw))
    one = wide[:1, 3:67].expand(5, 64)  # the same row for every token
    assert torch.equal(moe.route(one)[0], a[0][:1].expand(5, 6))
    idx, w = moe.route(wide[:0, :64])
    assert idx.shape == (0, 6) and w.shape == (0, 6)


# ---- dispatch -----------------------------------------------------------------
DISPATCHES = [  # tokens, experts, top_k, hidden, share of slots without an expert
    (0, 4, 2, 64, 0.0), (1, 64, 8, 2048, 0.0), (1, 3, 1, 8, 1.0), (33, 64, 8, 264, 0.1), (7, 512, 32, 8, 0.2),
    (1000, 5, 2, 72, 0.0), (1025, 512, 2, 16, 0.3), (3001, 64, 8, 40, 0.05), (20011, 1, 1, 8, 0.5),
    (5003, 300, 31, 8, 0.01), (70001, 64, 3, 8, 0.1),
]


def random_idx(rng, t, e, k, none):
    """Skewed experts; a token may name one twice: the dispatch does not care."""
    idx = np.minimum((rng.random((t, k)) ** 3 * e).astype(np.int32), e - 1)
    idx[rng.random((t, k)) < none] = -1
    return idx


@pytest.mark.parametrize("t,e,k,h,none", DISPATCHES)
def test_dispatch(z, t, e, k, h, none):
    rng = np.random.default_rng(t + e + k)
    idx = random_idx(rng, t, e, k, none)
    if t > 3:
        idx[2, 0] = e + 5  # out of range: sends nothing
    x = torch.from_numpy(rng.integers(-32768, 32768, (t, h + 24)).astype(np.int16)).cuda().view(torch.bfloat16)[:, 8:8 + h]
    moe = z.Moe(e, k) if k <= e else z.Moe(k, k)
    moe.experts = e
    pos, counts, offsets, order = ref.places(idx, e)
    for _ in range(2):  # the second call on the same workspace
        d = moe.dispatch(x, torch.from_numpy(idx).cuda())
        assert np.array_equal(d.pos.cpu().numpy(), pos)
        assert np.array_equal(d.counts.cpu().numpy(), counts)
        assert np.array_equal(d.offsets.cpu().numpy(), offsets)
        want = x.cpu().view(torch.int16).numpy()[order // k] if t else np.zeros((0, h), np.int16)
        want[offsets[-1]:] = 0
        assert np.array_equal(d.rows.cpu().view(torch.int16).numpy(), want)


@pytest.mark.parametrize("t,capacity", [(50, 3), (4000, 97), (4000, 0), (300, 10 ** 6)])
def test_dispatch_table_through_batched_compression(z, t, capacity):
    """The device-made segment table codes each expert's static and dynamic rows as the oracle does."""
    e, k, h = 16, 2, 64
    rng = np.random.default_rng(t + capacity)
    idx = random_idx(rng, t, e, k, 0.1)
    x = torch.from_numpy(rng.normal(size=(t, h)).astype(np.float32)).bfloat16().cuda()
    moe, codec = z.Moe(e, k), z.Codec("cuda:0")
    d = moe.dispatch(x, torch.from_numpy(idx).cuda(), capacity=capacity)
    lut = z.zccl_lut_from_sigma(1.0)
    sizes = torch.zeros(2 * e, dtype=torch.int64, device="cuda")
    ws, wsb = codec.workspace(z.zccl_workspace_bytes(z.OP_COMPRESS_BATCHED, t * k * h, 2 * e))
    z.check(z.zccl_compress_batched(d.table.data_ptr(), 2 * e, t * k * h, lut, sizes.data_ptr(), ws, wsb,
                                    codec.status.data_ptr(), torch.cuda.current_stream().cuda_stream), "batched")
    torch.cuda.synchronize()
    codec.check_status()
    from lossless_bf16_exponent_split_gb300.codec import SEGMENT_DTYPE
    table = d.table.cpu().numpy().view(SEGMENT_DTYPE)
    rows, counts, offsets = d.rows.cpu().view(torch.int16).numpy().view(np.uint16), d.counts.cpu().numpy(), d.offsets.cpu().numpy()
    base, end = d.streams.data_ptr(), d.streams.data_ptr() + d.streams.numel()
    last = base
    for i in range(2 * e):
        fixed = min(int(counts[i // 2]), capacity)
        lo = offsets[i // 2] + (fixed if i & 1 else 0)
        n = int(counts[i // 2]) - fixed if i & 1 else fixed
        assert table["in"][i] == d.rows.data_ptr() + int(lo) * h * 2 and table["n"][i] == n * h
        assert table["out"][i] >= last and table["out"][i] % 16 == 0
        last = int(table["out"][i]) + int(table["cap"][i])
        at = int(table["out"][i]) - base
        got = d.streams[at: at + int(sizes[i].item())].cpu().numpy().tobytes()
        assert got == oracle.compress(rows[lo: lo + n].reshape(-1), lut)
    assert last <= end


# ---- combine ------------------------------------------------------------------
@pytest.mark.parametrize("t,e,k,h,none", [c for c in DISPATCHES if c[0] < 20000] + [(3, 4, 9, 5000, 0.2), (64, 8, 2, 0, 0.0)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_and_gradient(z, t, e, k, h, none, weighted):
    rng = np.random.default_rng(t * 7 + h)
    idx = random_idx(rng, t, e, k, none)
    pos, _, offsets, _ = ref.places(idx, e)
    y = torch.from_numpy(rng.normal(size=(t * k, h)).astype(np.float32)).bfloat16()
    w = rng.normal(size=(t, k)).astype(np.float32)
    grad = torch.from_numpy(rng.normal(size=(t, h)).astype(np.float32)).bfloat16()
    moe = z.Moe(max(e, k), k)
    moe.experts = e
    posd, wd = torch.from_numpy(pos.astype(np.int32)).cuda(), torch.from_numpy(w).cuda()
    out = moe.combine(y.cuda(), posd, wd if weighted else None).float().cpu().numpy()
    y64, there = y.double().numpy(), pos >= 0
    ww = np.where(there, w.astype(np.float64) if weighted else 1.0, 0.0)
    terms = y64[np.maximum(pos, 0)] * ww[:, :, None] if t else np.zeros((0, k, h))
    # K additions in 32 bits and one rounding to BF16
    tol = np.abs(terms).sum(1) * (k + 1) * 2.0 ** -24
    want = terms.sum(1)
    assert (np.abs(out - want) <= tol + np.abs(want) * 2.0 ** -8).all()
    if not weighted:
        return
    offd = torch.from_numpy(offsets.astype(np.int32)).cuda()
    gy, gw = moe.combine_backward(grad.cuda(), y.cuda(), posd, wd, offd)
    g64 = grad.double().numpy()
    want_gy = np.zeros((t * k, h))
    want_gy[pos[there]] = (ww[:, :, None] * g64[:, None, :])[there]
    assert (np.abs(gy.double().cpu().numpy() - want_gy) <= np.abs(want_gy) * 2.0 ** -8).all()
    assert np.array_equal(gy.float().cpu().numpy()[offsets[-1]:], np.zeros((t * k - offsets[-1], h)))
    prod = np.where(there[:, :, None], y64[np.maximum(pos, 0)] * g64[:, None, :], 0.0) if t else np.zeros((0, k, h))
    bound = np.abs(prod).sum(2) * (h / 32 + 8) * 2.0 ** -24
    assert (np.abs(gw.double().cpu().numpy() - prod.sum(2)) <= bound + 1e-30).all()


def test_combine_is_the_inverse_of_dispatch(z):
    """With one expert per token, combining what was dispatched gives the tokens back; a token without one gets zeros."""
    x = torch.randn(777, 128, device="cuda").bfloat16()
    idx = torch.randint(0, 6, (777, 1), dtype=torch.int32, device="cuda")
    idx[5] = -1
    moe = z.Moe(6, 1)
    d = moe.dispatch(x, idx)
    x[5] = 0
    assert torch.equal(moe.combine(d.rows, d.pos), x)


def test_combine_ignores_places_out_of_range(z):
    y = torch.ones(4, 8, device="cuda").bfloat16()
    pos = torch.tensor([[0, 4], [2147483647, 3], [-7, -1]], dtype=torch.int32, device="cuda")
    moe = z.Moe(4, 2)
    assert moe.combine(y, pos).float().cpu()[:, 0].tolist() == [1.0, 1.0, 0.0]
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    off[4] = 4
    gy, gw = moe.combine_backward(torch.ones(3, 8, device="cuda").bfloat16(), y, pos, torch.ones(3, 2, device="cuda"), off)
    assert gw.cpu().tolist() == [[8.0, 0.0], [0.0, 8.0], [0.0, 0.0]]


def test_calls_on_other_streams(z):
    """One Moe used on two streams at once: each has a workspace of its own."""
    rng = np.random.default_rng(11)
    moe = z.Moe(64, 8)
    x = torch.randn(4000, 64, device="cuda").bfloat16()
    idxs = [torch.from_numpy(random_idx(rng, 4000, 64, 8, 0.1)).cuda() for _ in range(2)]
    want = [ref.places(i.cpu().numpy(), 64)[0] for i in idxs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, i in zip(streams, idxs):
            with torch.cuda.stream(s):
                got.append(moe.dispatch(x, i))
        torch.cuda.synchronize()
        for d, w in zip(got, want):
            assert np.array_equal(d.pos.cpu().numpy(), w)


def test_refusals(z):
    moe = z.Moe(8, 2)
    f = torch.zeros(3, 8, device="cuda")
    idx = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    x = torch.zeros(3, 16, device="cuda").bfloat16()
    for bad in (dict(experts=0, top_k=1), dict(experts=513, top_k=1), dict(experts=8, top_k=9), dict(experts=8, top_k=0),
                dict(experts=64, top_k=33), dict(experts=9, top_k=2, groups=2), dict(experts=8, top_k=5, groups=4, top_groups=2),
                dict(experts=8, top_k=2, groups=4, top_groups=5), dict(experts=8, top_k=2, scale=float("nan"))):
        with pytest.raises(z.ZcclError):
            z.Moe(bad.pop("experts"), bad.pop("top_k"), **bad)
    with pytest.raises(ValueError):
        z.Moe(8, 2, score="tanh")
    for call in (lambda: moe.route(f.cpu()), lambda: moe.route(f.double()), lambda: moe.route(f[:, :7]), lambda: moe.route(f.T),
                 lambda: moe.route(f, torch.zeros(7, device="cuda")), lambda: moe.route_backward(f, idx.long(), f[:, :2].contiguous()),
                 lambda: moe.route_backward(f, idx[:2], f[:, :2].contiguous()), lambda: moe.dispatch(x.float(), idx),
                 lambda: moe.dispatch(x, idx[:, :1]), lambda: moe.combine(x.float(), idx), lambda: moe.combine(x.T, idx),
                 lambda: moe.combine(x, idx, f[:, :1]), lambda: moe.dispatch(x, idx, capacity=-1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(z.ZcclError):
        moe.dispatch(x[:, :12], idx)  # not a multiple of 8
    with pytest.raises(z.ZcclError):
        moe.dispatch(torch.zeros(3, 20, device="cuda").bfloat16()[:, 1:17], idx)  # misaligned rows
