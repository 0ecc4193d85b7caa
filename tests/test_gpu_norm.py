"""GPU: the join of a block's output with the residual, the norms around it and
their gradients, against plain 64-bit forms.

An fp32 result is a sum of terms, each a product of a few factors; with N
roundings on the longest way from an input to it, it is off by at most N 2^-24 of
the sum of the terms' magnitudes.  The ways here: a row's sum (at most 8 values a
lane and a tile one after the other, over at most 16 tiles a warp, then 5 + 5
halvings: 138), twice for y's gradient, the rows of a worker (at most 64 in these
cases) and the workers (608 / 32 + 32 = 51), and about 20 products, roots and
differences: under 512.  A result of 16 bits is rounded once more, by at most 2^-8
of itself."""
import pytest
import torch

import norm_ref as ref
from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu
N = 512 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


def close(got, want, magnitude, what):
    tol = N * magnitude + HALF[got.dtype] * (want.abs() + N * magnitude) + 1e-37
    off = (got.double().cpu() - want).abs() - tol
    assert bool((off <= 0).all()), (what, float(off.max()), int((off > 0).sum()))


CASES = [  # rows, hidden, residual, block, weight (None: no weights), post, gates (0: none), scale, dropout
    (1, 4096, B, B, B, False, 0, 1.0, 0.0),
    (1, 1, F, F, F, True, 1, 1.0, 0.0),
    (2, 7, B, F, None, True, 2, 0.5, 0.0),
    (3, 8, F, B, B, True, 3, 1.0, 0.5),
    (33, 2048, B, B, F, True, 0, 1.0, 0.0),
    (70, 100, B, B, F, False, 7, 2.0, 0.1),
    (257, 256, F, B, F, True, 1, 1.0, 0.2),
    (130, 264, B, B, B, True, 5, 1.0, 0.0),
    (64, 255, F, F, F, True, 64, 1.0, 0.3),
    (61, 1001, F, B, F, True, 61, 1.0, 0.0),
    (40, 1032, B, B, None, False, 1, 1.0, 0.4),
    (26, 4104, B, B, B, True, 2, 1.0, 0.0),
    (13, 5000, B, F, F, True, 13, 1.0, 0.1),
    (12, 8192, B, B, F, True, 1, 1.0, 0.1),
    (10, 8200, B, B, B, False, 5, 1.0, 0.0),
    (9, 14336, B, B, B, True, 3, 0.25, 0.0),
    (7, 16384, B, B, F, True, 7, 1.0, 0.1),       # clusters of four
    (300, 12000, F, F, F, True, 3, 1.0, 0.1),
    (400, 9600, B, B, B, False, 4, 1.0, 0.2),     # clusters of two, several rows each
    (6, 16385, F, B, F, True, 2, 1.0, 0.1),
    (5, 65536, B, B, F, True, 1, 1.0, 0.0),
    (2500, 64, B, B, F, True, 50, 1.0, 0.0),      # more rows than workers, gate rows shared by some
    (3001, 40, F, F, F, True, 1, 1.0, 0.1),
    (1830, 24, F, B, F, False, 610, 1.0, 0.0),    # a gate row for three tokens
    (2600, 512, B, B, F, True, 100, 1.0, 0.0),
    (700, 2048, B, B, F, True, 1, 1.0, 0.1),
    (1300, 1280, F, B, F, True, 13, 1.0, 0.1),    # 20 warps an SM
    (650, 2560, F, B, B, True, 65, 1.0, 0.0),
    (640, 1536, B, F, F, False, 1, 1.0, 0.1),
    (310, 2305, B, B, F, True, 2, 1.0, 0.0),
    (400, 4095, B, B, B, True, 40, 1.0, 0.1),     # rows anywhere, two tiles a warp
    (340, 1803, B, B, F, False, 1, 0.5, 0.1),
    (1300, 1001, B, B, F, True, 13, 1.0, 0.1),
    (130, 10001, B, B, F, True, 13, 1.0, 0.0),    # in clusters of two
    (20, 16383, B, B, F, True, 1, 1.0, 0.1),
    (10000, 128, B, B, F, True, 50, 1.0, 0.1),    # two rows a warp
    (11001, 64, B, B, B, True, 57, 0.5, 0.0),     # four
    (777, 120, F, F, F, False, 777, 1.0, 0.1),
    (20011, 8, F, B, F, True, 1, 1.0, 0.1),
    (10100, 56, B, F, F, True, 5050, 1.0, 0.2),
    (5, 72, B, B, B, True, 5, 1.0, 0.0),
]


def inputs(z, rows, hidden, residual, block, weight, post, gates, scale, dropout, seed=0):
    g = torch.Generator(device="cuda").manual_seed(rows * 100003 + hidden + seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x = (randn(rows, hidden) * torch.exp(randn(rows, 1))).to(residual)
    y = (randn(rows, hidden) * torch.exp(randn(rows, 1))).to(block)
    w = p = gate = None
    if weight is not None:
        w, p = ((1 + 0.3 * randn(hidden)).to(weight) for _ in range(2))
    if gates:
        gate = (0.5 + 0.3 * randn(gates, hidden)).to(block)
    n = z.ResidualNorm(hidden, post=post, eps=1e-5, scale=scale, dropout=dropout, seed=0xFEDCBA9876543210)
    more = dict(post_weight=p if post else None, gate=gate)
    return n, x, y, w, more, randn(rows, hidden).to(residual), randn(rows, hidden).to(block)


@pytest.mark.parametrize("case", CASES)
def test_forward_and_gradients(z, case):
    rows, hidden, residual, block, weight, post, gates, scale, dropout = case
    n, x, y, w, more, grad_r, grad_h = inputs(z, *case)
    offset = (3 << 32) + 11
    r, h = n.add(x, y, w, offset=offset, **more)
    at = ref.Ref(x=x, y=y, weight=w, post=post, eps=1e-5, scale=scale, dropout=dropout, seed=0xFEDCBA9876543210, offset=offset, **more)
    close(r, *at.r(), "r")
    want = at.h(r)
    close(h, want, want.abs(), "h")
    if dropout:
        assert torch.equal(r.cpu()[~at.keep], x.cpu()[~at.keep])  # nothing joins there
    only, none = n.add(x, y, normed=False, offset=offset, **more)
    assert none is None and torch.equal(only, r)

    for gr, gh in ((grad_r, grad_h), (None, grad_h), (grad_r, None)):
        weights = (w if gh is not None else None)
        got = n.add_backward(gr, gh, None if gh is None else r, y, weights, offset=offset, **more)
        wanted = at.backward(gr, gh, r)
        for name, have in got._asdict().items():
            if name == "x" and gh is None:
                assert have is gr
            elif have is not None:
                close(have, *wanted[name], (name, gr is None, gh is None))
        assert (got.weight is None) == (weights is None) and (got.gate is None) == (gates == 0)
        assert got.x.dtype == residual and got.y.dtype == block
        again = n.add_backward(gr, gh, None if gh is None else r, y, weights, offset=offset, **more)
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))  # no order changes
    n.check_status()


@pytest.mark.parametrize("rows,hidden,residual,block,weight", [
    (1, 4096, B, B, B), (17, 1000, B, F, F), (5, 77, F, B, F), (300, 2048, B, B, None), (4, 20000, F, F, F), (1000, 128, B, B, F)])
def test_norm_alone(z, rows, hidden, residual, block, weight):
    n, x, _, w, _, _, grad = inputs(z, rows, hidden, residual, block, weight, False, 0, 1.0, 0.3)
    at = ref.Ref(x=x, weight=w, eps=1e-5)
    h = n.norm(x, w, dtype=block)
    want = at.h(x)
    close(h, want, want.abs(), "h")
    gx, gw = n.norm_backward(grad, x, w)
    wanted = at.backward(None, grad, x)
    close(gx, *wanted["x"], "x")
    assert (gw is None) == (w is None) and gx.dtype == residual
    if gw is not None:
        close(gw, *wanted["weight"], "weight")


@pytest.mark.parametrize("hidden", [256, 1001, 2048, 9000])
def test_strided_rows_give_the_same(z, hidden):
    """Rows of wider matrices, on and off 16 bytes, one row for all, and an r that takes x's place."""
    rows = 12
    n, x, y, w, more, grad_r, grad_h = inputs(z, rows, hidden, B, B, F, True, 3, 1.0, 0.2)
    r, h = n.add(x, y, w, offset=5, **more)
    grads = n.add_backward(grad_r, grad_h, r, y, w, offset=5, **more)
    for pad in (8, 3):
        def wide(t):
            out = torch.full((t.shape[0], hidden + 2 * pad), float("nan"), dtype=t.dtype, device="cuda")[:, pad:pad + hidden]
            out.copy_(t)
            return out
        other = dict(more, gate=wide(more["gate"]))
        r2, h2 = n.add(wide(x), wide(y), w, offset=5, **other)
        got = n.add_backward(wide(grad_r), wide(grad_h), wide(r), wide(y), w, offset=5, **other)
        at = ref.Ref(x=x, y=y, weight=w, post=True, eps=1e-5, dropout=0.2, seed=0xFEDCBA9876543210, offset=5, **more)
        close(r2, *at.r(), "r")
        wanted = at.backward(grad_r, grad_h, r)
        for name, have in got._asdict().items():
            close(have, *wanted[name], name)
        if pad == 8 and hidden % 8 == 0:
            assert torch.equal(r, r2) and torch.equal(h, h2) and all(torch.equal(a, b) for a, b in zip(grads, got))
    one = x[:1].expand(rows, hidden)
    r3, _ = n.add(one, y, w, offset=5, **more)
    close(r3, *ref.Ref(x=one, y=y, weight=w, post=True, eps=1e-5, dropout=0.2, seed=0xFEDCBA9876543210, offset=5, **more).r(), "r")
    place = x.clone()
    st = z.zccl_residual_norm(n.config, place.data_ptr(), z.BF16, hidden, y.data_ptr(), z.BF16, hidden, w.data_ptr(),
                              more["post_weight"].data_ptr(), z.F32, more["gate"].data_ptr(), z.BF16, hidden, 4, rows, 5,
                              None, place.data_ptr(), h.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
    assert st == z.OK and torch.equal(place, r)


@pytest.mark.parametrize("hidden,residual", [(200, F), (2048, B), (9000, B), (16384, F), (20000, B), (1003, F)])
def test_in_place_and_one_gate_for_all(z, hidden, residual):
    """The residual's place for the result, and a gate row that every token's row of a wider shape is."""
    n, x, y, w, more, grad_r, grad_h = inputs(z, 12, hidden, residual, B, F, True, 1, 1.0, 0.2)
    r, h = n.add(x, y, w, **more)
    place, again = x.clone(), torch.empty_like(h)
    st = z.zccl_residual_norm(n.config, place.data_ptr(), z.F32 if residual == F else z.BF16, hidden, y.data_ptr(), z.BF16,
                              hidden, w.data_ptr(), more["post_weight"].data_ptr(), z.F32, more["gate"].data_ptr(), z.BF16,
                              hidden, 12, 12, 0, None, place.data_ptr(), again.data_ptr(), None,
                              torch.cuda.current_stream().cuda_stream)
    assert st == z.OK and torch.equal(place, r) and torch.equal(again, h)
    each = dict(more, gate=more["gate"].expand(12, hidden))
    r2, h2 = n.add(x, y, w, **each)
    assert torch.equal(r2, r) and torch.equal(h2, h)
    one, all_of = (n.add_backward(grad_r, grad_h, r, y, w, **m) for m in (more, each))
    assert all_of.gate.shape == (12, hidden) and torch.equal(one.x, all_of.x) and torch.equal(one.y, all_of.y)
    at = ref.Ref(x=x, y=y, weight=w, post=True, eps=1e-5, dropout=0.2, seed=0xFEDCBA9876543210, **each)
    close(all_of.gate, *at.backward(grad_r, grad_h, r)["gate"], "gate")


def test_nothing_is_written_outside(z):
    """Guards around every output of the calls, at sizes that end inside a tile."""
    for rows, hidden in ((3, 9), (5, 264), (4, 1001), (3, 8200)):
        n, x, y, w, more, grad_r, grad_h = inputs(z, rows, hidden, B, F, F, True, rows, 1.0, 0.0)
        def guarded(count, dtype):
            return torch.full((count + 512,), 7.0, dtype=dtype, device="cuda")
        size = rows * hidden
        outs = [guarded(size, B), guarded(size, F)]
        stream = torch.cuda.current_stream().cuda_stream
        at = [o.data_ptr() + 256 * o.element_size() for o in outs]
        assert z.zccl_residual_norm(n.config, x.data_ptr(), z.BF16, hidden, y.data_ptr(), z.F32, hidden, w.data_ptr(),
                                    more["post_weight"].data_ptr(), z.F32, more["gate"].data_ptr(), z.F32, hidden, 1, rows, 0,
                                    None, *at, None, stream) == z.OK
        nbytes = z.zccl_residual_norm_workspace_bytes(hidden, rows)
        ws = torch.full((nbytes + 512,), 7, dtype=torch.uint8, device="cuda")
        backs = [guarded(size, B), guarded(size, F), guarded(hidden, F), guarded(hidden, F), guarded(size, F)]
        places = [o.data_ptr() + 256 * o.element_size() for o in backs]
        r = outs[0][256:256 + size].view(rows, hidden).clone()
        assert z.zccl_residual_norm_backward(
            n.config, grad_r.data_ptr(), hidden, grad_h.data_ptr(), hidden, r.data_ptr(), z.BF16, hidden, y.data_ptr(), z.F32,
            hidden, w.data_ptr(), more["post_weight"].data_ptr(), z.F32, more["gate"].data_ptr(), z.F32, hidden, 1, rows, 0, None,
            *places, ws.data_ptr() + 256, nbytes, None, stream) == z.OK
        for o in outs + backs:
            count = o.numel() - 512
            assert bool((o[:256] == 7).all()) and bool((o[256 + count:] == 7).all())
        assert bool((ws[:256] == 7).all()) and bool((ws[256 + nbytes:] == 7).all())


def test_rows_that_are_not_finite_stay_their_own(z):
    """Zeros give zeros; a NaN or an infinity of a row leaves the others as they are."""
    rows, hidden = 9, 520
    n, x, y, w, more, grad_r, grad_h = inputs(z, rows, hidden, F, F, F, True, rows, 1.0, 0.0)
    r0, h0 = n.add(x, y, w, **more)
    g0 = n.add_backward(grad_r, grad_h, r0, y, w, **more)
    x2, y2 = x.clone(), y.clone()
    y2[1] = 0.0
    y2[3, 100] = float("nan")
    y2[5, 7] = float("inf")
    x2[7] = 0.0
    y2[7] = 0.0
    r, h = n.add(x2, y2, w, **more)
    g = n.add_backward(grad_r, grad_h, r, y2, w, **more)
    assert torch.equal(r[1], x[1]) and bool((r[7] == 0).all()) and bool((h[7] == 0).all())
    assert bool(r[3].isnan().all()) and bool(r[5, 7].isnan())
    for a, b in ((r, r0), (h, h0), (g.x, g0.x), (g.y, g0.y), (g.gate, g0.gate)):
        for t in (0, 2, 4, 6, 8):
            assert torch.equal(a[t], b[t])
    assert bool(g.x[1].isfinite().all()) and bool(g.y[1].isfinite().all()) and bool(g.x[7].isfinite().all())
    # a dropped element adds nothing, whatever it holds
    m = z.ResidualNorm(hidden, dropout=0.5, seed=4)
    keep = ref.kept(rows, hidden, 0.5, 4, 0).cuda()
    bad = torch.where(keep, y, float("inf"))
    r, h = m.add(x, bad, w)
    assert torch.equal(r, m.add(x, y, w)[0]) and bool(r.isfinite().all()) and bool(h.isfinite().all())


@pytest.mark.parametrize("hidden", [520, 1001, 9000])
def test_all_dropped(z, hidden):
    n, x, y, w, more, grad_r, grad_h = inputs(z, 8, hidden, B, B, F, True, 2, 1.0, 1.0)
    r, h = n.add(x, y, w, **more)
    assert torch.equal(r, x) and torch.equal(h, n.norm(x, w))
    g = n.add_backward(grad_r, grad_h, r, y, w, **more)
    assert torch.equal(g.x, n.norm_backward(grad_h, x, w, residual=grad_r)[0])
    assert all(bool((t == 0).all()) for t in (g.y, g.post_weight, g.gate))


@pytest.mark.parametrize("hidden", [2048, 1001])
def test_more_than_2_to_31_values(z, hidden):
    """Addresses beyond 32 bits: the last rows against the same rows by themselves, and the weight's gradient of ones."""
    rows = (1 << 31) // hidden + 7
    n = z.ResidualNorm(hidden, dropout=0.5, seed=3)
    x = torch.ones(rows, hidden, dtype=B, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    tail = torch.randn(5, hidden, generator=g, device="cuda").to(B)
    x[-5:] = tail
    r, h = n.add(x, x, offset=4)
    at = ref.Ref(x=tail, y=tail)
    keep = torch.from_numpy(kept_rows(rows - 5, 5, hidden, 0.5, 3, 4))
    want = torch.where(keep, 3 * tail.double().cpu(), tail.double().cpu())  # x + x / (1 - p)
    close(r[-5:], want, want.abs(), "r")
    close(h[-5:], at.h(r[-5:]), at.h(r[-5:]).abs(), "h")
    one, half = n.norm(x[-5:]), torch.ones(hidden, device="cuda")
    gx, gw = n.norm_backward(x, x, half)
    want = n.norm_backward(tail, tail, half)[0]
    assert torch.equal(gx[-5:], want) and torch.equal(one, n.norm(x)[-5:])
    # a row of ones has the norm 1 / sqrt(1 + 1e-6) each time
    total = (rows - 5) / (1 + 1e-6) ** 0.5 + (tail.double() * ref.inverse_rms(tail.double(), 1e-6) * tail.double()).sum(0)
    # a worker adds its n rows, 14,200 at most, one after the other: n / 2 half steps of the sum, and the joined parts' few
    assert float((gw.double() / total - 1).abs().max()) < 8192 * 2.0 ** -24


def kept_rows(first, rows, cols, p, seed, offset):
    """The dropout's kept elements of some rows."""
    import numpy as np
    blocks = -(-cols // 8)
    b, r = np.meshgrid(np.arange(blocks, dtype=np.uint64), np.arange(first, first + rows, dtype=np.uint64))
    words = ref.philox((b, r, np.full_like(b, offset), np.zeros_like(b)), (seed, 0))
    halves = np.stack([np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1) for w in words], -2)
    return halves.reshape(rows, blocks * 8)[:, :cols] >= ref.dropped_of(p)


def test_large_and_small_values(z):
    """Squares up to 2^126 and down to where eps takes over."""
    n = z.ResidualNorm(1024, post=True, eps=1e-20)
    g = torch.Generator(device="cuda").manual_seed(3)
    for size in (2.0 ** 57, 2.0 ** -30, 2.0 ** -60):
        x = torch.randn(4, 1024, generator=g, device="cuda") * size
        y = torch.randn(4, 1024, generator=g, device="cuda") * size
        r, h = n.add(x, y)
        at = ref.Ref(x=x, y=y, post=True, eps=1e-20)
        close(r, *at.r(), "r")
        close(h, at.h(r), at.h(r).abs(), "h")


@pytest.mark.parametrize("rows,hidden,gates,dropout", [(300, 696, 1, 0.0), (40, 4104, 4, 0.3), (3, 20000, 3, 0.3), (129, 77, 1, 0.1)])
def test_join_has_the_bits_of_its_operations(z, rows, hidden, gates, dropout):
    """Without a norm after the block: each product and sum in 32 bits, rounded in the documented order."""
    n, x, y, _, more, _, _ = inputs(z, rows, hidden, B, F, None, False, gates, 0.3, dropout)
    r, _ = n.add(x, y, normed=False, offset=9, **more)
    k = more["gate"].repeat_interleave(rows // gates, 0) * torch.tensor(0.3, device="cuda")
    want = x.float() + (k * torch.tensor(ref.gain(dropout), device="cuda") if dropout else k) * y
    if dropout:
        want = torch.where(ref.kept(rows, hidden, dropout, 0xFEDCBA9876543210, 9).cuda(), want, x.float())
    assert torch.equal(r, want.bfloat16())


def test_offset_on_the_device_in_a_graph(z):
    """Captured once, replayed with an offset that the graph moves on, beside a second graph and eager calls."""
    n, x, y, w, more, grad_r, grad_h = inputs(z, 50, 2048, B, B, F, True, 2, 1.0, 0.3)
    offset = torch.full((1,), (1 << 33) + 5, dtype=torch.int64, device="cuda")

    def step():
        r, h = n.add(x, y, w, offset=offset, **more)
        return (r, h, *n.add_backward(grad_r, grad_h, r, y, w, offset=offset, **more))

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
            offset += 1
        graphs.append((g, out))
    masks = []
    for i, (g, out) in enumerate(graphs * 2):
        now = (1 << 33) + 5 + i
        assert int(offset) == now
        g.replay()
        r, h = n.add(x, y, w, offset=now, **more)
        want = (r, h, *n.add_backward(grad_r, grad_h, r, y, w, offset=now, **more))
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        masks.append(r)
    assert not any(torch.equal(masks[0], m) for m in masks[1:])


def test_other_streams_and_threads(z):
    from test_gpu_moe_threads import check
    n, *args = inputs(z, 300, 1024, B, B, F, True, 1, 1.0, 0.1)
    x, y, w, more, grad_r, grad_h = args

    def work(i):
        r, h = n.add(x[i:], y[i:], w, offset=i, **more)
        return [r, h, *n.add_backward(grad_r[i:], grad_h[i:], r, y[i:], w, offset=i, **more)]

    for own_stream in (False, True):
        check(work, own_stream)


def test_empty(z):
    n = z.ResidualNorm(64, post=True)
    x, w = torch.zeros(0, 64, device="cuda"), torch.ones(64, device="cuda")
    r, h = n.add(x, x, w, post_weight=w)
    assert r.shape == h.shape == (0, 64) and n.norm(x, w).shape == (0, 64)
    g = n.add_backward(x, x, x, x, w, post_weight=w, gate=torch.ones(1, 64, device="cuda"))
    assert g.x.shape == (0, 64) and all(bool((t == 0).all()) for t in (g.weight, g.post_weight, g.gate))


def test_nothing_is_recorded_for_autograd(z):
    n = z.ResidualNorm(64)
    x = torch.randn(3, 64, device="cuda", requires_grad=True)
    r, h = n.add(x, x)
    assert not r.requires_grad and not h.requires_grad and not z.Dropout(0.5).apply(x).requires_grad
