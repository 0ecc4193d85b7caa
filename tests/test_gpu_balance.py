"""GPU: the balance loss, each expert's slots and the logits' gradient against plain
64-bit forms, a sequence at a time.

Counts are exact.  A share q is off by at most 64 2^-24 of itself (the difference
l - max of logits below 40 in size, an exponential, a sum of at most 512, a
quotient); the loss adds positive terms, at most 128 of a warp one after the other,
8 warps, 304 parts or 256 sequences' share and 512 experts' by halves: under 1024
roundings in all.  A gradient is q (f - sum f q), each with its sums: under 512
roundings of the magnitude q (f + sum f q), and 2^-8 of itself in 16 bits."""
import pytest
import torch

import norm_ref as ref
from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu
LOSS, GRAD = 1024 * 2.0 ** -24, 512 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


def close(got, want, magnitude):
    tol = GRAD * magnitude + HALF[got.dtype] * (want.abs() + GRAD * magnitude) + 1e-37
    off = (got.double().cpu() - want).abs() - tol
    assert bool((off <= 0).all()), (float(off.max()), int((off > 0).sum()))


def inputs(tokens, experts, top_k, dtype, masked=0.05, seed=0):
    g = torch.Generator().manual_seed(tokens * 1009 + experts + seed)
    l = torch.randn(tokens, experts, generator=g) * 3
    l[torch.rand(tokens, experts, generator=g) < masked] = -float("inf")
    idx = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :top_k]
    idx[l.gather(1, idx) == -float("inf")] = -1
    pad = torch.rand(tokens, generator=g) < masked
    idx[pad] = -1
    l[pad & (torch.rand(tokens, generator=g) < 0.5)] = -float("inf")
    return l.to(dtype).cuda(), idx.to(torch.int32).cuda()


CASES = [  # tokens, experts, top_k, score, dtype, bounds (None: one sequence without a table)
    (1, 64, 8, "softmax", F, None),
    (1, 1, 1, "sigmoid", B, None),
    (7, 5, 2, "softmax", B, [0, 7]),
    (64, 64, 8, "softmax", F, [0, 10, 10, 40, 64]),          # one without tokens
    (513, 60, 4, "sigmoid", F, [0, 1, 500]),                 # tokens behind the last one
    (1000, 256, 8, "sigmoid", F, None),
    (2049, 512, 32, "softmax", B, [0, 700, 2049]),
    (4097, 33, 3, "sigmoid", B, [0, 4000, 4001, 4097]),
    (20000, 64, 8, "softmax", B, None),
    (20001, 128, 2, "softmax", F, None),
    (3000, 16, 2, "softmax", F, list(range(0, 3001, 6))),    # 500 short ones
    (900, 8, 1, "sigmoid", F, [0, 0, 0, 900, 900]),
    (50, 130, 4, "softmax", B, [0, 0]),                      # all behind the last one
    (9000, 24, 6, "softmax", B, [0, 3000, 6000, 9000]),
]


@pytest.mark.parametrize("tokens,experts,top_k,score,dtype,bounds", CASES)
def test_loss_counts_and_gradient(z, tokens, experts, top_k, score, dtype, bounds):
    l, idx = inputs(tokens, experts, top_k, dtype)
    moe = z.Moe(experts, top_k, score=score)
    seq = None if bounds is None else torch.tensor(bounds, dtype=torch.int32, device="cuda")
    loss, counts, live, grad, mag = ref.balance(l, idx, bounds or [0, tokens], score, 0.25)
    got = moe.balance(l, idx, seq, coefficient=0.25)
    assert torch.equal(got.counts.cpu(), counts) and torch.equal(got.tokens.cpu(), live)
    assert abs(float(got.loss) - loss) <= LOSS * abs(loss)
    again = moe.balance(l, idx, seq, coefficient=0.25)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    have = moe.balance_backward(l, idx, got, seq, coefficient=0.25)
    close(have, grad, mag)
    scale = torch.tensor(-3.0, device="cuda")
    close(moe.balance_backward(l, idx, got, seq, coefficient=0.25, grad_loss=scale), -3 * grad, 3 * mag)
    # added to a gradient that is there, in rows of a wider matrix; what surrounds it stays
    wide = torch.randn(tokens, experts + 3, device="cuda").to(dtype)
    before, out = wide.clone(), wide[:, 1:1 + experts]
    moe.balance_backward(l, idx, got, seq, coefficient=0.25, out=out)
    base = before[:, 1:1 + experts].double().cpu()
    close(out, base + grad, base.abs() + mag)
    assert torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, 1 + experts:], before[:, 1 + experts:])
    # strided logits
    rows = torch.full((tokens, experts + 5), float("nan"), dtype=dtype, device="cuda")[:, 2:2 + experts]
    rows.copy_(l)
    other = moe.balance(rows, idx, seq, coefficient=0.25)
    assert torch.equal(other.counts, got.counts) and abs(float(other.loss) - loss) <= LOSS * abs(loss)
    close(moe.balance_backward(rows, idx, got, seq, coefficient=0.25), grad, mag)


def test_against_the_router(z):
    """The router's own choice; an even choice gives the coefficient."""
    g = torch.Generator(device="cuda").manual_seed(1)
    l = torch.randn(5000, 64, generator=g, device="cuda")
    moe = z.Moe(64, 8, score="sigmoid", groups=8, top_groups=4)
    idx, _ = moe.route(l)
    b = moe.balance(l, idx)
    d = moe.dispatch(torch.zeros(5000, 8, dtype=B, device="cuda"), idx)
    assert torch.equal(b.counts[0], d.counts) and int(b.tokens[0]) == 5000
    even = (torch.arange(64 * 8, device="cuda", dtype=torch.int32) % 64).view(64, 8)
    assert abs(float(moe.balance(l[:64], even, coefficient=0.01).loss) - 0.01) < 0.01 * LOSS


def test_odd_indices_and_rows(z):
    """Entries outside 0..E-1 choose nothing, an expert named twice counts twice, a row without a usable score adds
    no shares, far logits keep their shares, and what does not count may hold NaN."""
    moe, soft = z.Moe(4, 2, score="sigmoid"), z.Moe(4, 2)
    nan, inf = float("nan"), float("inf")
    l = torch.tensor([[1.0, 2, 3, 4], [nan, nan, 1, 1], [-inf] * 4, [-200, -201, -250, -300], [200, 100, -300, 0]], device="cuda")
    idx = torch.tensor([[2, 2], [-1, 4], [0, 1], [1, -7], [3, 0]], dtype=torch.int32, device="cuda")
    for m, score in ((moe, "sigmoid"), (soft, "softmax")):
        got = m.balance(l, idx)
        safe = l.clone()
        safe[1] = 0.0
        if score == "sigmoid":  # in 64 bits these scores underflow neither
            safe[2] = -inf
        loss, counts, tokens, grad, mag = ref.balance(safe, idx, [0, 5], score)
        assert got.counts.tolist() == [[2, 2, 2, 1]] == counts.tolist() and got.tokens.tolist() == [4, 1]
        assert abs(float(got.loss) - loss) <= LOSS * loss
        have = m.balance_backward(l, idx, got)
        close(have, grad, mag)
        assert bool((have[1] == 0).all()) and bool((have[2] == 0).all())


def test_tables_out_of_range_stay_in_bounds(z):
    """A table that runs backwards or past the tokens is cut to what there is."""
    l, idx = inputs(100, 16, 2, F, masked=0.0)
    moe = z.Moe(16, 2)
    for table, bounds in (([0, 5000], [0, 100]), ([-9, 40, 20, 60], [0, 40, 40, 60]), ([0, -5], [0, 0]),
                          ([0, 7, 3, 900] + [50] * 40, [0, 7])):
        seq = torch.tensor(table, dtype=torch.int32, device="cuda")
        got = moe.balance(l, idx, seq)
        assert int(got.counts.sum()) <= 2 * 200 and bool(got.loss.isfinite())
        assert bool(moe.balance_backward(l, idx, got, seq).isfinite().all())
        assert torch.equal(got.counts[0].cpu(), ref.balance(l, idx, bounds, "softmax")[1][0])


@pytest.mark.parametrize("sequences", [31, 33, 303, 304, 305])
@pytest.mark.parametrize("experts", [12, 256])
def test_sequences_around_the_most_that_are_cut(z, sequences, experts):
    """Up to 304 sequences are cut into parts, each is one beyond.  Some have no tokens."""
    g = torch.Generator().manual_seed(sequences)
    tokens = 5000
    bounds = sorted(torch.randint(0, tokens - 50, (sequences + 1,), generator=g).tolist())
    bounds[0], bounds[5] = 0, bounds[4]
    l, idx = inputs(tokens, experts, 4, F)
    moe, seq = z.Moe(experts, 4, score="sigmoid"), torch.tensor(bounds, dtype=torch.int32, device="cuda")
    loss, counts, live, grad, mag = ref.balance(l, idx, bounds, "sigmoid")
    got = moe.balance(l, idx, seq)
    assert torch.equal(got.counts.cpu(), counts) and torch.equal(got.tokens.cpu(), live)
    assert abs(float(got.loss) - loss) <= LOSS * abs(loss)
    close(moe.balance_backward(l, idx, got, seq), grad, mag)


def test_sigmoid_of_all_sizes(z):
    """Scores below 2^-126 may read as none: of a sum of 2^-80 or more (smaller sums take a common factor) that is a
    share below 2^-46."""
    g = torch.Generator().manual_seed(3)
    level = torch.linspace(-140, 140, 2000)[:, None]
    l = (level + torch.randn(2000, 16, generator=g) * torch.linspace(0, 40, 16)).cuda()
    idx = torch.topk(l, 2).indices.to(torch.int32)
    moe = z.Moe(16, 2, score="sigmoid")
    loss, counts, live, grad, mag = ref.balance(l, idx, [0, 2000], "sigmoid")
    got = moe.balance(l, idx)
    assert torch.equal(got.counts.cpu(), counts) and abs(float(got.loss) - loss) <= LOSS * loss
    f = counts.double() * 16 / (2.0 * 2000 * 2000)  # what a share weighs
    off = (moe.balance_backward(l, idx, got).double().cpu() - grad).abs()
    assert bool((off <= (GRAD + 2.0 ** -24) * mag + 2.0 ** -46 * f.max()).all())


def test_one_workspace_for_calls_of_all_sizes(z):
    moe = z.Moe(64, 8)
    l, idx = inputs(6000, 64, 8, F)
    for bounds in ([0, 6000], list(range(0, 6001, 3)), [0, 17, 6000], [0, 6000], [0, 5]):
        seq = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        loss, counts, tokens, _, _ = ref.balance(l, idx, bounds, "softmax")
        got = moe.balance(l, idx, seq)
        assert torch.equal(got.counts.cpu(), counts) and torch.equal(got.tokens.cpu(), tokens)
        assert abs(float(got.loss) - loss) <= LOSS * loss


def test_more_than_2_to_31_logits(z):
    """Addresses beyond 32 bits: equal logits give equal shares, and the last tokens the gradient that they give by themselves."""
    tokens, experts = (1 << 22) + 5, 512
    l = torch.zeros(tokens, experts, dtype=B, device="cuda")
    idx = (torch.arange(tokens, device="cuda") % experts).to(torch.int32)[:, None].contiguous()
    l[-1, :7] = 1.0
    moe = z.Moe(experts, 1)
    seq = torch.tensor([0, tokens - 3, tokens], dtype=torch.int32, device="cuda")
    got = moe.balance(l, idx, seq)
    loss, counts, live, grad, mag = ref.balance(l[-3:], idx[-3:], [0, 3], "softmax", 0.5)
    assert torch.equal(got.counts[1:].cpu(), counts) and got.tokens.tolist() == [tokens - 3, 3, 2]
    assert int(got.counts[0].max() - got.counts[0].min()) <= 1
    assert abs(float(got.loss) - (0.5 + loss)) < LOSS
    have = moe.balance_backward(l, idx, got, seq)
    close(have[-3:], grad, mag)
    assert float(have[:-3].abs().max()) < 1e-9  # shares of 1 / 512, slots that differ by one of 8192


def test_empty(z):
    moe = z.Moe(8, 2)
    l, idx = torch.zeros(0, 8, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    b = moe.balance(l, idx)
    assert float(b.loss) == 0 and b.counts.tolist() == [[0] * 8] and b.tokens.tolist() == [0, 0]
    assert moe.balance_backward(l, idx, b).shape == (0, 8)
    none = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    b = moe.balance(torch.zeros(5, 8, device="cuda"), none)
    assert float(b.loss) == 0 and b.tokens.tolist() == [0, 0]
    assert bool((moe.balance_backward(torch.zeros(5, 8, device="cuda"), none, b) == 0).all())


def test_in_two_graphs_and_threads(z):
    from test_gpu_moe_threads import check
    moe = z.Moe(64, 8)
    l, idx = inputs(9000, 64, 8, B)

    def work(i):
        b = moe.balance(l[i:], idx[i:])
        return [*b, moe.balance_backward(l[i:], idx[i:], b)]

    for own_stream in (False, True):
        check(work, own_stream)
    want = [t.clone() for t in work(0)]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = work(0)
        graphs.append((g, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (g, _), s in zip(graphs, streams):  # at the same time: each has a workspace of its own
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
