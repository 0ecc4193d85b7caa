"""GPU: the balance over tables of sequences that do not cover all tokens, or run backwards."""
import pytest
import torch

import norm_ref as ref
from gpu_util import load_lib, require_gpu
from test_gpu_balance import LOSS, close, inputs

pytestmark = pytest.mark.gpu
F = torch.float32


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


def gradient(z, moe, l, idx, got, seq, fill):
    """balance_backward into a buffer that holds `fill`."""
    out = torch.full_like(l, fill)
    st = z.zccl_balance_backward(moe.config, l.data_ptr(), z.F32, l.shape[1], idx.data_ptr(), l.shape[0], seq.data_ptr(),
                                 seq.shape[0] - 1, got.counts.data_ptr(), got.tokens.data_ptr(), 1.0, None, out.data_ptr(),
                                 l.shape[1], 0, torch.cuda.current_stream().cuda_stream)
    assert st == z.OK
    return out


# the first sequence's first token, sequences, the tokens of each, tokens behind them
@pytest.mark.parametrize("first,sequences,each,behind", [
    (7, 1, 93, 0), (64, 3, 100, 30), (1, 304, 5, 1), (1000, 2, 0, 0), (5, 305, 3, 0), (2000, 400, 2, 0), (300, 400, 2, 5000),
    (70000, 305, 1, 1), (1, 305, 0, 0), (2, 310, 0, 3)])
def test_tokens_before_the_first_and_behind_the_last(z, first, sequences, each, behind):
    """They do not count, and every row of the gradient is written."""
    tokens = first + sequences * each + behind
    l, idx = inputs(tokens, 12, 3, F)
    bounds = [first + s * each for s in range(sequences + 1)]
    moe, seq = z.Moe(12, 3), torch.tensor(bounds, dtype=torch.int32, device="cuda")
    loss, counts, live, grad, mag = ref.balance(l, idx, bounds, "softmax")
    got = moe.balance(l, idx, seq)
    assert torch.equal(got.counts.cpu(), counts) and torch.equal(got.tokens.cpu(), live)
    assert abs(float(got.loss) - loss) <= LOSS * abs(loss)
    have = gradient(z, moe, l, idx, got, seq, 7.0)
    close(have, grad, mag)
    assert bool((have[:first] == 0).all()) and bool((have[tokens - behind:] == 0).all())
    base = torch.randn_like(l)
    out = moe.balance_backward(l, idx, got, seq, out=base.clone())
    close(out, base.double().cpu() + grad, base.double().cpu().abs() + mag)
    assert torch.equal(out[:first], base[:first]) and torch.equal(out[tokens - behind:], base[tokens - behind:])


@pytest.mark.parametrize("table,runs", [([0, 5000], [0, 100]), ([-9, 40, 20, 60], [0, 40, 40, 60]), ([30, 10, 80, 50, 90], [30, 30, 80, 80, 90]),
                                        ([90, 10, 120], [90, 90, 100]), ([0, 7, 3, 900] + [50] * 40, [0, 7, 7] + [100] * 41)])
def test_few_sequences_out_of_order_are_runs(z, table, runs):
    """Each begins where the last one ended: no token counts twice."""
    l, idx = inputs(100, 16, 2, F, masked=0.0)
    moe, seq = z.Moe(16, 2), torch.tensor(table, dtype=torch.int32, device="cuda")
    loss, counts, live, grad, mag = ref.balance(l, idx, runs, "softmax")
    got = moe.balance(l, idx, seq)
    assert torch.equal(got.counts.cpu(), counts) and torch.equal(got.tokens.cpu(), live)
    assert abs(float(got.loss) - loss) <= LOSS * abs(loss)
    close(gradient(z, moe, l, idx, got, seq, 7.0), grad, mag)


@pytest.mark.parametrize("at,value", [(1, -7), (200, 0), (400, 5), (399, 6000), (3, 4000)])
def test_many_sequences_out_of_order_have_no_loss(z, at, value):
    """Entries are cut to 0..tokens first, and where they are in order then nothing else changes.  Else some of more than
    304 sequences would share tokens: NaN, no gradient, and what it would be added to stays."""
    tokens, n = 4000, 400
    l, idx = inputs(tokens, 12, 3, F)
    table = [10 * i for i in range(n + 1)]
    table[at] = value
    moe, seq = z.Moe(12, 3), torch.tensor(table, dtype=torch.int32, device="cuda")
    cut = [min(max(v, 0), tokens) for v in table]
    if cut == sorted(cut):
        loss, counts, live, grad, mag = ref.balance(l, idx, cut, "softmax")
        got = moe.balance(l, idx, seq)
        assert torch.equal(got.counts.cpu(), counts) and abs(float(got.loss) - loss) <= LOSS * loss
        return close(gradient(z, moe, l, idx, got, seq, 7.0), grad, mag)
    l[50, 3] = float("nan")
    got = moe.balance(l, idx, seq)
    assert bool(got.loss.isnan()) and int(got.tokens[-1]) == 0
    assert [i for i, m in enumerate(got.tokens[:-1].tolist()) if m < 0] == [i for i in range(n) if cut[i + 1] < cut[i]]
    assert bool((gradient(z, moe, l, idx, got, seq, 7.0) == 0).all())
    base = torch.randn_like(l)
    assert torch.equal(moe.balance_backward(l, idx, got, seq, out=base.clone()), base)
    # the same handle's next call has its loss again
    l[50, 3] = 0.0
    bounds = [10 * i for i in range(n + 1)]
    loss, counts, live, grad, mag = ref.balance(l, idx, bounds, "softmax")
    seq = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    got = moe.balance(l, idx, seq)
    assert torch.equal(got.counts.cpu(), counts) and abs(float(got.loss) - loss) <= LOSS * loss
    close(gradient(z, moe, l, idx, got, seq, 7.0), grad, mag)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bounds", [[0, 500], [10, 200, 460], [10] + list(range(11, 471))])
def test_what_does_not_count_has_no_gradient_of_any_loss(z, bounds, score):
    """Also where the loss's own gradient has overflowed."""
    l, idx = inputs(500, 12, 3, F, masked=0.3)
    moe, seq = z.Moe(12, 3, score=score), torch.tensor(bounds, dtype=torch.int32, device="cuda")
    got = moe.balance(l, idx, seq)
    counts = (idx >= 0).any(1)
    counts[:bounds[0]] = counts[bounds[-1]:] = False
    assert 0 < int(counts.sum()) < 400
    for value in (float("inf"), float("nan")):
        grad = moe.balance_backward(l, idx, got, seq, grad_loss=torch.full((1,), value, device="cuda"))
        assert bool((grad[~counts] == 0).all()) and not bool(grad[counts].isfinite().all(1).any())
        base = torch.randn_like(l)
        out = moe.balance_backward(l, idx, got, seq, grad_loss=torch.full((1,), value, device="cuda"), out=base.clone())
        assert torch.equal(out[~counts], base[~counts])
