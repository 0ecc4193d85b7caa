"""CPU: argument errors of the norm, dropout and balance calls are returned before
any CUDA call, their classes check each argument, and a handle of a device that is
not the current one refuses."""
import pytest
import torch


@pytest.fixture(scope="module")
def z():
    from lossless_bf16_exponent_split_gb300 import build
    build.build()
    import lossless_bf16_exponent_split_gb300 as z
    z.lib()
    return z


A = 1 << 20  # a fake, aligned "device" address: never dereferenced
INF, NAN = float("inf"), float("nan")


def config(z, **kw):
    return z.Norm(**dict(dict(hidden=16, post=1, eps=1e-6, scale=1.0, dropout=0.0, seed=0), **kw))


BAD_CONFIGS = [dict(hidden=0), dict(hidden=65537), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF),
               dict(scale=INF), dict(scale=NAN), dict(dropout=-0.1), dict(dropout=1.1), dict(dropout=NAN)]


def test_norm_refusals(z):
    ok = dict(d_x=A, x_dtype=z.BF16, x_stride=16, d_y=A, dtype=z.BF16, y_stride=16, d_weight=A, d_post_weight=A,
              weight_dtype=z.F32, d_gate=A, gate_dtype=z.BF16, gate_stride=16, gate_span=1, rows=4, offset=0, d_offset=None,
              d_r=A, d_h=A, d_status=A, stream=None)

    def call(c=None, **kw):
        return z.zccl_residual_norm(c or config(z), **dict(ok, **kw))

    for kw in BAD_CONFIGS:
        assert call(config(z, **kw)) == z.INVALID_ARG, kw
    for kw in (dict(d_x=None), dict(d_x=A + 1), dict(x_dtype=2), dict(dtype=-1), dict(weight_dtype=2), dict(gate_dtype=7),
               dict(d_y=A + 1), dict(d_weight=A + 2), dict(d_post_weight=A + 1), dict(d_gate=A + 1), dict(gate_span=0),
               dict(rows=1 << 31), dict(x_stride=1 << 40), dict(y_stride=1 << 40), dict(gate_stride=1 << 40),
               dict(d_offset=A + 4), dict(d_r=None), dict(d_r=A + 1), dict(d_h=A + 1), dict(d_status=A + 2),
               dict(d_y=None),                                      # a join's output without a join
               dict(d_y=None, d_r=None),                            # its weights too
               dict(d_y=None, d_r=None, d_gate=None),
               dict(d_y=None, d_r=None, d_gate=None, d_post_weight=None, d_h=None),
               dict(d_h=None),                                      # a weight of nothing
               dict(x_stride=24)):                                  # rows of x and r in one place, apart differently
        assert call(**kw) == z.INVALID_ARG, kw
    assert call(config(z, post=0)) == z.INVALID_ARG                 # a post weight without post
    assert z.lib().zccl_residual_norm(None, A, 0, 16, A, 0, 16, A, A, 1, A, 0, 16, 1, 4, 0, None, A, A, None, None) == z.INVALID_ARG
    assert call(rows=0, d_x=None, d_y=None, d_r=None, d_h=None) == z.OK


def test_norm_backward_refusals(z):
    need = z.zccl_residual_norm_workspace_bytes(16, 4)
    ok = dict(d_grad_r=A, grad_r_stride=16, d_grad_h=A, grad_h_stride=16, d_r=A, x_dtype=z.F32, r_stride=16, d_y=A,
              dtype=z.BF16, y_stride=16, d_weight=A, d_post_weight=A, weight_dtype=z.F32, d_gate=A, gate_dtype=z.BF16,
              gate_stride=16, gate_span=2, rows=4, offset=0, d_offset=None, d_grad_x=A, d_grad_y=A, d_grad_weight=A,
              d_grad_post_weight=A, d_grad_gate=A, d_ws=A, ws_bytes=need, d_status=None, stream=None)

    def call(c=None, **kw):
        return z.zccl_residual_norm_backward(c or config(z), **dict(ok, **kw))

    for kw in BAD_CONFIGS:
        assert call(config(z, **kw)) == z.INVALID_ARG, kw
    for kw in (dict(d_grad_r=A + 2), dict(d_grad_h=A + 1), dict(d_r=None), dict(d_r=A + 2), dict(d_y=None), dict(d_y=A + 1),
               dict(d_grad_r=None, d_grad_h=None, d_weight=None, d_grad_weight=None), dict(d_grad_h=None), dict(x_dtype=2),
               dict(dtype=2), dict(weight_dtype=2), dict(gate_dtype=2), dict(d_grad_x=A + 2), dict(d_grad_y=A + 1),
               dict(d_grad_weight=A + 2), dict(d_grad_post_weight=A + 2), dict(d_grad_gate=A + 1), dict(gate_span=0),
               dict(d_weight=None), dict(d_post_weight=None), dict(d_gate=None),  # gradients of what is not there
               dict(d_grad_y=None),                                              # a norm alone with a join's weights
               dict(rows=1 << 31), dict(grad_r_stride=1 << 40), dict(grad_h_stride=1 << 40), dict(r_stride=1 << 40),
               dict(y_stride=1 << 40), dict(d_ws=None), dict(d_ws=A + 8), dict(d_offset=A + 4), dict(d_status=A + 1)):
        assert call(**kw) == z.INVALID_ARG, kw
    alone = dict(d_grad_y=None, d_gate=None, d_grad_gate=None, d_post_weight=None, d_grad_post_weight=None)
    assert call(**alone, d_grad_x=None, d_grad_weight=None) == z.INVALID_ARG  # nothing is wanted
    assert call(ws_bytes=need - 1) == z.BUFFER_TOO_SMALL
    assert call(rows=0, d_grad_weight=None, d_grad_post_weight=None, d_ws=None, ws_bytes=0) == z.OK
    for bad in ((0, 4), (65537, 4), (16, 1 << 31)):
        with pytest.raises(z.ZcclError):
            z.zccl_residual_norm_workspace_bytes(*bad)
    assert z.zccl_residual_norm_workspace_bytes(65536, (1 << 31) - 1) < 1 << 28


def test_dropout_refusals(z):
    ok = dict(d_x=A, dtype=z.BF16, stride=16, rows=4, cols=16, p=0.5, seed=1, offset=2, d_offset=None, d_out=A + 4096,
              stream_handle=None)
    for kw in (dict(d_x=None), dict(d_x=A + 1), dict(dtype=2), dict(rows=1 << 32), dict(cols=1 << 24), dict(p=-0.5), dict(p=1.5),
               dict(p=NAN), dict(d_offset=A + 4), dict(d_out=None), dict(d_out=A + 1), dict(stride=1 << 40),
               dict(rows=1 << 31, cols=1 << 20), dict(d_out=A, stride=24)):
        assert z.zccl_dropout(**dict(ok, **kw)) == z.INVALID_ARG, kw
    assert z.zccl_dropout(**dict(ok, rows=0, d_x=None, d_out=None)) == z.OK
    assert z.zccl_dropout(**dict(ok, cols=0, d_x=None, d_out=None)) == z.OK


def test_balance_refusals(z):
    def cfg(**kw):
        return z.Route(*dict(dict(experts=8, top_k=2, groups=1, top_groups=1, score=0, renormalize=1, scale=1.0), **kw).values())

    need = z.zccl_balance_workspace_bytes(3, 8)
    both = dict(d_logits=A, dtype=z.F32, stride=8, d_idx=A, tokens=4, d_seq=A, sequences=3, coefficient=1.0)
    ok = dict(both, d_loss=A, d_counts=A, d_tokens=A, d_ws=A, ws_bytes=need, stream=None)
    back = dict(both, d_counts=A, d_tokens=A, d_grad_loss=None, d_grad_logits=A, grad_stride=8, accumulate=False, stream=None)
    for c in (cfg(experts=0), cfg(experts=513), cfg(top_k=0), cfg(top_k=33), cfg(score=2)):
        assert z.zccl_balance(c, **ok) == z.INVALID_ARG
        assert z.zccl_balance_backward(c, **back) == z.INVALID_ARG
    for kw in (dict(d_logits=None), dict(d_logits=A + 2), dict(dtype=2), dict(d_idx=None), dict(d_idx=A + 2), dict(tokens=1 << 30),
               dict(stride=1 << 40), dict(d_seq=None), dict(d_seq=A + 2), dict(sequences=0), dict(sequences=65537),
               dict(coefficient=NAN), dict(coefficient=INF)):
        assert z.zccl_balance(cfg(), **dict(ok, **kw)) == z.INVALID_ARG, kw
        assert z.zccl_balance_backward(cfg(), **dict(back, **kw)) == z.INVALID_ARG, kw
    for kw in (dict(d_loss=None), dict(d_counts=None), dict(d_tokens=A + 1), dict(d_ws=None)):
        assert z.zccl_balance(cfg(), **dict(ok, **kw)) == z.INVALID_ARG, kw
    for kw in (dict(d_counts=None), dict(d_tokens=None), dict(d_grad_loss=A + 2), dict(d_grad_logits=None), dict(grad_stride=7),
               dict(grad_stride=1 << 40)):
        assert z.zccl_balance_backward(cfg(), **dict(back, **kw)) == z.INVALID_ARG, kw
    assert z.zccl_balance(cfg(), **dict(ok, ws_bytes=need - 1)) == z.BUFFER_TOO_SMALL
    assert z.zccl_balance_backward(cfg(), **dict(back, tokens=0, d_logits=None, d_idx=None, d_grad_logits=None)) == z.OK
    for bad in ((0, 8), (65537, 8), (1, 0), (1, 513)):
        with pytest.raises(z.ZcclError):
            z.zccl_balance_workspace_bytes(*bad)


# ---- the classes: on the CPU's tensors, with a library that launches nothing ----
class Launches:
    def __init__(self):
        self.names = []

    def __getattr__(self, name):
        def call(*args):
            self.names.append(name)
            return 0
        return call


@pytest.fixture
def fake(z, monkeypatch):
    from lossless_bf16_exponent_split_gb300 import moe, norm
    monkeypatch.setattr(moe, "current_stream", lambda device: 0)
    monkeypatch.setattr(norm, "current_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return z


def test_class_refusals(fake):
    z = fake
    for kw in (dict(hidden=0), dict(hidden=65537), dict(hidden=8, seed=-1), dict(hidden=8, seed=1 << 64)):
        with pytest.raises(ValueError):
            z.ResidualNorm(**kw, device="cpu")
    for kw in (dict(eps=0.0), dict(scale=NAN), dict(dropout=1.5)):
        with pytest.raises(z.ZcclError):
            z.ResidualNorm(8, **kw, device="cpu")
    for kw in (dict(p=-0.1), dict(p=1.1), dict(p=NAN), dict(p=0.5, seed=1 << 64)):
        with pytest.raises(ValueError):
            z.Dropout(**kw, device="cpu")
    n, plain, drop = z.ResidualNorm(8, post=True, device="cpu"), z.ResidualNorm(8, device="cpu"), z.Dropout(0.5, device="cpu")
    n._lib = plain._lib = drop._lib = lib = Launches()
    x, y, w = torch.zeros(6, 8), torch.zeros(6, 8).bfloat16(), torch.ones(8)
    half = torch.zeros(6, 8, dtype=torch.float16)
    bad = [
        lambda: n.norm(half), lambda: n.norm(x[:, :7]), lambda: n.norm(x[0]), lambda: n.norm(x.t().contiguous().t()),
        lambda: n.norm(x, w[:7]), lambda: n.norm(x, w.half()), lambda: n.norm(x, torch.ones(16)[::2]), lambda: n.norm(x, dtype=torch.float16),
        lambda: n.norm([1.0]), lambda: n.norm(x, w.tolist()),
        lambda: n.norm_backward(y[:5], x), lambda: n.norm_backward(half, x), lambda: n.norm_backward(y, half),
        lambda: n.add(x, y[:5]), lambda: n.add(x[:5], y), lambda: n.add(x, half), lambda: n.add(x, y, w, normed=False),
        lambda: n.add(x, y, w, post_weight=w.bfloat16()), lambda: plain.add(x, y, post_weight=w),
        lambda: n.add(x, y, gate=torch.zeros(4, 8)), lambda: n.add(x, y, gate=torch.zeros(0, 8)), lambda: n.add(x, y, gate=torch.zeros(6, 7)),
        lambda: n.add(x, y, gate=half), lambda: n.add(x, y, gate=torch.zeros(12, 8)), lambda: n.add(x, y, offset=-1), lambda: n.add(x, y, offset=1 << 64),
        lambda: n.add(x, y, offset=torch.zeros(2, dtype=torch.int64)), lambda: n.add(x, y, offset=torch.zeros(1, dtype=torch.int32)),
        lambda: n.add_backward(None, None, x, y), lambda: n.add_backward(x, y, None, y), lambda: n.add_backward(x, x, x, y),
        lambda: n.add_backward(y, y, x, y), lambda: n.add_backward(x, None, None, y, w), lambda: n.add_backward(x[:5], y, x, y),
        lambda: n.add_backward(x, y[:5], x, y), lambda: n.add_backward(x, y, x[:5], y),
        lambda: drop.apply(half), lambda: drop.apply(x[0]), lambda: drop.apply(x, out=y), lambda: drop.apply(x, out=x[:5]),
        lambda: drop.apply(x, out=torch.zeros(6, 16)[:, :8]), lambda: drop.apply(x, offset=-1),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    assert not lib.names
    gate = torch.zeros(2, 24)[:, 8:16]  # rows of a wider matrix
    r, h = n.add(x, y, w, post_weight=w, gate=gate, offset=torch.zeros((), dtype=torch.int64))
    assert (r.dtype, h.dtype) == (torch.float32, torch.bfloat16) and n.add(x, y, normed=False)[1] is None
    g = n.add_backward(x, None, None, y, gate=gate)
    assert g.x is x and g.weight is None and g.post_weight is None and g.gate.shape == gate.shape
    empty = n.add_backward(x[:0], y[:0], x[:0], y[:0], w, gate=gate)
    assert empty.x.shape == (0, 8) and bool((empty.gate == 0).all())
    assert lib.names == ["zccl_residual_norm"] * 2 + ["zccl_residual_norm_backward"] * 2


def test_balance_class_refusals(fake):
    z = fake
    moe = z.Moe(4, 2, device="cpu")
    moe._lib = lib = Launches()
    l, idx = torch.zeros(5, 4), torch.zeros(5, 2, dtype=torch.int32)
    seq = torch.tensor([0, 2, 5], dtype=torch.int32)
    b = z.Balance(torch.zeros(1), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    bad = [
        lambda: moe.balance(l.half(), idx), lambda: moe.balance(l[:, :3], idx), lambda: moe.balance(l, idx.long()),
        lambda: moe.balance(l, idx[:4]), lambda: moe.balance(l, idx[:, :1]), lambda: moe.balance(l, idx, seq.long()),
        lambda: moe.balance(l, idx, seq[:1]), lambda: moe.balance(l, idx, seq[None]),
        lambda: moe.balance_backward(l, idx, b, seq), lambda: moe.balance_backward(l, idx, b._replace(tokens=b.tokens[:1])),
        lambda: moe.balance_backward(l, idx, b, grad_loss=torch.zeros(2)), lambda: moe.balance_backward(l, idx, b, grad_loss=torch.zeros(1).double()),
        lambda: moe.balance_backward(l, idx, b, out=l.bfloat16()), lambda: moe.balance_backward(l, idx, b, out=l[:4]),
        lambda: moe.balance_backward(l, idx, b, out=torch.zeros(1, 4).expand(5, 4)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    assert not lib.names
    got = moe.balance(l, idx, seq)
    assert got.counts.shape == (2, 4) and got.tokens.shape == (3,)
    out = torch.zeros(5, 4)
    assert moe.balance_backward(l, idx, got, seq, grad_loss=torch.ones(()), out=out) is out
    assert lib.names == ["zccl_balance", "zccl_balance_backward"]


def test_a_handle_of_another_device_refuses(z, monkeypatch):
    from lossless_bf16_exponent_split_gb300 import moe
    monkeypatch.setattr(moe, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    n, drop, m = z.ResidualNorm(8, device="cpu"), z.Dropout(0.5, device="cpu"), z.Moe(4, 2, device="cpu")
    n._lib = drop._lib = m._lib = lib = Launches()
    x, l, idx = torch.zeros(6, 8), torch.zeros(5, 4), torch.zeros(5, 2, dtype=torch.int32)
    b = z.Balance(torch.zeros(1), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    for call in (lambda: n.norm(x), lambda: n.norm_backward(x, x), lambda: n.add(x, x), lambda: n.add_backward(x, x, x, x),
                 lambda: drop.apply(x), lambda: m.balance(l, idx), lambda: m.balance_backward(l, idx, b)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    assert not lib.names
