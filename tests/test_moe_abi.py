"""CPU: argument errors of the mixture-of-experts calls are returned before any
CUDA call, and the size formulas bound what they size."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def z():
    from lossless_bf16_exponent_split_gb300 import build
    build.build()
    import lossless_bf16_exponent_split_gb300 as z
    z.lib()
    return z


A = 1 << 20  # a fake, aligned "device" address: never dereferenced


def test_route_refusals(z):
    def cfg(**kw):
        base = dict(experts=8, top_k=2, groups=1, top_groups=1, score=0, renormalize=1, scale=1.0)
        return z.Route(*dict(base, **kw).values())

    def route(c=None, **kw):
        a = dict(d_logits=A, dtype=z.F32, stride=8, d_bias=None, tokens=4, d_idx=A, d_weights=A, d_status=A, stream=None)
        return z.zccl_route(c or cfg(), **dict(a, **kw))

    for c in (cfg(experts=0), cfg(experts=513), cfg(top_k=0), cfg(top_k=9), cfg(groups=3), cfg(groups=0),
              cfg(groups=2, top_groups=3), cfg(groups=4, top_groups=1, top_k=3), cfg(score=2), cfg(scale=float("inf")),
              cfg(experts=64, groups=64)):
        assert route(c) == z.INVALID_ARG
        assert z.zccl_route_backward(c, A, z.F32, 8, A, A, 4, A, 8, None) == z.INVALID_ARG
    for kw in (dict(d_logits=None), dict(d_logits=A + 2), dict(dtype=2), dict(d_idx=None), dict(d_weights=A + 1),
               dict(tokens=1 << 30), dict(d_bias=A + 2), dict(d_status=A + 1)):
        assert route(**kw) == z.INVALID_ARG, kw
    assert route(tokens=0, d_logits=None, d_idx=None, d_weights=None) == z.OK
    assert z.zccl_route_backward(cfg(), A, z.F32, 8, A, A, 4, A, 7, None) == z.INVALID_ARG  # rows overlap
    assert z.lib().zccl_route(None, A, z.F32, 8, None, 4, A, A, None, None) == z.INVALID_ARG


def test_dispatch_and_combine_refusals(z):
    ws = z.zccl_dispatch_workspace_bytes(4, 8, 2)
    room = z.zccl_dispatch_stream_bytes(8, 16, 8)
    ok = dict(d_idx=A, tokens=4, experts=8, top_k=2, d_x=A, stride=16, hidden=16, d_rows=A, d_pos=A, d_counts=A,
              d_offsets=A, d_segs=A, capacity=1, d_streams=A, stream_bytes=room, d_ws=A, ws_bytes=ws, stream_handle=None)
    for kw in (dict(d_idx=None), dict(experts=0), dict(experts=513), dict(top_k=33), dict(tokens=1 << 30), dict(hidden=12),
               dict(stride=20), dict(d_x=A + 8), dict(d_rows=None), dict(d_rows=A + 8), dict(d_pos=None), dict(d_counts=None),
               dict(d_offsets=A + 2), dict(d_segs=A + 4), dict(d_streams=None), dict(d_streams=A + 8), dict(d_ws=None),
               dict(hidden=1 << 24)):
        assert z.zccl_dispatch(**dict(ok, **kw)) == z.INVALID_ARG, kw
    assert z.zccl_dispatch(**dict(ok, ws_bytes=ws - 1)) == z.BUFFER_TOO_SMALL
    assert z.zccl_dispatch(**dict(ok, stream_bytes=room - 1)) == z.BUFFER_TOO_SMALL
    for bad in ((0, 0), (513, 1), (8, 0), (8, 33)):
        with pytest.raises(z.ZcclError):
            z.zccl_dispatch_workspace_bytes(4, *bad)
    ok = dict(d_y=A, rows=8, hidden=16, d_pos=A, d_weights=A, tokens=4, top_k=2, d_out=A, stream=None)
    for kw in (dict(d_y=A + 8), dict(d_y=None), dict(hidden=12), dict(d_pos=None), dict(d_weights=A + 2), dict(top_k=0),
               dict(d_out=None), dict(d_out=A + 4), dict(rows=1 << 31)):
        assert z.zccl_combine(**dict(ok, **kw)) == z.INVALID_ARG, kw
    assert z.zccl_combine(**dict(ok, tokens=0)) == z.OK
    ok = dict(d_grad_out=A, d_y=A, rows=8, hidden=16, d_pos=A, d_weights=A, d_total=A, tokens=4, top_k=2, d_grad_y=A,
              d_grad_weights=A, stream=None)
    for kw in (dict(d_grad_out=None), dict(d_y=None), dict(d_grad_y=None), dict(d_grad_y=A + 8), dict(d_total=A + 2),
               dict(d_pos=None), dict(d_grad_weights=A + 1)):
        assert z.zccl_combine_backward(**dict(ok, **kw)) == z.INVALID_ARG, kw
    assert z.zccl_combine_backward(**dict(ok, tokens=0, rows=0)) == z.OK


def test_stream_room_bounds_every_split(z):
    rng = np.random.default_rng(0)
    for _ in range(200):
        experts, hidden = int(rng.integers(1, 20)), 8 * int(rng.integers(1, 300))
        rows = rng.integers(0, 40, 2 * experts)
        need = sum(-(-z.zccl_max_compressed_bytes(int(r) * hidden) // 128) * 128 for r in rows)
        assert need <= z.zccl_dispatch_stream_bytes(int(rows.sum()), hidden, experts)
