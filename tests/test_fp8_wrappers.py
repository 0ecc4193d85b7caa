"""CPU: the package's functions of the block-scaled e4m3 calls hand their
arguments on in the library's order: each bad one alone is refused."""
import pytest

A = 1 << 20  # a fake, aligned "device" address: never dereferenced


@pytest.fixture(scope="module")
def z():
    from lossless_bf16_exponent_split_gb300 import build
    build.build()
    import lossless_bf16_exponent_split_gb300 as z
    z.lib()
    return z


def refused(z, call, ok, changes):
    for change in changes:
        assert call(**dict(ok, **change)) == z.INVALID_ARG, change


def test_weights(z):
    both = dict(groups=2, n=130, k=200, d_weight=A, d_weight_t=A, stream=None)
    changes = (dict(groups=0), dict(n=0), dict(k=0), dict(n=1 << 24), dict(d_weight=A + 8), dict(d_weight_t=A + 8),
               dict(d_weight=None, d_weight_t=None))
    refused(z, z.zccl_fp8_weight_quantize, dict(both, d_w=A, dtype=z.F32), changes + (dict(d_w=None), dict(d_w=A + 2), dict(dtype=2)))
    refused(z, z.zccl_fp8_weight_pack, dict(both, d_codes=A, d_scale=A), changes + (dict(d_codes=None), dict(d_scale=A + 2)))


def test_products(z):
    both = dict(dtype=z.BF16, rows=64, k=200, n=130, groups=2, d_offsets=A, out_dtype=z.F32, d_ws=A, d_status=A, stream=None)
    changes = (dict(dtype=2), dict(rows=1 << 31), dict(k=0), dict(n=0), dict(groups=0), dict(d_offsets=None), dict(out_dtype=2),
               dict(d_ws=None), dict(d_status=A + 2))
    ws = z.zccl_fp8_linear_workspace_bytes(64, 200, 130, 2, False)
    ok = dict(both, d_x=A, stride=200, d_weight=A, d_out=A, ws_bytes=ws)
    refused(z, z.zccl_fp8_linear, ok, changes + (dict(d_x=A + 1), dict(stride=1 << 40), dict(d_weight=A + 8), dict(d_out=A + 2)))
    assert z.zccl_fp8_linear(**dict(ok, ws_bytes=ws - 1)) == z.BUFFER_TOO_SMALL
    assert z.zccl_fp8_linear(**dict(ok, rows=0)) == z.OK
    ws = z.zccl_fp8_linear_workspace_bytes(64, 200, 130, 2, True)
    ok = dict(both, d_grad=A, d_x=A, grad_stride=130, x_stride=200, d_weight_t=A, d_grad_x=A, d_grad_w=A, ws_bytes=ws)
    refused(z, z.zccl_fp8_linear_backward, ok, changes + (
        dict(d_grad=None), dict(d_x=None), dict(grad_stride=1 << 40), dict(x_stride=1 << 40), dict(d_weight_t=None),
        dict(d_grad_x=A + 2), dict(d_grad_w=A + 2)))
    assert z.zccl_fp8_linear_backward(**dict(ok, ws_bytes=ws - 1)) == z.BUFFER_TOO_SMALL
