"""CPU: argument errors of the block-scaled e4m3 calls are returned before any
CUDA call, the size formulas follow the documented blocks, and the tests' own
rounding to e4m3 agrees with PyTorch's."""
import numpy as np
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


def call(z, name, *args):
    return getattr(z.lib(), name)(*args)


def refused(z, name, ok, changes):
    for change in changes:
        assert call(z, name, *dict(ok, **change).values()) == z.INVALID_ARG, (name, change)


def test_weight_refusals(z):
    ok = dict(d_w=A, dtype=z.BF16, groups=2, n=130, k=200, d_weight=A, d_weight_t=A, stream=None)
    refused(z, "zccl_fp8_weight_quantize", ok, (
        dict(d_w=None), dict(d_w=A + 1), dict(dtype=2), dict(groups=0), dict(n=0), dict(k=0), dict(n=1 << 24), dict(k=1 << 24),
        dict(d_weight=A + 8), dict(d_weight_t=A + 8), dict(d_weight=None, d_weight_t=None)))
    ok = dict(d_codes=A, d_scale=A, groups=2, n=130, k=200, d_weight=A, d_weight_t=A, stream=None)
    refused(z, "zccl_fp8_weight_pack", ok, (
        dict(d_codes=None), dict(d_scale=None), dict(d_scale=A + 2), dict(groups=0), dict(n=0), dict(k=1 << 24),
        dict(d_weight=A + 4), dict(d_weight=None, d_weight_t=None)))
    for shape in ((0, 1, 1), (1, 0, 1), (1, 1, 1 << 24)):
        with pytest.raises(z.ZcclError):
            z.zccl_fp8_weight_bytes(*shape)


def test_linear_refusals(z):
    ws = z.zccl_fp8_linear_workspace_bytes(64, 200, 130, 2, False)
    ok = dict(d_x=A, dtype=z.BF16, stride=200, rows=64, k=200, d_weight=A, n=130, groups=2, d_offsets=A, d_out=A,
              out_dtype=z.BF16, d_ws=A, ws_bytes=ws, d_status=A, stream=None)
    refused(z, "zccl_fp8_linear", ok, (
        dict(d_x=None), dict(d_x=A + 1), dict(dtype=3), dict(out_dtype=-1), dict(stride=1 << 40), dict(rows=1 << 31), dict(k=0),
        dict(n=0), dict(n=1 << 24), dict(groups=0), dict(d_weight=None), dict(d_weight=A + 8), dict(d_offsets=None),
        dict(d_offsets=A + 2), dict(d_out=None), dict(d_out=A + 1), dict(d_ws=None), dict(d_status=A + 1)))
    assert call(z, "zccl_fp8_linear", *dict(ok, ws_bytes=ws - 1).values()) == z.BUFFER_TOO_SMALL


def test_linear_backward_refusals(z):
    ws = z.zccl_fp8_linear_workspace_bytes(64, 200, 130, 2, True)
    ok = dict(d_grad=A, d_x=A, dtype=z.BF16, grad_stride=130, x_stride=200, rows=64, k=200, d_weight_t=A, n=130, groups=2,
              d_offsets=A, d_grad_x=A, d_grad_w=A, out_dtype=z.F32, d_ws=A, ws_bytes=ws, d_status=A, stream=None)
    refused(z, "zccl_fp8_linear_backward", ok, (
        dict(d_grad=None), dict(d_x=None), dict(dtype=2), dict(out_dtype=2), dict(grad_stride=1 << 40), dict(x_stride=1 << 40),
        dict(rows=1 << 31), dict(k=1 << 24), dict(groups=0), dict(d_weight_t=None), dict(d_offsets=None), dict(d_grad_x=A + 2),
        dict(d_grad_w=A + 2), dict(groups=513), dict(d_ws=None), dict(d_status=A + 2)))
    assert call(z, "zccl_fp8_linear_backward", *dict(ok, ws_bytes=ws - 1).values()) == z.BUFFER_TOO_SMALL


def test_weight_bytes_hold_the_codes_and_their_scales(z):
    for groups, n, k in ((1, 1, 1), (3, 128, 128), (2, 129, 257), (64, 1024, 2048)):
        blocks = -(-n // 128) * -(-k // 128)
        assert z.zccl_fp8_weight_bytes(groups, n, k) >= groups * (n * -(-k // 128) * 128 + 4 * blocks)


def test_reference_rounding_is_torch_rounding():
    import fp8_ref
    v = np.concatenate([np.random.default_rng(0).uniform(-448, 448, 4000).astype(np.float32),
                        np.arange(-470, 470, dtype=np.float32) / 16, np.float32(2.0) ** np.arange(-14, 9)])
    v = v[np.abs(v) <= 448]
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(fp8_ref.round_e4m3(v), want)
