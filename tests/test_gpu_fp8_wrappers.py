"""GPU: a block-scaled e4m3 layer through the package's functions, without the
convenience class: the same bits."""
import pytest
import torch

from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


def test_layer_and_gradients(z):
    rows, k, n, groups = 150, 200, 136, 3
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rows, k, generator=gen, device="cuda").bfloat16()
    grad = torch.randn(rows, n, generator=gen, device="cuda").bfloat16()
    w = torch.randn(groups, n, k, generator=gen, device="cuda")
    offsets = torch.tensor([0, 40, 40, 141], dtype=torch.int32, device="cuda")
    fp8 = z.BlockFp8()
    weight = fp8.quantize_weight(w, backward=True)
    y, (dx, dw) = fp8.linear(x, weight, offsets), fp8.linear_backward(grad, x, weight, offsets)

    def buffer(nbytes):
        return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")

    stream, status = torch.cuda.current_stream().cuda_stream, torch.zeros(1, dtype=torch.int32, device="cuda")
    packed, packed_t = buffer(z.zccl_fp8_weight_bytes(groups, n, k)), buffer(z.zccl_fp8_weight_bytes(groups, k, n))
    z.check(z.zccl_fp8_weight_quantize(w.data_ptr(), z.F32, groups, n, k, packed.data_ptr(), packed_t.data_ptr(), stream), "quantize")
    ws = buffer(max(z.zccl_fp8_linear_workspace_bytes(rows, k, n, groups, b) for b in (False, True)))
    out, out_x, out_w = torch.empty_like(y), torch.empty_like(dx), torch.empty_like(dw)
    z.check(z.zccl_fp8_linear(x.data_ptr(), z.BF16, k, rows, k, packed.data_ptr(), n, groups, offsets.data_ptr(), out.data_ptr(),
                              z.BF16, ws.data_ptr(), ws.numel(), status.data_ptr(), stream), "linear")
    z.check(z.zccl_fp8_linear_backward(grad.data_ptr(), x.data_ptr(), z.BF16, n, k, rows, k, packed_t.data_ptr(), n, groups,
                                       offsets.data_ptr(), out_x.data_ptr(), out_w.data_ptr(), z.BF16, ws.data_ptr(), ws.numel(),
                                       status.data_ptr(), stream), "backward")
    assert torch.equal(out, y) and torch.equal(out_x, dx) and torch.equal(out_w, dw)
    assert status.item() == z.OK

    # codes and scales, all 1: what a checkpoint brings
    codes, scale = torch.ones(groups, n, k, device="cuda").to(torch.float8_e4m3fn), torch.ones(groups, 2, 2, device="cuda")
    z.check(z.zccl_fp8_weight_pack(codes.data_ptr(), scale.data_ptr(), groups, n, k, packed.data_ptr(), packed_t.data_ptr(), stream),
            "pack")
    same = fp8.weight(codes, scale, backward=True)
    code_bytes = groups * 2 * n * 128  # blocks of k, then the scales
    assert torch.equal(packed[:code_bytes], same.packed[:code_bytes])
    assert torch.equal(packed[code_bytes:].view(torch.float32), torch.ones(groups * 4, device="cuda"))
    assert torch.equal(packed_t, same.packed_t)
