"""CPU: the calls launch on the current CUDA device, so a handle of another
device refuses them and launches nothing."""
import pytest
import torch


class Launches:
    def __init__(self):
        self.names = []

    def __getattr__(self, name):
        def call(*args):
            self.names.append(name)
            return 0
        return call


@pytest.fixture
def z(monkeypatch):
    from lossless_bf16_exponent_split_gb300 import build
    build.build()
    import lossless_bf16_exponent_split_gb300 as z
    from lossless_bf16_exponent_split_gb300 import moe
    z.lib()
    monkeypatch.setattr(moe, "_raw_stream", lambda index: 0)  # the default stream has this handle on every device
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    return z


def calls(z):
    """(handle, call) of every call that launches; the handles' tensors are the CPU's, which is never current."""
    moe, fp8 = z.Moe(4, 2, device="cpu"), z.BlockFp8(device="cpu")
    logits, slots = torch.zeros(5, 4), torch.zeros(5, 2, dtype=torch.int32)
    weights, offsets = torch.zeros(5, 2), torch.zeros(5, dtype=torch.int32)
    x, rows = torch.zeros(5, 8, dtype=torch.bfloat16), torch.zeros(10, 8, dtype=torch.bfloat16)
    w = z.Fp8Weight(1, 8, 16, torch.zeros(4096, dtype=torch.uint8), torch.zeros(4096, dtype=torch.uint8))
    a, grad = torch.zeros(3, 16), torch.zeros(3, 8)
    return [
        (moe, lambda: moe.route(logits)),
        (moe, lambda: moe.route_backward(logits, slots, weights)),
        (moe, lambda: moe.dispatch(x, slots)),
        (moe, lambda: moe.dispatch(x, slots, capacity=2)),
        (moe, lambda: moe.combine(rows, slots, weights)),
        (moe, lambda: moe.combine_backward(x, rows, slots, weights, offsets)),
        (fp8, lambda: fp8.quantize_weight(torch.zeros(1, 8, 16))),
        (fp8, lambda: fp8.weight(torch.zeros(1, 8, 16).to(torch.float8_e4m3fn), torch.ones(1, 1, 1))),
        (fp8, lambda: fp8.linear(a, w)),
        (fp8, lambda: fp8.linear_backward(grad, a, w)),
    ]


@pytest.mark.parametrize("i", range(10))
def test_a_handle_of_another_device_refuses(z, i):
    handle, call = calls(z)[i]
    handle._lib = lib = Launches()
    with pytest.raises(ValueError, match="current CUDA device"):
        call()
    assert not lib.names


def test_the_current_device_is_taken(z):
    from lossless_bf16_exponent_split_gb300 import moe
    assert moe.current_stream(torch.device("cuda", 1)) == 0
    for other in (torch.device("cuda", 0), torch.device("cuda", 2)):
        with pytest.raises(ValueError, match="current CUDA device"):
            moe.current_stream(other)
