"""CPU: a handle of the mixture-of-experts calls may be used by several host
threads on one stream: the kernels of one call that share a workspace are
queued one after the other, with no other call's between them."""
import threading
import time

import pytest
import torch


class Recorder:
    """Stands for the library: a call takes a while, as one that queues several
    kernels does, and is noted if another call has its workspace meanwhile."""

    def __init__(self, **workspace_at):
        self._at, self._guard, self._busy = workspace_at, threading.Lock(), set()
        self.calls, self.shared = 0, 0

    def __getattr__(self, name):
        at = self._at[name]

        def call(*args):
            with self._guard:
                self.calls += 1
                self.shared += args[at] in self._busy
                self._busy.add(args[at])
            time.sleep(0.002)
            with self._guard:
                self._busy.discard(args[at])
            return 0

        return call


@pytest.fixture
def z(monkeypatch):
    from lossless_bf16_exponent_split_gb300 import build
    build.build()
    import lossless_bf16_exponent_split_gb300 as z
    from lossless_bf16_exponent_split_gb300 import fp8, moe
    z.lib()
    for module in (fp8, moe):
        monkeypatch.setattr(module, "current_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return z


def in_threads(work, threads=4, times=5):
    start, errors = threading.Barrier(threads), []

    def run(i):
        try:
            start.wait()
            for _ in range(times):
                work(i)
        except Exception as e:  # a failed thread fails the test
            errors.append(e)

    pool = [threading.Thread(target=run, args=(i,)) for i in range(threads)]
    for t in pool:
        t.start()
    for t in pool:
        t.join()
    assert not errors, errors


def test_threads_do_not_share_a_product_s_workspace(z):
    fp8 = z.BlockFp8(device="cpu")
    fp8._lib = lib = Recorder(zccl_fp8_linear=11, zccl_fp8_linear_backward=14)
    w = z.Fp8Weight(1, 8, 16, torch.zeros(4096, dtype=torch.uint8), torch.zeros(4096, dtype=torch.uint8))
    x, grad = torch.zeros(3, 16), torch.zeros(3, 8)
    in_threads(lambda i: fp8.linear(x, w) if i % 2 else fp8.linear_backward(grad, x, w))
    assert lib.calls == 20 and lib.shared == 0


def test_threads_do_not_share_a_dispatch_s_workspace(z):
    moe = z.Moe(4, 2, device="cpu")
    moe._lib = lib = Recorder(zccl_dispatch=15)
    x, idx = torch.zeros(5, 8, dtype=torch.bfloat16), torch.zeros(5, 2, dtype=torch.int32)
    in_threads(lambda i: moe.dispatch(x, idx))
    assert lib.calls == 20 and lib.shared == 0


def test_a_call_that_fails_leaves_the_handle_usable(z):
    fp8 = z.BlockFp8(device="cpu")

    class Refuses:
        def zccl_fp8_linear(self, *args):
            return z.CUDA_ERROR

    w = z.Fp8Weight(1, 8, 16, torch.zeros(4096, dtype=torch.uint8), None)
    fp8._lib = Refuses()
    with pytest.raises(z.ZcclError):
        fp8.linear(torch.zeros(3, 16), w)
    fp8._lib = lib = Recorder(zccl_fp8_linear=11)
    done = threading.Thread(target=fp8.linear, args=(torch.zeros(3, 16), w), daemon=True)
    done.start()
    done.join(10)
    assert not done.is_alive() and lib.calls == 1
