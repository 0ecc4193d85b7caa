"""GPU: handles of the mixture-of-experts calls shared by host threads, on one
stream and on several: every result is the one the call gives alone, bit for bit."""
import threading

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


def run_threads(work, own_stream, threads=4, times=20):
    """work(i) -> list of tensors, `times` times in each thread; the last results of each."""
    start, results, errors = threading.Barrier(threads), [[] for _ in range(threads)], []

    def run(i):
        try:
            stream = torch.cuda.Stream() if own_stream else torch.cuda.current_stream()
            stream.wait_stream(torch.cuda.default_stream())
            start.wait()
            with torch.cuda.stream(stream):
                for _ in range(times):
                    results[i].append(work(i))
            stream.synchronize()
        except Exception as e:  # a failed thread fails the test
            errors.append(e)

    pool = [threading.Thread(target=run, args=(i,)) for i in range(threads)]
    for t in pool:
        t.start()
    for t in pool:
        t.join()
    assert not errors, errors
    return results


def check(work, own_stream):
    want = [[t.clone() for t in work(i)] for i in range(4)]
    torch.cuda.synchronize()
    for i, outs in enumerate(run_threads(work, own_stream)):
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


# rows: a serving step's kernel, the tensor-core kernel, that kernel with its reduction in parts
@pytest.mark.parametrize("own_stream", [False, True])
@pytest.mark.parametrize("rows,k,n", [(3, 512, 384), (300, 512, 384), (70, 4096, 256)])
def test_products(z, rows, k, n, own_stream):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    fp8 = z.BlockFp8()
    w = fp8.quantize_weight(torch.randn(1, n, k, generator=gen, device="cuda"), backward=True)
    x = [torch.randn(rows + i, k, generator=gen, device="cuda").bfloat16() for i in range(4)]
    grad = [torch.randn(rows + i, n, generator=gen, device="cuda").bfloat16() for i in range(4)]
    check(lambda i: [fp8.linear(x[i], w), *fp8.linear_backward(grad[i], x[i], w)], own_stream)
    assert fp8.read_status() == z.OK


# slots: counted by every CTA, and by the counting kernel
@pytest.mark.parametrize("own_stream", [False, True])
@pytest.mark.parametrize("tokens", [50, 4000])
def test_dispatch(z, tokens, own_stream):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    moe = z.Moe(16, 8)
    x = [torch.randn(tokens + i, 64, generator=gen, device="cuda").bfloat16() for i in range(4)]
    idx = [torch.randint(-1, 16, (tokens + i, 8), generator=gen, device="cuda", dtype=torch.int32) for i in range(4)]

    def work(i):
        d = moe.dispatch(x[i], idx[i])
        return [d.rows, d.pos, d.counts, d.offsets]

    check(work, own_stream)
    assert moe.read_status() == z.OK
