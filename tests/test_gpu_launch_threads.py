"""GPU: host threads that call one kernel at different sizes at once.  How much shared
memory a kernel may be launched with belongs to the kernel and not to the launch: a
call must not take from another thread's what that is about to be launched with."""
import ctypes
import threading

import pytest
import torch

from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


def statuses(calls, times):
    """What calls[i]() returned in thread i, which makes it `times` times with nothing in between."""
    start, got = threading.Barrier(len(calls)), [None] * len(calls)

    def run(i):
        call, seen = calls[i], set()
        start.wait()
        for _ in range(times):
            seen.add(call())
        got[i] = seen

    pool = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in pool:
        t.start()
    for t in pool:
        t.join()
    torch.cuda.synchronize()
    return got


def bound(fn, *args):
    """fn with its arguments converted once, so that a thread's calls follow one another closely."""
    converted = [a if t is ctypes.c_void_p and a is None else t(a) for t, a in zip(fn.argtypes, args)]
    return lambda: fn(*converted)


# two widths that one kernel serves: two tiles a warp, one, rows that begin anywhere
@pytest.mark.parametrize("dtype,widths", [(B, (4096, 8192)), (F, (2816, 4096)), (B, (4095, 8191))])
def test_norms_of_two_widths(z, dtype, widths):
    rows, code = 4, z.BF16 if dtype == B else z.F32
    keep, forward, backward = [], [], []
    for i in range(8):
        hidden, stream = widths[i % 2], torch.cuda.Stream()
        n = z.ResidualNorm(hidden, eps=1e-5)
        x = torch.randn(rows, hidden, device="cuda").to(dtype)
        h, gx = torch.empty_like(x), torch.empty_like(x)
        ws = torch.empty(z.zccl_residual_norm_workspace_bytes(hidden, rows), dtype=torch.uint8, device="cuda")
        keep.append((n, x, h, gx, ws, stream))
        forward.append(bound(z.lib().zccl_residual_norm, ctypes.addressof(n.config), x.data_ptr(), code, hidden, None, code, 0,
                             None, None, z.F32, None, z.F32, 0, 1, rows, 0, None, None, h.data_ptr(), n.status.data_ptr(),
                             stream.cuda_stream))
        backward.append(bound(z.lib().zccl_residual_norm_backward, ctypes.addressof(n.config), None, 0, x.data_ptr(), hidden,
                              x.data_ptr(), code, hidden, None, code, 0, None, None, z.F32, None, z.F32, 0, 1, rows, 0, None,
                              gx.data_ptr(), None, None, None, None, ws.data_ptr(), ws.numel(), n.status.data_ptr(),
                              stream.cuda_stream))
    torch.cuda.synchronize()
    for calls in (forward, backward):
        assert statuses(calls, 3000) == [{z.OK}] * 8
    for n, x, h, gx, ws, _ in keep:
        assert torch.equal(h, n.norm(x)) and torch.equal(gx, n.norm_backward(x, x)[0])
        n.check_status()


def test_compressions_of_few_and_many_segments(z):
    keep, calls = [], []
    lut = z.zccl_lut_from_sigma(1.0)
    for i in range(4):
        count, n, stream = (1, 3000)[i % 2], 40, torch.cuda.Stream()
        codec = z.Codec()
        x = torch.randn(count, n, device="cuda").to(B).view(torch.int16)
        outs = torch.zeros(count, z.zccl_max_compressed_bytes(n), dtype=torch.uint8, device="cuda")
        table = codec.segment_table(list(zip(x, outs)))
        sizes = codec.compress_batched(list(zip(x, outs)), lut, table=table)
        torch.cuda.synchronize()
        want, again = (outs.clone(), sizes.clone()), torch.zeros_like(sizes)
        outs.zero_()
        ws, nbytes = codec.workspace(0)
        buffer = ctypes.create_string_buffer(lut, 7)
        keep.append((codec, x, outs, table, again, want, buffer))
        calls.append(bound(z.lib().zccl_compress_batched, table.data_ptr(), count, count * n, ctypes.addressof(buffer),
                           again.data_ptr(), ws, nbytes, codec.status.data_ptr(), stream.cuda_stream))
    assert statuses(calls, 500) == [{z.OK}] * 4
    for codec, _, outs, _, sizes, want, _ in keep:
        assert codec.read_status() == z.OK and torch.equal(sizes, want[1]) and torch.equal(outs, want[0])


@pytest.mark.parametrize("own", [False, True])
def test_reductions_of_few_and_many_shards(z, own):
    """own: with a plain shard of the rank's own."""
    keep, calls = [], []
    lut, n = z.zccl_lut_from_sigma(1.0), 40
    codec = z.Codec()
    x = torch.randn(n, device="cuda").to(B).view(torch.int16)
    one, size = codec.compress(x, lut)
    for i in range(4):
        count, stream, codec = (2, 1000)[i % 2], torch.cuda.Stream(), z.Codec()
        streams, sizes = [one] * count, [int(size)] * count
        want = (codec.decompress_reduce_local(streams, sizes, n, local=x, local_pos=1) if own else
                codec.decompress_reduce(streams, sizes, n)).clone()
        ptrs, lengths = (torch.tensor(v, dtype=torch.int64, device="cuda") for v in ([one.data_ptr()] * count, sizes))
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        ws, nbytes = codec.workspace(0)
        tail = (out.data_ptr(), n, ws, nbytes, codec.status.data_ptr(), stream.cuda_stream)
        keep.append((codec, ptrs, lengths, out, want))
        calls.append(bound(z.lib().zccl_decompress_reduce_local, ptrs.data_ptr(), lengths.data_ptr(), count, x.data_ptr(), 1, 0,
                           *tail) if own else
                     bound(z.lib().zccl_decompress_reduce, ptrs.data_ptr(), lengths.data_ptr(), count, *tail))
    assert statuses(calls, 500) == [{z.OK}] * 4
    for codec, _, _, out, want in keep:
        assert codec.read_status() == z.OK and torch.equal(out, want)
