"""Calls of one C entry point from several host threads at once, each on its own
stream and buffers (needs a B200). ctypes lets go of the interpreter lock during
a call, so the calls' host sides really overlap."""
import ctypes
import threading

import pytest
import torch

from mixture_experts_layer_limited_b200 import native as N

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
U8 = dict(dtype=torch.uint8, device=DEV)


def _at_once(fn, calls, n=10000):
    """Runs fn on each argument list of `calls` n times, a thread and a stream
    (the last argument) each: the statuses other than MOE_OK."""
    bad, start = [], threading.Barrier(len(calls))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def work(args, stream):
        torch.cuda.set_device(0)
        args = (*args, stream.cuda_stream)
        start.wait()
        for _ in range(n):
            status = fn(*args)
            if status != N.MOE_OK:
                bad.append((status, N.load_library().moe_last_cuda_error()))
    threads = [threading.Thread(target=work, args=a) for a in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


def test_4bit_products_of_different_tiles():
    """Decode-like calls (tiles of 32 rows) beside prefill-like ones (192): they
    take different amounts of shared memory from the same kernel."""
    H, I = 256, 128
    lib = N.load_library()
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    code = lambda *s: torch.randint(0, 256, s, generator=g, device=DEV, dtype=torch.uint8)
    w2, w2s = code(H, I // 2), torch.full((H // 128, I // 128, 512), 127, **U8)
    w = N.FFNWeights(None, w2.data_ptr(), None, w2s.data_ptr(), N.MOE_MXFP4, 1, I)
    w.tiled = 0
    calls, keep = [], []
    for rows in (1, 200, 2, 300):
        h, hs, out = code(rows, I // 2), torch.full((I // 128, rows, 4), 127, **U8), torch.empty(rows, H, dtype=BF, device=DEV)
        args = (rows, H, ctypes.byref(w), h.data_ptr(), hs.data_ptr(), None, None, out.data_ptr(), None)
        assert lib.moe_down_proj(*args, None) == N.MOE_OK
        torch.cuda.synchronize()
        calls.append(args)
        keep.append((out, out.clone(), h, hs))
    assert not _at_once(lib.moe_down_proj, calls)
    for out, want, _, _ in keep:
        assert torch.equal(out, want)
