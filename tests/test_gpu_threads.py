"""cache_attend from host threads at once, with numbers of requests whose shared memory differs: each call gets what it
asks for, whatever the other's asked for in between."""
import ctypes as C
import sys
import threading

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_draft_round_gb300 as ds

pytestmark = pytest.mark.gpu
DEV = "cuda"
CALLS = 2000


def _call(R, max_q, dtype, D):
    """A call for R requests, one row of the first and the last each, over two pages that all requests share."""
    i32 = dict(dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(R)
    pool = ds.cache_pool(2, 1, 16, D)
    at = torch.arange(32, **i32)
    kv = torch.randn((2, 32, 1, D), device=DEV, generator=g)
    ds.cache_append(kv[0], kv[1], pool, torch.arange(2, **i32)[None], torch.zeros_like(at), at, torch.zeros(1, **i32))
    table = torch.arange(2, **i32).repeat(R, 1)
    offsets = torch.ones(R + 1, **i32)
    offsets[0], offsets[R] = 0, 2
    q = torch.randn((2, 1, D), device=DEV, generator=g).to(dtype)
    ctx = torch.full((R,), 20, **i32)
    if R == 1:
        offsets = torch.tensor([0, 2], **i32)
    a, out = ds.cache_attend_args(q, pool, table, offsets, ctx, max_q=max_q)
    ws = torch.zeros(ds.workspace_bytes("cache_attend", a), dtype=torch.uint8, device=DEV)
    run, args = ds.lib().dspark_cache_attend, (C.byref(a), ws.data_ptr(), ws.numel())
    keep = (a, q, pool, table, offsets, ctx)
    return lambda stream, keep=keep: run(*args, stream), out, ws


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_q,dtype,R", [(2, torch.float32, 8192), (16, torch.bfloat16, 8192), (512, torch.bfloat16, 7000)])
def test_threads_with_different_numbers_of_requests(max_q, dtype, R, D):
    ds.lib()
    calls = [_call(n, max_q, dtype, D) for n in (R, 1) * 3]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    start, codes = threading.Barrier(len(calls)), [None] * len(calls)

    def run(i):
        call, s = calls[i][0], streams[i].cuda_stream
        start.wait()
        codes[i] = {call(s) for _ in range(CALLS)}
        streams[i].synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert codes == [{0}] * len(calls)
    for call, out, ws in calls:
        assert ds.check(ws) == 0
        got = {n: t.clone() for n, t in out.items()}
        assert call(torch.cuda.current_stream().cuda_stream) == 0
        for n in got:
            assert torch.equal(got[n], out[n]) and torch.isfinite(got[n]).all()
