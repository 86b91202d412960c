"""The wait limit bounds each wait of the attention kernel of many rows, not the time the kernel takes."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_draft_round_gb300 as ds

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def long_call():
    """A call of some 10 ms whose single waits take 0.2 ms at most: 2048 requests of 16 rows over 8192 keys, in pages they
    share. Returns the call, its outputs and its time in ns."""
    ds.lib()
    R, Q, Hq, Hkv, D, page, ctx, n_pages = 2048, 16, 32, 8, 64, 64, 8176, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    i32 = dict(dtype=torch.int32, device=DEV)
    pool = ds.cache_pool(n_pages, Hkv, page, D)
    at = torch.arange(n_pages * page, **i32)
    kv = torch.randn((2, n_pages * page, Hkv, D), device=DEV, generator=g)
    ds.cache_append(kv[0], kv[1], pool, torch.arange(n_pages, **i32)[None], torch.zeros_like(at), at, torch.zeros(1, **i32))
    table = torch.randint(0, n_pages, (R, (ctx + Q) // page), generator=g, **i32)
    q = torch.randn((R * Q, Hq, D), device=DEV, generator=g).bfloat16()
    args = (q, pool, table, torch.arange(R + 1, **i32) * Q, torch.full((R,), ctx, **i32))

    def call():
        out = ds.cache_attend(*args, max_q=Q)
        return out, ds.check(out["workspace"])

    call()
    timer = ds.KernelTimer("cache_attend", 1)
    with timer:
        out, code = call()
    assert code == 0
    return call, out, int(timer.durations_ms()[0] * 1e6)


@pytest.fixture(autouse=True)
def _limit():
    yield
    ds.set_wait_limit(0)


def _equal(a, b):
    return all(torch.equal(a[n], b[n]) for n in ("out", "lse"))


def test_a_limit_below_the_kernels_time_ends_nothing(long_call):
    call, want, ns = long_call
    assert ns > 6_000_000
    ds.set_wait_limit(ns // 6)
    for _ in range(3):
        out, code = call()
        assert code == 0 and _equal(out, want)


@pytest.mark.parametrize("limit", [(1 << 62) - 1, 1 << 62, 1 << 63, (1 << 64) - 1])
def test_a_limit_near_the_largest_number(long_call, limit):
    call, want, _ = long_call
    ds.set_wait_limit(limit)
    out, code = call()
    assert code == 0 and _equal(out, want)
