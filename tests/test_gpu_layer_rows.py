"""dspark_cache_attend where a request can have many rows (bf16, heads of 64 and 128: blocks of 128 rows), against the
formula in 64 bits: groups that divide no block, rows that end inside one, requests without rows between others with
many, windows, pages out of range, runs that cut a block's keys, other streams and a wait that runs out. The bound on
the outputs is the one of the other attention tests."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref
import speculative_decoding_draft_round_gb300 as ds
import test_gpu_layer as layer

pytestmark = pytest.mark.gpu
DEV = "cuda"
MAX_Q = 512   # rows that a request could have: so many that its calls take 128 rows at a time


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ds.lib()


def _case(ctx, each, Hq, Hkv, D, page, **kw):
    kw.setdefault("max_q", max(MAX_Q, max(each)))
    return layer._attend_case(ctx, each, Hq, Hkv, D, page, "bf16", **kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 2), (5, 1), (7, 1), (48, 1), (130, 1), (40, 8)])
def test_heads(Hq, Hkv, D):
    _case([0, 1, 127, 128, 200, 700], [1, 2, 1, 33, 5, 40], Hq, Hkv, D, 16, seed=D + Hq)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 112, 128, 256])
def test_pages(page):
    _case([0, page - 1, page, 3 * page + 7, 500], [65, 1, 9, 34, 17], 8, 2, 128, page, seed=page)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 64), (64, 0), (100, 3), (128, 130), (129, 1),
                                          (255, 256), (4000, 5), (2147483647, 2147483647)])
def test_window_and_sinks(window, sinks):
    _case([0, 3, 100, 129, 900], [5, 90, 1, 17, 33], 4, 1, 64, 32, window=window, sinks=sinks, seed=window % 1000)


@pytest.mark.parametrize("each", [[0, 0, 1], [0], [1, 0, 33], [33, 1, 0, 2], [64], [65], [129, 0, 3], [1], [31, 32, 33]])
def test_row_counts(each):
    _case([40 * i for i in range(len(each))], each, 4, 2, 128, 16, seed=len(each))


def test_one_request_among_empty_ones():
    each = [0] * 70
    each[0], each[33], each[69] = 2, 70, 1
    _case([5 * i for i in range(70)], each, 4, 2, 64, 16, seed=3)


def test_many_requests():
    rng = np.random.default_rng(1)
    R = 300
    _case(rng.integers(0, 400, R).tolist(), rng.integers(0, 6, R).tolist(), 4, 1, 64, 16, seed=9)


@pytest.mark.parametrize("R", [7679, 7680, 8100, 8192])
def test_as_many_requests_as_there_can_be(R):
    """Around the number whose places still fit shared memory, and the most the library takes."""
    each = np.zeros(R, dtype=int)
    each[::97] = 1
    each[R - 1], each[R // 2] = 3, 40
    _case((np.arange(R) % 23).tolist(), each.tolist(), 2, 1, 128, 16, seed=R)


def test_long_keys_of_one_request():
    """One item over every run: its parts are joined by the next kernel."""
    _case([20011, 3], [33, 2], 4, 2, 64, 64, seed=5)
    _case([9000], [5], 8, 1, 128, 16, window=5000, sinks=70, seed=6)


@pytest.mark.parametrize("spread,scale", [(100.0, None), (1e-3, 1.0), (1.0, 30.0)])
def test_sharp_and_flat_weights(spread, scale):
    """Maxima that rise from tile to tile by far more than a weight's range, and scores all alike."""
    _case([70, 700], [3, 35], 4, 2, 64, 16, spread=spread, scale=scale, seed=8)


@pytest.mark.parametrize("D", [64, 128])
def test_large_and_small_queries(D):
    ctx, each = [300], [3]
    pool, table, keys, values = layer._filled(ctx, each, 16, 1, D, 3)
    q = torch.randn((3, 2, D), device=DEV)
    q[0] *= 1e6
    q[1] *= 1e-9
    q[2] = 0
    q = q.bfloat16()
    out = ds.cache_attend(q, pool, layer._i32(table), layer._i32([0, 3]), layer._i32(ctx), max_q=MAX_Q, scale=1e-5)
    assert ds.check(out["workspace"]) == 0
    want = ref.attend(layer._f64(q), keys, values, ctx, [0, 3], 1e-5, 0, 0)
    layer._check_attend(layer._f64(out["out"]), layer._f64(out["lse"]), want, "bf16", values, 303)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nonfinite_query(bad):
    """The bad row alone is NaN, in a whole block as in one whose keys were cut."""
    ctx, each = [2000, 9], [37, 1]
    q, pool, table, offsets, ok = _case(ctx, each, 4, 2, 128, 16, seed=21)
    q[2, 1, 77] = bad
    q[37, 3, 0] = bad
    out = ds.cache_attend(q, pool, layer._i32(table), layer._i32(offsets), layer._i32(ctx), max_q=MAX_Q)
    assert ds.check(out["workspace"]) == ds.ERR_NONFINITE_INPUT
    rest = torch.ones(q.shape[:2], dtype=torch.bool)
    rest[2, 1] = rest[37, 3] = False
    for n in ("out", "lse"):
        assert torch.isnan(out[n][2, 1]).all() and torch.isnan(out[n][37, 3]).all()
        assert torch.equal(out[n].cpu()[rest], ok[n].cpu()[rest])


def test_bad_pages_and_offsets():
    """Pages out of range hide their keys, all of them leave a row empty; counts past max_q end there."""
    ctx, each, D, page = [40, 10, 0], [2, 1, 1], 64, 16
    pool, table, keys, values = layer._filled(ctx, each, page, 1, D, 31)
    offsets = [0, 2, 3, 4]
    q = torch.randn((4, 64, D), device=DEV).bfloat16()
    bad = table.copy()
    bad[0, 1] = pool.shape[0]          # tokens 16 .. 31 of request 0
    bad[1, :] = -1                     # all of request 1
    args = lambda t, o, c: (q, pool, layer._i32(t), layer._i32(o), layer._i32(c))
    out = ds.cache_attend(*args(bad, offsets, ctx), max_q=2)
    assert ds.check(out["workspace"]) == ds.ERR_DEVICE_INPUT
    assert not out["out"][2].any() and torch.all(out["lse"][2] == -math.inf)
    gone = np.r_[0:16, 32:42]
    for j in range(2):                 # request 0 without its second page
        k, v = ([x[0][gone[gone <= 40 + j]]] for x in (keys, values))
        w = ref.attend(layer._f64(q[j:j + 1]), k, v, [k[0].shape[0] - 1], [0, 1], 1 / 8, 0, 0)
        layer._check_attend(layer._f64(out["out"][j:j + 1]), layer._f64(out["lse"][j:j + 1]), w, "bf16", v, 42)
    full = ds.cache_attend(*args(table, offsets, ctx), max_q=3)
    assert ds.check(full["workspace"]) == 0
    short = ds.cache_attend(*args(table, [0, 2, 3, 4], ctx), max_q=2)
    assert ds.check(short["workspace"]) == 0
    assert torch.equal(short["out"], full["out"])
    odd = ds.cache_attend(*args(table, [0, 2, 1, 4], ctx), max_q=2)
    assert ds.check(odd["workspace"]) == ds.ERR_DEVICE_INPUT
    neg = ds.cache_attend(*args(table, offsets, [-1, 10, 0]), max_q=2)
    assert ds.check(neg["workspace"]) == ds.ERR_DEVICE_INPUT
    assert torch.equal(neg["out"][2:], full["out"][2:])


def test_rows_past_max_q_are_not_computed():
    ctx, each = [40, 10], [70, 2]
    q, pool, table, offsets, full = _case(ctx, each, 4, 2, 64, 16, seed=77)
    out = ds.cache_attend(q, pool, layer._i32(table), layer._i32(offsets), layer._i32(ctx), max_q=45)
    assert ds.check(out["workspace"]) == ds.ERR_DEVICE_INPUT
    rows = np.r_[0:45, 70:72]
    for n in ("out", "lse"):
        assert torch.equal(out[n][rows], full[n][rows])


def test_the_same_every_time_and_on_another_stream():
    ctx, each = [3000, 17, 900], [39, 2, 9]
    q, pool, table, offsets, a = _case(ctx, each, 8, 2, 128, 32, seed=41)
    args = (pool, layer._i32(table), layer._i32(offsets), layer._i32(ctx))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = ds.cache_attend(q, *args, max_q=MAX_Q, stream=s)
    c = ds.cache_attend(q, *args, max_q=MAX_Q)
    torch.cuda.synchronize()
    for n in ("out", "lse"):
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n])


@pytest.mark.parametrize("shift", [3, 8])
def test_any_strides_and_no_lse(shift):
    ctx, each = [100, 30], [23, 42]
    q, pool, table, offsets, a = _case(ctx, each, 4, 2, 64, 16, seed=51, tail=0)
    args = (pool, layer._i32(table), layer._i32(offsets), layer._i32(ctx))
    odd = torch.zeros((4, 65, 64 + shift), device=DEV, dtype=torch.bfloat16)[:, :, shift:].permute(1, 0, 2)
    odd.copy_(q)
    b = ds.cache_attend(odd, *args, max_q=MAX_Q, lse=False)
    assert "lse" not in b and torch.equal(a["out"], b["out"])


def test_a_wait_that_runs_out_records_a_timeout_and_the_next_call_recovers():
    ctx, each = [3000, 17], [39, 2]
    q, pool, table, offsets, a = _case(ctx, each, 8, 2, 128, 32, seed=43)
    args = (q, pool, layer._i32(table), layer._i32(offsets), layer._i32(ctx))
    codes = []
    old = ds.set_wait_limit(1)   # 1 ns: a wait that is not over at once runs out
    try:
        for _ in range(3):
            out = ds.cache_attend(*args, max_q=MAX_Q)
            codes.append(ds.check(out["workspace"]))
    finally:
        ds.set_wait_limit(0)
    assert old == 4_000_000_000
    assert ds.ERR_TIMEOUT in codes, codes
    again = ds.cache_attend(*args, max_q=MAX_Q)
    assert ds.check(again["workspace"]) == 0
    for n in ("out", "lse"):
        assert torch.equal(a[n], again[n])
