"""The target layer's attention on the GPU against the 64-bit reference of layer_ref.py: head norms with
rotation, the 4-bit cache's rows, attention over the cache, their error paths, and the calls together."""
import math

import numpy as np
import pytest
import torch

import layer_ref as ref
import speculative_decoding_draft_round_gb300 as ds

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # relative, of one rounding


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    ds.lib()


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ norms and rotation

def _rope_case(T, Hq, Hkv, D, rot, dtype, inter, norm, gains, far, pad=0, shift=0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    width = (Hq + 2 * Hkv) * D + pad
    rows = (torch.randn((T, width + shift), device=DEV, generator=g) * 3).to(TYPES[dtype])[:, shift:]
    q = rows[:, :Hq * D].unflatten(1, (Hq, D))
    k = rows[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    gq = 1 + 0.2 * torch.randn(D, device=DEV, generator=g) if gains else None
    gk = 1 + 0.2 * torch.randn(D, device=DEV, generator=g) if gains else None
    R = 3
    ctx = rng.integers(0, far, R)
    request = rng.integers(-1, R, T)
    request[0] = 0
    position = rng.integers(0, 33, T)
    freq = ds.rope_frequencies(rot) if rot else None
    out = ds.qk_norm_rope(q, k, freq, _i32(position), request=_i32(request), ctx_len=_i32(ctx), q_gain=gq, k_gain=gk,
                          eps=1e-5, norm=norm, interleaved=inter)
    assert ds.check(out["workspace"]) == 0
    pos = np.where(request < 0, 0, ctx[request.clip(0)] + position)
    f = [int(x) % (1 << 64) for x in freq.tolist()] if rot else []
    for name, x, gain in (("q", q, gq), ("k", k, gk)):
        want = ref.norm_rope(_f64(x), None if gain is None else _f64(gain), pos, f, norm, 1e-5, inter)
        want[request < 0] = 0
        got = _f64(out[name])
        # the norm's sum (D terms, then root and quotient), gain, the sine and cosine of an angle off by
        # 2^-25 of half a turn, two products and their sum: counted against the row's largest value
        y = np.abs(want).max(-1, keepdims=True)
        tol = (D / 2 + 24) * 2.0 ** -24 * 2 * y + HALF_STEP[dtype] * np.abs(want)
        assert np.all(np.abs(got - want) <= tol), (name, np.max(np.abs(got - want) - tol))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [(1, 1, 1, 2, 2), (5, 3, 1, 32, 16), (7, 4, 2, 64, 64), (9, 5, 5, 96, 48),
                                            (6, 8, 2, 128, 128), (33, 2, 1, 128, 64), (3, 2, 2, 256, 256),
                                            (4, 3, 1, 80, 20), (2, 1, 1, 1024, 1024), (5, 40, 8, 128, 128)])
def test_norm_and_rotation(T, Hq, Hkv, D, rot, inter, dtype):
    _rope_case(T, Hq, Hkv, D, rot, dtype, inter, True, True, 4096, seed=T + D)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kw", [dict(norm=False, gains=False), dict(norm=False, gains=True), dict(gains=False),
                                dict(rot=0), dict(far=1 << 30), dict(pad=3), dict(shift=1), dict(shift=5, pad=1)])
def test_norm_and_rotation_options(kw, dtype):
    base = dict(rot=128, norm=True, gains=True, far=1000, pad=0, shift=0)
    base.update(kw)
    _rope_case(6, 4, 2, 128, base["rot"], dtype, False, base["norm"], base["gains"], base["far"], base["pad"],
               base["shift"], seed=11)


def test_rotation_without_requests_and_with_bad_ones():
    q, k = torch.randn((4, 2, 64), device=DEV), torch.randn((4, 1, 64), device=DEV)
    f = ds.rope_frequencies(64)
    pos = _i32([0, 5, -3, 2147483647])
    out = ds.qk_norm_rope(q, k, f, pos)
    assert ds.check(out["workspace"]) == 0
    want = ref.norm_rope(_f64(q), None, pos.tolist(), f.tolist(), True, 1e-6, False)
    assert np.max(np.abs(_f64(out["q"]) - want)) < 64 * 2.0 ** -24 * 2 * np.abs(want).max()
    out = ds.qk_norm_rope(q, k, f, pos, request=_i32([0, 1, 2, 0]), ctx_len=_i32([0, 0]))
    assert ds.check(out["workspace"]) == ds.ERR_DEVICE_INPUT
    assert not out["q"][2].any() and out["q"][1].any()


def test_norm_of_zeros_nan_and_nothing():
    f = ds.rope_frequencies(64)
    q = torch.zeros((3, 2, 64), device=DEV, dtype=torch.bfloat16)
    q[1, 0, 7] = float("nan")
    q[2, 1] = 1.0
    out = ds.qk_norm_rope(q, q[:, :1], f, _i32([0, 1, 0]))
    assert not out["q"][0].any() and torch.isnan(out["q"][1, 0]).all() and not out["q"][1, 1].any()
    assert torch.all(out["q"][2, 1] == 1.0)
    out = ds.qk_norm_rope(q[:0], q[:0, :1], f, _i32([]))
    assert out["q"].shape == (0, 2, 64)


# ------------------------------------------------------------------ rows into the cache and back

def _pages(ctx, each, page, seed, spare=0):
    """A table of scattered pages for each request's ctx + each tokens; -1 elsewhere."""
    rng = np.random.default_rng(seed)
    R = len(ctx)
    need = [-(-(c + n) // page) for c, n in zip(ctx, each)]
    width = max(1, max(need)) + spare
    ids = rng.permutation(R * width)
    table = np.full((R, width), -1, np.int64)
    for r in range(R):
        table[r, :need[r]] = ids[r * width:r * width + need[r]]
    return table, R * width


def _flat(each, tail=0):
    request = np.concatenate([np.full(n, r) for r, n in enumerate(each)] + [np.full(tail, -1)]).astype(np.int64)
    position = np.concatenate([np.arange(n) for n in each] + [np.full(tail, -1)]).astype(np.int64)
    offsets = np.concatenate([[0], np.cumsum(each)])
    return request, position, offsets


def _blocks(pool):
    return pool.cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 48, 256])
@pytest.mark.parametrize("D,Hkv", [(32, 3), (64, 1), (96, 2), (128, 4), (256, 2)])
def test_append_and_read_are_exact(D, Hkv, page, dtype):
    ctx, each = [0, 15, 37, 300], [1, 33, 0, 17]
    table, n_pages = _pages(ctx, each, page, D + page)
    request, position, _ = _flat(each, tail=3)
    T = len(request)
    g = torch.Generator(device=DEV).manual_seed(D)
    rows = torch.randn((T, 2 * Hkv * D), device=DEV, generator=g)
    rows = rows * torch.exp(torch.empty((T, 1), device=DEV).uniform_(-12, 12, generator=g))
    rows[0] = 0
    rows[1, :40] = 1e-30                                     # a scale that becomes 0
    rows[2, :32] = torch.arange(32, device=DEV) * 0.5 - 7   # ties
    rows[3, :32] = 1e9                                       # above what the cache holds
    rows = rows.to(TYPES[dtype])
    k, v = rows[:, :Hkv * D].unflatten(1, (Hkv, D)), rows[:, Hkv * D:].unflatten(1, (Hkv, D))
    pool = ds.cache_pool(n_pages, Hkv, page, D)
    pool.fill_(0xA5)
    where = (pool, _i32(table), _i32(request), _i32(position), _i32(ctx))
    out = ds.cache_append(k, v, *where)
    assert ds.check(out["workspace"]) == 0
    blocks = _blocks(pool)
    touched = np.zeros(n_pages, bool)
    for t in range(T):
        if request[t] < 0:
            continue
        at = ctx[request[t]] + position[t]
        pg = table[request[t], at // page]
        touched[pg] = True
        for h in range(Hkv):
            for half, x in ((0, k), (1, v)):
                got = ref.block_row(blocks[pg, h], at % page, page, D, half)
                np.testing.assert_array_equal(got, ref.stored(x[t, h].float().cpu().numpy()))
    assert np.all(blocks[~touched] == 0xA5)                  # nothing else is written
    for dt in ("f32", "bf16"):
        back = ds.cache_read(*where, D=D, dtype=TYPES[dt])
        assert ds.check(back["workspace"]) == 0
        for name, x in (("k", k), ("v", v)):
            want = torch.as_tensor(ref.stored(x.float().cpu().numpy())).float().to(TYPES[dt])
            want[request < 0] = 0
            assert torch.equal(back[name].cpu(), want)


def test_append_leaves_the_neighbours():
    """One token into the middle of a page that others filled."""
    D, Hkv, page = 64, 2, 32
    pool = ds.cache_pool(1, Hkv, page, D)
    table, ctx = _i32([[0]]), _i32([0])
    k = torch.randn((page, Hkv, D), device=DEV)
    v = torch.randn((page, Hkv, D), device=DEV)
    all_ = (_i32(np.zeros(page)), _i32(np.arange(page)), ctx)
    ds.cache_append(k, v, pool, table, *all_)
    before = ds.cache_read(pool, table, *all_, D=D, dtype=torch.float32)
    k2, v2 = torch.randn((1, Hkv, D), device=DEV), torch.randn((1, Hkv, D), device=DEV)
    ds.cache_append(k2, v2, pool, table, _i32([0]), _i32([13]), ctx)
    after = ds.cache_read(pool, table, *all_, D=D, dtype=torch.float32)
    keep = np.arange(page) != 13
    for n in ("k", "v"):
        assert torch.equal(after[n].cpu()[keep], before[n].cpu()[keep])
        assert not torch.equal(after[n][13], before[n][13])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_takes_any_strides(dtype):
    """Rows off 16-byte boundaries, a head axis that is not the inner one, heads that share a row."""
    D, page, T = 64, 16, 9
    table, ctx = _i32([[0]]), _i32([2])
    where = (table, _i32(np.zeros(T)), _i32(np.arange(T)), ctx)
    base = torch.randn((3, T, D + 1), device=DEV).to(TYPES[dtype])
    for view in (base[:, :, 1:].permute(1, 0, 2), base[:1, :, :D].permute(1, 0, 2).expand(T, 3, D),
                 base[:, :, :D].permute(1, 0, 2)):
        a, b = ds.cache_pool(1, 3, page, D), ds.cache_pool(1, 3, page, D)
        ds.cache_append(view, view, a, *where)
        ds.cache_append(view.contiguous(), view.contiguous(), b, *where)
        assert torch.equal(a, b)


def test_append_and_read_out_of_range():
    D, Hkv, page = 32, 1, 16
    pool = ds.cache_pool(2, Hkv, page, D)
    table, ctx = _i32([[0, 7], [1, -1], [1, 1]]), _i32([0, 3, -5])
    request = _i32([0, 0, 1, 1, 3, 2, -1, 0, 0])
    position = _i32([0, 16, 0, 13, 0, 6, 0, 32, -1])   # good, page 7, good, page -1, no request, ctx < 0, pad, past, negative
    k = torch.ones((9, Hkv, D), device=DEV)
    for t in range(9):
        out = ds.cache_append(k[t:t + 1], k[t:t + 1], pool, table, request[t:t + 1], position[t:t + 1], ctx)
        assert ds.check(out["workspace"]) == (0 if t in (0, 2, 6) else ds.ERR_DEVICE_INPUT), t
    out = ds.cache_read(pool, table, request, position, ctx, D=D, dtype=torch.float32)
    assert ds.check(out["workspace"]) == ds.ERR_DEVICE_INPUT
    want = torch.as_tensor(ref.stored(np.ones((1, D), np.float32))).float()
    for t in range(9):
        assert torch.equal(out["k"][t].cpu(), want if t in (0, 2) else torch.zeros((1, D))), t


def test_append_nonfinite():
    D, page = 64, 16
    pool = ds.cache_pool(1, 1, page, D)
    k = torch.linspace(-2, 2, D, device=DEV).view(1, 1, D).clone()
    k[0, 0, 3], k[0, 0, 40], k[0, 0, 41] = float("nan"), float("inf"), -float("inf")
    where = (pool, _i32([[0]]), _i32([0]), _i32([0]), _i32([0]))
    out = ds.cache_append(k, k, *where)
    assert ds.check(out["workspace"]) == ds.ERR_NONFINITE_INPUT
    x = k.cpu().numpy().copy()
    x[0, 0, 3] = x[0, 0, 40] = x[0, 0, 41] = 0
    want = ref.stored(x)
    s = ref.scales_of(x)[0, 0, 1]
    want[0, 0, 40], want[0, 0, 41] = 7 * s, -7 * s
    np.testing.assert_array_equal(_f64(ds.cache_read(*where, D=D, dtype=torch.float32)["k"]), want)


# ------------------------------------------------------------------ attention

def _filled(ctx, each, page, Hkv, D, seed, spread=1.0):
    """A pool filled through cache_append, and the values it holds by request."""
    table, n_pages = _pages(ctx, each, page, seed, spare=1)
    pool = ds.cache_pool(n_pages, Hkv, page, D)
    pool.fill_(0xFF)                                  # what no token wrote must not be read: scales of NaN
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = [c + e for c, e in zip(ctx, each)]
    request, position, _ = _flat(n)
    zero = _i32(np.zeros(len(ctx)))
    k = torch.randn((len(request), Hkv, D), device=DEV, generator=g) * spread
    v = torch.randn((len(request), Hkv, D), device=DEV, generator=g)
    where = (pool, _i32(table), _i32(request), _i32(position), zero)
    ds.cache_append(k, v, *where)
    got = ds.cache_read(*where, D=D, dtype=torch.float32)
    edge = np.concatenate([[0], np.cumsum(n)])
    keys = [_f64(got["k"][edge[r]:edge[r + 1]]) for r in range(len(n))]
    values = [_f64(got["v"][edge[r]:edge[r + 1]]) for r in range(len(n))]
    return pool, table, keys, values


def _check_attend(out, lse, want, dtype, values, n_most):
    o, l, mag = want
    live = np.isfinite(l)
    assert np.array_equal(np.isfinite(lse), live) and not out[~live].any()
    vmax = max([np.abs(v).max() for v in values if v.size] or [0.0])
    # a product of D terms off by (D + 8) 2^-24 of its largest sum, which moves a weight by as much; a weight
    # rounded to fp16 (2^-11) for bf16 rows, to two fp16 terms (2^-22) for fp32 ones; the sums of up to n_most
    # terms, added 16 at a time in a tensor core or one at a time, 2^-23 each; one rounding at the end
    D = out.shape[-1]
    z = (D + 8) * 2.0 ** -23 * mag + 2.0 ** -20
    weight = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
    tol = (2 * (z + weight) + (math.sqrt(n_most) + 16) * 2.0 ** -23)[..., None] * vmax + HALF_STEP[dtype] * np.abs(o)
    err = np.abs(out - o)
    assert np.all(err <= tol), ("out", float((err / tol).max()), np.unravel_index(np.argmax(err / tol), err.shape))
    ltol = z + (math.sqrt(n_most) + 16) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(live, l, 0))
    lerr = np.abs(np.where(live, lse - np.where(live, l, 0), 0))
    assert np.all(lerr <= ltol), ("lse", float((lerr / ltol).max()))


def _attend_case(ctx, each, Hq, Hkv, D, page, dtype, window=0, sinks=0, path=ds.PATH_AUTO, seed=0, tail=2, spread=1.0,
                 scale=None, max_q=None):
    pool, table, keys, values = _filled(ctx, each, page, Hkv, D, seed, spread)
    _, _, offsets = _flat(each)
    T = int(offsets[-1]) + tail
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    q = torch.randn((T, Hq, D), device=DEV, generator=g).to(TYPES[dtype])
    out = ds.cache_attend(q, pool, _i32(table), _i32(offsets), _i32(ctx), window=window, sinks=sinks, path=path,
                          scale=scale, max_q=max_q or max(1, max(each)))
    assert ds.check(out["workspace"]) == 0
    sc = scale or 1 / math.sqrt(D)
    want = ref.attend(_f64(q), keys, values, ctx, offsets, sc, window, sinks)
    _check_attend(_f64(out["out"]), _f64(out["lse"]), want, dtype, values, max(c + e for c, e in zip(ctx, each)))
    return q, pool, table, offsets, out


PATHS = {"auto": ds.PATH_AUTO, "cuda": ds.PATH_CUDA_CORE}


@pytest.mark.parametrize("path", sorted(PATHS))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (64, 8, 2), (128, 8, 1), (128, 5, 1), (32, 2, 1), (96, 6, 2),
                                      (256, 2, 1), (128, 40, 8)])
def test_attend_heads(D, Hq, Hkv, dtype, path):
    _attend_case([0, 1, 15, 16, 63, 64, 65, 200], [1, 2, 1, 3, 1, 1, 5, 2], Hq, Hkv, D, 16, dtype, path=PATHS[path],
                 seed=D + Hq)


@pytest.mark.parametrize("path", sorted(PATHS))
@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 256])
def test_attend_pages(page, path):
    _attend_case([0, page - 1, page, 3 * page + 7, 500], [17, 1, 9, 2, 17], 8, 2, 128, page, "bf16", path=PATHS[path],
                 seed=page)


@pytest.mark.parametrize("path", sorted(PATHS))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 64), (64, 0), (100, 3), (128, 130),
                                          (4000, 5), (2147483647, 2147483647)])
def test_attend_window_and_sinks(window, sinks, dtype, path):
    _attend_case([0, 3, 100, 129, 700], [5, 9, 1, 17, 9], 4, 1, 64, 32, dtype, window, sinks, path=PATHS[path],
                 seed=window % 1000)


@pytest.mark.parametrize("path", sorted(PATHS))
@pytest.mark.parametrize("each", [[0, 0, 1], [0], [1, 0, 33], [33, 1, 0, 2], [64], [129, 0, 3]])
def test_attend_row_counts(each, path):
    _attend_case([40 * i for i in range(len(each))], each, 4, 2, 128, 16, "bf16", path=PATHS[path], seed=len(each))


@pytest.mark.parametrize("Q,ctx", [(300, 0), (257, 130), (700, 65)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_prompt(Q, ctx, window, sinks, D):
    _attend_case([ctx, 5], [Q, 1], 4, 2, D, 64, "bf16", window, sinks, seed=Q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_long_context(dtype):
    _attend_case([20011, 3], [1, 2], 4, 2, 64, 64, dtype, seed=5)
    _attend_case([9000], [3], 8, 1, 128, 16, dtype, window=5000, sinks=70, seed=6)


@pytest.mark.parametrize("path", sorted(PATHS))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("spread,scale", [(100.0, None), (1e-3, 1.0), (1.0, 30.0)])
def test_attend_sharp_and_flat_weights(spread, scale, dtype, path):
    """Scores far apart (one weight is 1) and all alike; the bound grows with the products."""
    _attend_case([70, 300], [3, 5], 4, 2, 64, 16, dtype, path=PATHS[path], spread=spread, scale=scale, seed=8)


@pytest.mark.parametrize("path", sorted(PATHS))
def test_attend_many_requests(path):
    rng = np.random.default_rng(0)
    R = 300
    ctx, each = rng.integers(0, 90, R).tolist(), rng.integers(0, 4, R).tolist()
    _attend_case(ctx, each, 2, 1, 64, 16, "bf16", path=PATHS[path], seed=9)


@pytest.mark.parametrize("path", sorted(PATHS))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_large_and_small_queries(dtype, path):
    """Rows whose magnitude no fp16 holds: the products are scaled, not the result."""
    ctx, each, D = [50], [3], 64
    pool, table, keys, values = _filled(ctx, each, 16, 1, D, 3)
    q = torch.randn((3, 2, D), device=DEV)
    q[0] *= 1e6
    q[1] *= 1e-9
    q[2] = 0
    q = q.to(TYPES[dtype])
    offsets = [0, 3]
    out = ds.cache_attend(q, pool, _i32(table), _i32(offsets), _i32(ctx), max_q=3, path=PATHS[path], scale=1e-5)
    assert ds.check(out["workspace"]) == 0
    want = ref.attend(_f64(q), keys, values, ctx, offsets, 1e-5, 0, 0)
    _check_attend(_f64(out["out"]), _f64(out["lse"]), want, dtype, values, 53)


@pytest.mark.parametrize("path", sorted(PATHS))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attend_nonfinite_query(bad, dtype, path):
    ctx, each, D, Hq = [200, 9], [5, 1], 128, 4
    q, pool, table, offsets, ok = _attend_case(ctx, each, Hq, 2, D, 16, dtype, path=PATHS[path], seed=21)
    q[2, 1, 77] = bad
    out = ds.cache_attend(q, pool, _i32(table), _i32(offsets), _i32(ctx), max_q=5, path=PATHS[path])
    assert ds.check(out["workspace"]) == ds.ERR_NONFINITE_INPUT
    rest = torch.ones(q.shape[:2], dtype=torch.bool)
    rest[2, 1] = False
    assert torch.isnan(out["out"][2, 1]).all() and torch.isnan(out["lse"][2, 1])
    assert torch.equal(out["out"].cpu()[rest], ok["out"].cpu()[rest])
    assert torch.equal(out["lse"].cpu()[rest], ok["lse"].cpu()[rest])


@pytest.mark.parametrize("path", sorted(PATHS))
def test_attend_bad_pages_and_offsets(path):
    """Pages out of range hide their keys, all of them leave a row empty; counts past max_q end there."""
    ctx, each, D, page = [40, 10, 0], [2, 1, 1], 64, 16
    pool, table, keys, values = _filled(ctx, each, page, 1, D, 31)
    _, _, offsets = _flat(each)
    q = torch.randn((4, 2, D), device=DEV).bfloat16()
    bad = table.copy()
    bad[0, 1] = pool.shape[0]          # tokens 16 .. 31 of request 0
    bad[1, :] = -1                     # all of request 1
    out = ds.cache_attend(q, pool, _i32(bad), _i32(offsets), _i32(ctx), max_q=2, path=PATHS[path])
    assert ds.check(out["workspace"]) == ds.ERR_DEVICE_INPUT
    assert not out["out"][2].any() and torch.all(out["lse"][2] == -math.inf)
    gone = np.r_[0:16, 32:42]
    for j in range(2):                 # request 0 without its second page
        k = [keys[0][gone[gone <= 40 + j]]]
        v = [values[0][gone[gone <= 40 + j]]]
        w = ref.attend(_f64(q[j:j + 1]), k, v, [k[0].shape[0] - 1], [0, 1], 1 / 8, 0, 0)
        _check_attend(_f64(out["out"][j:j + 1]), _f64(out["lse"][j:j + 1]), w, "bf16", v, 42)
    # one row of request 0 only; and offsets that decrease
    short = ds.cache_attend(q, pool, _i32(table), _i32(offsets), _i32(ctx), max_q=1, path=PATHS[path])
    assert ds.check(short["workspace"]) == ds.ERR_DEVICE_INPUT
    full = ds.cache_attend(q, pool, _i32(table), _i32(offsets), _i32(ctx), max_q=2, path=PATHS[path])
    assert ds.check(full["workspace"]) == 0
    assert torch.equal(short["out"][[0, 2, 3]], full["out"][[0, 2, 3]])
    odd = ds.cache_attend(q, pool, _i32(table), _i32([0, 2, 1, 4]), _i32(ctx), max_q=4, path=PATHS[path])
    assert ds.check(odd["workspace"]) == ds.ERR_DEVICE_INPUT
    neg = ds.cache_attend(q, pool, _i32(table), _i32(offsets), _i32([-1, 10, 0]), max_q=2, path=PATHS[path])
    assert ds.check(neg["workspace"]) == ds.ERR_DEVICE_INPUT
    assert torch.equal(neg["out"][2:], full["out"][2:])


@pytest.mark.parametrize("path", sorted(PATHS))
def test_attend_is_the_same_every_time_and_on_another_stream(path):
    ctx, each = [3000, 17, 900], [9, 2, 9]
    q, pool, table, offsets, a = _attend_case(ctx, each, 8, 2, 128, 32, "bf16", path=PATHS[path], seed=41)
    args = (pool, _i32(table), _i32(offsets), _i32(ctx))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = ds.cache_attend(q, *args, max_q=9, path=PATHS[path], stream=s)
    c = ds.cache_attend(q, *args, max_q=9, path=PATHS[path])
    torch.cuda.synchronize()
    for n in ("out", "lse"):
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n])


def test_attend_takes_any_strides_and_no_lse():
    ctx, each = [100, 30], [3, 2]
    q, pool, table, offsets, a = _attend_case(ctx, each, 4, 2, 64, 16, "bf16", seed=51, tail=0)
    args = (pool, _i32(table), _i32(offsets), _i32(ctx))
    odd = torch.zeros((4, 5, 67), device=DEV, dtype=torch.bfloat16)[:, :, 3:].permute(1, 0, 2)
    odd.copy_(q)
    b = ds.cache_attend(odd, *args, max_q=3, lse=False)
    assert "lse" not in b and torch.equal(a["out"], b["out"])


# ------------------------------------------------------------------ together

def test_calls_captured_into_a_graph():
    """Norms, append and attention captured once and replayed on new inputs in the same buffers."""
    D, Hq, Hkv, page, ctx, each = 128, 8, 2, 32, [50, 7, 130], [5, 1, 9]
    pool, table, _, _ = _filled(ctx, each, page, Hkv, D, 61)
    request, position, offsets = _flat(each, tail=1)
    T = len(request)
    rows = torch.empty((T, (Hq + 2 * Hkv) * D), device=DEV, dtype=torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split([Hq * D, Hkv * D, Hkv * D], 1))
    f = ds.rope_frequencies(D)
    tb, rq, ps, of, cx = _i32(table), _i32(request), _i32(position), _i32(offsets), _i32(ctx)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    o1 = {"q": torch.empty((T, Hq, D), device=DEV, dtype=torch.bfloat16),
          "k": torch.empty((T, Hkv, D), device=DEV, dtype=torch.bfloat16)}
    o2 = {"out": torch.empty((T, Hq, D), device=DEV, dtype=torch.bfloat16),
          "lse": torch.empty((T, Hq), device=DEV)}

    def layer():
        ds.qk_norm_rope(q, k, f, ps, request=rq, ctx_len=cx, out=o1, workspace=ws)
        ds.cache_append(o1["k"], v, pool, tb, rq, ps, cx, workspace=ws)
        ds.cache_attend(o1["q"], pool, tb, of, cx, max_q=9, out=o2, workspace=ws)

    rows.normal_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for seed in (1, 2):
        rows.normal_(generator=torch.Generator(device=DEV).manual_seed(seed))
        layer()
        torch.cuda.synchronize()
        names = ("out", "lse")
        want = {n: o2[n].clone() for n in names}
        for n in names:
            o2[n].fill_(7)
        g.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(o2[n], want[n])
    assert ds.check(ws) == 0
