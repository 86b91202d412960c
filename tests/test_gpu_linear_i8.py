"""linear_i8 against whole numbers and 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import pass_ref as ref
import speculative_decoding_draft_round_gb300 as ds

pytestmark = pytest.mark.gpu
DEV = "cuda"
PATHS = [ds.PATH_AUTO, ds.PATH_CUDA_CORE]


def _case(T, K, N, seed=0, lo=-127, hi=128):
    rng = np.random.default_rng((seed, T, K, N))
    x, w = (rng.integers(lo, hi, s).astype(np.int8) for s in ((T, K), (N, K)))
    xs, ws = (np.exp(rng.standard_normal(n)).astype(np.float32) / 100 for n in (T, N))
    return x, xs, w, ws, rng.standard_normal(N).astype(np.float32)


def _dev(*a):
    return [torch.as_tensor(t, device=DEV) for t in a]


def _allowed(want, mag, most, K, bf16, path):
    # conversion of the sum, its two products with the scales (the second one with the bias' sum) and, where partial sums
    # can pass 2^24 outside the integers, 2^-23 of the largest for each 16 products
    part = 0.0 if path == ds.PATH_CUDA_CORE else np.where(most < 2 ** 24, 0.0, -(-K // 16) * 2.0 ** -23 * most)
    unit = np.where(most > 0, mag / np.maximum(most, 1), 0)
    return 4 * 2.0 ** -24 * mag + part * unit + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(want)


SHAPES = [(1, 1, 1), (1, 16, 1), (3, 5, 7), (2, 128, 128), (16, 64, 130), (17, 127, 256), (31, 129, 257), (33, 256, 300),
          (64, 512, 255), (65, 1000, 513), (128, 1024, 128), (191, 144, 640), (192, 1041, 256), (193, 160, 258),
          (200, 2048, 100), (385, 320, 1537), (129, 4096, 33), (7, 4097, 520), (20, 8192, 129), (600, 272, 1030)]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_against_whole_numbers(T, K, N, bf16, path):
    x, xs, w, ws, bias = _case(T, K, N)
    want, mag, most = ref.linear(x, xs, w, ws, bias)
    got = ds.linear_i8(*_dev(x, xs, w, ws), bias=torch.as_tensor(bias, device=DEV), path=path,
                       dtype=torch.bfloat16 if bf16 else torch.float32)
    assert ds.check(got["workspace"]) == 0
    out = got["out"].double().cpu().numpy()
    assert np.all(np.abs(out - want) <= _allowed(want, mag, most, K, bf16, path))


@pytest.mark.parametrize("path", PATHS)
def test_without_scales_the_sums_are_whole(path):
    """Partial sums below 2^24 lose nothing: the outputs are the sums themselves."""
    for T, K, N in ((40, 1024, 384), (130, 1030, 200), (300, 640, 515)):
        x, _, w, _, _ = _case(T, K, N, seed=1, lo=-128)
        one = lambda n: torch.ones(n, device=DEV)
        got = ds.linear_i8(*_dev(x), one(T), *_dev(w), one(N), path=path, dtype=torch.float32)["out"]
        assert np.array_equal(got.cpu().numpy().astype(np.int64), x.astype(np.int64) @ w.astype(np.int64).T)


@pytest.mark.parametrize("path", PATHS)
def test_the_largest_sums(path):
    """Codes of one sign at their ends, as many as a row holds: sums past 2^24 and up to 2^31."""
    for K in (4096, 131071):
        for a, b in ((-128, -128), (127, -128), (127, 127)):
            x, w = np.full((2, K), a, np.int8), np.full((3, K), b, np.int8)
            one = np.ones(3, np.float32)
            want, mag, most = ref.linear(x, one[:2], w, one, None)
            got = ds.linear_i8(*_dev(x, one[:2], w, one), path=path, dtype=torch.float32)["out"].double().cpu().numpy()
            assert np.all(np.abs(got - want) <= _allowed(want, mag, most, K, False, path))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T,K,N", [(37, 256, 300), (250, 144, 260), (9, 1000, 64)])
def test_strides_and_alignment(T, K, N, path):
    """Rows inside wider ones, at every offset from a 16-byte boundary that differs."""
    x, xs, w, ws, bias = _case(T, K, N)
    want, mag, most = ref.linear(x, xs, w, ws, bias)
    allow = _allowed(want, mag, most, K, True, path)
    for off in (0, 1, 4, 16):
        wide_x, wide_w = torch.zeros((T, K + 33), dtype=torch.int8, device=DEV), torch.zeros((N, K + 48), dtype=torch.int8, device=DEV)
        wide_x[:, off:off + K], wide_w[:, off:off + K] = _dev(x, w)
        big = torch.full((T, N + 5), 7.0, dtype=torch.bfloat16, device=DEV)
        got = ds.linear_i8(wide_x[:, off:off + K], *_dev(xs), wide_w[:, off:off + K], *_dev(ws),
                           bias=torch.as_tensor(bias, device=DEV), path=path, out={"out": big[:, 1:1 + N]})
        assert ds.check(got["workspace"]) == 0
        assert np.all(np.abs(got["out"].double().cpu().numpy() - want) <= allow)
        assert bool((big[:, 0] == 7).all()) and bool((big[:, 1 + N:] == 7).all())


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T,live", [(40, 33), (40, 0), (40, 40), (300, 195), (300, 1), (500, 384)])
def test_rows_scattered_and_rows_behind_the_last(T, live, path):
    K, N, rows = 192, 270, 700
    x, xs, w, ws, _ = _case(T, K, N)
    want, mag, most = ref.linear(x, xs, w, ws, None)
    allow = _allowed(want, mag, most, K, False, path)
    rng = np.random.default_rng(T + live)
    place = rng.permutation(rows)[:T].astype(np.int32)
    place[rng.random(T) < .2] = -1
    out = torch.full((rows // 10, 10, N), 9.0, device=DEV)
    n = torch.tensor([live], dtype=torch.int32, device=DEV)
    got = ds.linear_i8(*_dev(x, xs, w, ws), out_row=torch.as_tensor(place, device=DEV), n_rows=n, path=path, out={"out": out})
    assert ds.check(got["workspace"]) == 0
    flat = out.view(rows, N).double().cpu().numpy()
    left = np.ones(rows, bool)
    for t in range(live):
        if place[t] >= 0:
            left[place[t]] = False
            assert np.all(np.abs(flat[place[t]] - want[t]) <= allow[t])
    assert np.all(flat[left] == 9)
    # a place that is none, and a count of rows that is none
    place[:] = -1
    place[0] = rows
    got = ds.linear_i8(*_dev(x, xs, w, ws), out_row=torch.as_tensor(place, device=DEV), path=path, out={"out": out})
    assert ds.check(got["workspace"]) == ds.ERR_DEVICE_INPUT
    assert np.array_equal(out.view(rows, N).double().cpu().numpy(), flat)
    for bad in (-3, T + 1):
        plain = torch.full((T, N), 9.0, device=DEV)
        n.fill_(bad)
        got = ds.linear_i8(*_dev(x, xs, w, ws), n_rows=n, path=path, out={"out": plain})
        assert ds.check(got["workspace"]) == ds.ERR_DEVICE_INPUT
        plain = plain.double().cpu().numpy()
        assert np.all(plain == 9) if bad < 0 else np.all(np.abs(plain - want) <= allow)


@pytest.mark.parametrize("path", PATHS)
def test_a_scale_that_is_none_stays_in_its_row(path):
    x, xs, w, ws, _ = _case(50, 256, 300)
    xs[7] = np.nan
    got = ds.linear_i8(*_dev(x, xs, w, ws), path=path)["out"].float().cpu().numpy()
    assert np.isnan(got[7]).all() and np.isfinite(np.delete(got, 7, 0)).all()


def test_runs_give_the_same_bits_and_streams_do_not_mix():
    x, xs, w, ws, _ = _case(70, 8192, 520)
    args = _dev(x, xs, w, ws)
    a = ds.linear_i8(*args, dtype=torch.float32)["out"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for i in range(6):
        outs.append(ds.linear_i8(*args, dtype=torch.float32, stream=side if i % 2 else None)["out"])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for b in outs)


def test_captured_and_replayed():
    x, xs, w, ws, _ = _case(150, 1024, 600)
    dx, dxs, dw, dws = _dev(x, xs, w, ws)
    out = torch.empty((150, 600), device=DEV)
    work = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    call = lambda: ds.linear_i8(dx, dxs, dw, dws, out={"out": out}, workspace=work)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (5, 6):
        x, xs, w, ws, _ = _case(150, 1024, 600, seed=seed)
        for d, s in ((dx, x), (dxs, xs), (dw, w), (dws, ws)):
            d.copy_(torch.as_tensor(s))
        g.replay()
        want, mag, most = ref.linear(x, xs, w, ws, None)
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= _allowed(want, mag, most, 1024, False, ds.PATH_AUTO))
    assert ds.check(work) == 0


def test_empty_and_refused():
    i8 = dict(dtype=torch.int8, device=DEV)
    x, w = torch.zeros((3, 64), **i8), torch.zeros((5, 64), **i8)
    xs, ws = torch.ones(3, device=DEV), torch.ones(5, device=DEV)
    assert ds.linear_i8(x[:0], xs[:0], w, ws)["out"].shape == (0, 5)
    with pytest.raises(ValueError):
        ds.linear_i8(x, xs, w[:, :32], ws)
    with pytest.raises(TypeError):
        ds.linear_i8(x.float(), xs, w, ws)
    with pytest.raises(ValueError):
        ds.linear_i8(x, xs, w, ws, out_row=torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        ds.linear_i8(x, xs, w, ws, out={"out": torch.empty((2, 5), device=DEV)})
    with pytest.raises(TypeError):
        ds.linear_i8(x, xs, w, ws, dtype=torch.float16)
    with pytest.raises(ds.DsparkError) as e:
        ds.linear_i8(x, xs, w, ws, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == 3


@pytest.mark.parametrize("T,K,N", [(20, 2048, 300), (300, 1024, 40000)])
def test_a_wait_that_runs_out_is_recorded(T, K, N):
    """Under a limit of 1 ns the call ends with the status, and the next one without it is right."""
    x, xs, w, ws, _ = _case(T, K, N)
    args = _dev(x, xs, w, ws)
    want = ds.linear_i8(*args, path=ds.PATH_CUDA_CORE, dtype=torch.float32)["out"]
    ds.set_wait_limit(1)
    try:
        got = ds.linear_i8(*args, path=ds.PATH_TENSOR_CORE, dtype=torch.float32)
        assert ds.check(got["workspace"]) == ds.ERR_TIMEOUT
    finally:
        ds.set_wait_limit(0)
    for _ in range(3):
        got = ds.linear_i8(*args, path=ds.PATH_TENSOR_CORE, dtype=torch.float32)
        assert ds.check(got["workspace"]) == 0 and torch.equal(got["out"], want)


def test_calls_that_fill_every_sm_back_to_back():
    """Tiles by the hundred, several to a pair, in calls that nothing waits between."""
    x, xs, w, ws, _ = _case(700, 640, 8000)
    args = _dev(x, xs, w, ws)
    a, out = ds.linear_i8_args(*args, dtype=torch.float32)
    work = torch.zeros(ds.workspace_bytes("linear_i8", a), dtype=torch.uint8, device=DEV)
    want = ds.linear_i8(*args, path=ds.PATH_CUDA_CORE, dtype=torch.float32)["out"]
    for _ in range(300):
        ds.linear_i8(*args, out=out, workspace=work)
    assert ds.check(work) == 0 and torch.equal(out["out"], want)
