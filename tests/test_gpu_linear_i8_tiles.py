"""linear_i8 over many tiles a pair of CTAs, several bands of rows, and wide K: the sums bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_draft_round_gb300 as ds

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _codes(rows, cols, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-127, 128, (rows, cols), dtype=torch.int8, device=DEV, generator=g)


def _sums(x, w):
    """Whole sums: products of codes and sums of 2^17 of them are exact in 64 bits."""
    return torch.cat([x.double() @ w[a:a + 4096].double().t() for a in range(0, len(w), 4096)], 1)


def _run(T, K, N, calls, seed=0, **kw):
    x, w = _codes(T, K, seed), _codes(N, K, seed + 1)
    one = lambda n: torch.ones(n, device=DEV)
    # codes of random sign: the largest partial sum over K, in any range of it, stays below 2^24 (2^24 is over eight standard
    # deviations of a sum of 131071 products), so every order of summation gives the whole number
    want = _sums(x, w)
    assert float(want.abs().max()) < 2 ** 24
    a, out = ds.linear_i8_args(x, one(T), w, one(N), dtype=torch.float32)
    work = torch.zeros(ds.workspace_bytes("linear_i8", a), dtype=torch.uint8, device=DEV)
    for _ in range(calls):
        out["out"].fill_(7.0)
        ds.linear_i8(x, one(T), w, one(N), out=out, workspace=work, path=ds.PATH_TENSOR_CORE, **kw)
    assert ds.check(work) == 0
    assert torch.equal(out["out"].double(), want)


@pytest.mark.parametrize("T,K,N,calls", [
    (700, 640, 16200, 40),       # 4 x 64 tiles: four for some pairs, so that accumulators are emptied and filled again
    (190, 256, 120000, 40),      # one run of rows, 469 tiles
    (2176, 512, 5000, 40),       # 12 x 20 tiles
    (385, 128, 50000, 10),       # one step of K a tile
    (129, 200, 40000, 10),       # 129 rows are 160 columns; a last step of K that is part empty
])
def test_many_tiles_a_pair(T, K, N, calls):
    _run(T, K, N, calls)


@pytest.mark.parametrize("T,K,N", [
    (600, 131071, 700),          # a band is one run of rows: 3 to 4 bands; weights laid out anew
    (2000, 40000, 600),          # bands of two runs, the last one of one
    (2100, 16384, 1030),         # bands of five runs
])
def test_more_runs_of_rows_than_a_band(T, K, N):
    _run(T, K, N, 2)


@pytest.mark.parametrize("T,K,N", [(7, 4097, 520), (20, 8192, 129), (64, 8192, 3000), (192, 4097, 1000), (250, 12300, 300),
                                   (16, 131071, 260)])
def test_wide_k_bit_for_bit(T, K, N):
    """Split along K over the pairs of a cluster, or not: no product is lost or taken twice."""
    _run(T, K, N, 3)


def test_two_streams_that_fill_the_gpu():
    """Calls on two streams at once, each with more tiles than the GPU holds pairs."""
    side = torch.cuda.Stream()
    cases = []
    for seed, (T, K, N) in enumerate(((700, 640, 16200), (190, 256, 120000))):
        x, w = _codes(T, K, seed), _codes(N, K, 9 + seed)
        xs, ws = torch.ones(T, device=DEV), torch.ones(N, device=DEV)
        a, out = ds.linear_i8_args(x, xs, w, ws, dtype=torch.float32)
        work = torch.zeros(ds.workspace_bytes("linear_i8", a), dtype=torch.uint8, device=DEV)
        cases.append((x, xs, w, ws, out, work, _sums(x, w)))
    torch.cuda.synchronize()
    for _ in range(60):
        for stream, (x, xs, w, ws, out, work, _) in zip((torch.cuda.current_stream(), side), cases):
            ds.linear_i8(x, xs, w, ws, out=out, workspace=work, stream=stream)
    torch.cuda.synchronize()
    for *_, out, work, want in cases:
        assert ds.check(work) == 0 and torch.equal(out["out"].double(), want)


def test_rows_scattered_over_many_tiles():
    """n_rows and out_row where live rows end inside a run of rows and pairs take several tiles."""
    T, K, N, rows = 700, 384, 30000, 900
    x, w = _codes(T, K, 3), _codes(N, K, 4)
    place = np.random.default_rng(5).permutation(rows)[:T].astype(np.int32)
    place[::7] = -1
    at = torch.as_tensor(place, device=DEV)
    one = lambda n: torch.ones(n, device=DEV)
    want = _sums(x, w)
    for live in (700, 577, 193, 1, 0):
        out = torch.full((rows, N), 9.0, device=DEV)
        n = torch.tensor([live], dtype=torch.int32, device=DEV)
        got = ds.linear_i8(x, one(T), w, one(N), out_row=at, n_rows=n, out={"out": out})
        assert ds.check(got["workspace"]) == 0
        full = torch.full((rows, N), 9.0, dtype=torch.float64, device=DEV)
        keep = torch.as_tensor(np.flatnonzero(place[:live] >= 0), device=DEV)
        full[at[keep].long()] = want[keep]
        assert torch.equal(out.double(), full)
