"""add_norm_quant against 64 bits: codes and sums exactly, values and scales to what their roundings allow."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import pass_ref as ref
import speculative_decoding_draft_round_gb300 as ds

pytestmark = pytest.mark.gpu
DEV = "cuda"
# the sum of squares has at most 128 products a thread and 13 steps over threads, each off by 2^-24 of a sum of positive
# terms; the root halves that; division, sum with eps, root, reciprocal, the product s * gain, its product with the
# reciprocal and the quotient by 127 add one rounding each: 71 + 7 < 2^7 roundings
REL = 2.0 ** -17


def _dt(bf16):
    return torch.bfloat16 if bf16 else torch.float32


def _put(x, bf16):
    return torch.as_tensor(np.ascontiguousarray(x)).to(_dt(bf16)).to(DEV)


def _check(got, x, res, gain, norm, eps, bf16, rows=None):
    s, y, c, scale = ref.norm_quant(x, res, gain, norm, eps, bf16)
    n = len(x) if rows is None else rows
    if "sum" in got:
        assert np.array_equal(got["sum"].float().cpu().numpy()[:n], s[:n])
    if "codes" in got:
        assert np.array_equal(got["codes"].cpu().numpy()[:n].astype(np.int64), c[:n])
        assert np.all(np.abs(got["scale"].cpu().numpy()[:n] - scale[:n]) <= REL * scale[:n] + 2.0 ** -149)
    if "y" in got:
        err = np.abs(got["y"].double().cpu().numpy()[:n] - y[:n])
        assert np.all(err <= ((2.0 ** -8 if bf16 else 2.0 ** -24) + REL) * np.abs(y[:n]) + 2.0 ** -133)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,N", [(1, 1), (3, 7), (5, 8), (9, 256), (2, 264), (7, 512), (17, 1000), (4, 1024), (3, 1032),
                                 (5, 2049), (33, 4096), (2, 4104), (3, 5120), (6, 8192), (2, 8200), (3, 12288), (2, 16384),
                                 (2, 16392), (1, 32768), (2, 32767)])
@pytest.mark.parametrize("res,gain,norm", [(True, True, True), (False, False, False), (True, False, True),
                                           (False, True, True)])
def test_against_64_bits(T, N, bf16, res, gain, norm):
    rng = np.random.default_rng(T * 100003 + N)
    make = lambda: ref.rows(rng.standard_normal((T, N)) * np.exp(rng.standard_normal((T, 1))), bf16)
    x, r = make(), make() if res else None
    g = (1 + 0.3 * rng.standard_normal(N)).astype(np.float32) if gain else None
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    got = ds.add_norm_quant(_put(x, bf16), residual=None if r is None else _put(r, bf16),
                            gain=None if g is None else torch.as_tensor(g, device=DEV), eps=1e-5, norm=norm, values=True,
                            workspace=ws)
    assert ds.check(ws) == 0
    _check(got, x, r, g, norm, 1e-5, bf16)
    if T <= 7:   # one output alone
        for kw in (dict(codes=False, values=True), dict(codes=True)):
            one = ds.add_norm_quant(_put(x, bf16), residual=None if r is None else _put(r, bf16),
                                    gain=None if g is None else torch.as_tensor(g, device=DEV), eps=1e-5, norm=norm, **kw)
            assert all(torch.equal(one[k], got[k]) for k in one if k != "workspace")


@pytest.mark.parametrize("N", [4096, 1021])
def test_codes_at_the_borders(N):
    """Quotients that lie on a half and next to it: whole numbers of halves of a step, with and without a nudge."""
    rng = np.random.default_rng(N)
    k = rng.integers(-254, 255, (64, N)).astype(np.float64)
    k[:, 0] = 254
    x = (k / 2 * np.exp2(rng.integers(-20, 20, (64, 1)))).astype(np.float32)
    g = np.where(rng.random(N) < .5, 1.0, 1 + 2.0 ** -23 * rng.integers(-3, 4, N)).astype(np.float32)
    g[0] = 1.0
    for gain in (None, g):
        got = ds.add_norm_quant(torch.as_tensor(x, device=DEV), gain=None if gain is None else torch.as_tensor(gain, device=DEV))
        _check(got, x, None, gain, True, 1e-6, False)
    # several products that round to the same largest one
    x[:, 1:] = rng.choice([1.0, 1.0 + 2.0 ** -23, 0.5], (64, N - 1)) * x[:, :1]
    got = ds.add_norm_quant(torch.as_tensor(x, device=DEV), gain=torch.as_tensor(g, device=DEV))
    _check(got, x, None, g, True, 1e-6, False)


@pytest.mark.parametrize("N", [512, 333])
@pytest.mark.parametrize("bf16", [True, False])
def test_rows_at_the_ends_of_the_range(N, bf16):
    rng = np.random.default_rng(3)
    x = ref.rows(rng.standard_normal((7, N)), bf16)
    x[0] = 0
    x[1] *= np.float32(1e-38)
    x[2] *= np.float32(2.0 ** -130)
    x[3] *= np.float32(2.0 ** 124)
    x[4] *= np.float32(1e-18)
    x[5] *= np.float32(1e18)
    x = ref.rows(x, bf16)
    g = np.full(N, 3.0, np.float32)
    for gain, eps in ((None, 0.0), (g, 0.0), (None, 1e-6)):
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        got = ds.add_norm_quant(_put(x, bf16), gain=None if gain is None else torch.as_tensor(gain, device=DEV), eps=eps,
                                values=True, workspace=ws)
        assert ds.check(ws) == 0
        _check(got, x, None, gain, True, eps, bf16)


@pytest.mark.parametrize("N", [256, 2048, 77])
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
def test_a_row_that_is_not_finite_stays_alone(N, what):
    rng = np.random.default_rng(N)
    x = rng.standard_normal((6, N)).astype(np.float32)
    x[2, N // 2] = what
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    got = ds.add_norm_quant(_put(x, False), values=True, workspace=ws)
    assert ds.check(ws) == ds.ERR_NONFINITE_INPUT
    assert torch.isnan(got["scale"][2]) and not got["codes"][2].any()
    assert torch.isnan(got["y"][2]).any()
    keep = [0, 1, 3, 4, 5]
    _check({k: got[k][keep] for k in ("codes", "scale", "y")}, x[keep], None, None, True, 1e-6, False)
    # a gain that is none
    g = np.ones(N, np.float32)
    g[N // 3] = what
    got = ds.add_norm_quant(_put(x[:2], False), gain=torch.as_tensor(g, device=DEV), workspace=ws)
    assert ds.check(ws) == ds.ERR_NONFINITE_INPUT and torch.isnan(got["scale"]).all() and not got["codes"].any()


@pytest.mark.parametrize("N,off", [(512, 0), (512, 1), (99, 3), (2048, 8)])
@pytest.mark.parametrize("bf16", [True, False])
def test_strides_in_place_and_rows_behind_the_last(N, off, bf16):
    """Views into wider rows, the sum over the residual, y over x, and rows past n_rows as they were."""
    rng = np.random.default_rng(N + off)
    T, live = 9, 6
    wide = _put(rng.standard_normal((T, N + 24)), bf16)
    res = _put(rng.standard_normal((T, N + 16)), bf16)
    x, r = wide[:, off:off + N], res[:, off:off + N]
    wide0, res0 = wide.clone(), res.clone()
    codes = torch.full((T, N + 8), 77, dtype=torch.int8, device=DEV)
    scale = torch.full((T,), -5.0, device=DEV)
    n = torch.tensor([live], dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    ds.add_norm_quant(x, residual=r, values=True, n_rows=n, workspace=ws,
                      out={"codes": codes[:, :N], "scale": scale, "y": x, "sum": r})
    assert ds.check(ws) == 0
    a, b = wide0[:, off:off + N].float().cpu().numpy(), res0[:, off:off + N].float().cpu().numpy()
    _check({"codes": codes[:, :N], "scale": scale, "y": x, "sum": r}, a, b, None, True, 1e-6, bf16, live)
    assert torch.equal(wide[live:], wide0[live:]) and torch.equal(res[live:], res0[live:])
    assert torch.equal(wide[:, off + N:], wide0[:, off + N:]) and torch.equal(wide[:, :off], wide0[:, :off])
    assert bool((codes[live:] == 77).all()) and bool((codes[:, N:] == 77).all()) and bool((scale[live:] == -5).all())
    for bad, rows in ((T + 1, T), (-1, 0)):
        scale.fill_(-5.0)
        ds.add_norm_quant(wide0[:, :N], n_rows=torch.tensor([bad], dtype=torch.int32, device=DEV), workspace=ws,
                          out={"codes": codes[:, :N], "scale": scale})
        assert ds.check(ws) == ds.ERR_DEVICE_INPUT
        assert int((scale != -5).sum()) == rows


def test_empty_and_refused():
    x = torch.empty((0, 64), device=DEV)
    got = ds.add_norm_quant(x, values=True)
    assert got["codes"].shape == (0, 64) and got["scale"].shape == (0,)
    x = torch.zeros((4, 64), device=DEV)
    with pytest.raises(ValueError):
        ds.add_norm_quant(x, out={"codes": torch.empty((4, 64), dtype=torch.int8, device=DEV)})
    with pytest.raises(ValueError):
        ds.add_norm_quant(x.t())
    with pytest.raises(TypeError):
        ds.add_norm_quant(x.half())
    with pytest.raises(TypeError):
        ds.add_norm_quant(x, residual=x.bfloat16())
    with pytest.raises(ds.DsparkError):
        ds.add_norm_quant(x, codes=False)
    with pytest.raises(ds.DsparkError):
        ds.add_norm_quant(x, codes=False, values=True, out={"y": x[:1].expand(4, 64)})
