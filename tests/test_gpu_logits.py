"""seen_add and adjust_logits against the definitions in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import pass_ref as ref
import speculative_decoding_draft_round_gb300 as ds

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _f32(x):
    return None if x is None else torch.as_tensor(np.asarray(x, np.float32), device=DEV)


# ------------------------------------------------------------------ the table

@pytest.mark.parametrize("R,W,V", [(1, 1, 1), (3, 5, 9), (4, 300, 1003), (2, 4000, 8191), (2, 700, 8192), (3, 1000, 8193),
                                   (5, 257, 40000), (130, 17, 3001), (2, 0, 50)])
def test_table_against_the_definition(R, W, V):
    rng = np.random.default_rng(R * 7 + W + V)
    table = ds.seen_table(R, V)
    want = table.cpu().numpy()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    for step in range(5):
        tokens = np.minimum(rng.zipf(1.3, (R, W)) - 1, V - 1).astype(np.int32) if W else None
        n = rng.integers(0, W + 1, R).astype(np.int32) if step != 1 else None
        extra = rng.integers(0, V, R).astype(np.int32) if step % 2 else None
        fresh = (rng.random(R) < .5).astype(np.uint8) if step in (0, 3) else None
        if step == 0:
            table.random_(-32768, 32767)
            want = table.cpu().numpy()
        prompt = step in (0, 4)
        ds.seen_add(table, None if tokens is None else _i32(tokens), V=V, n=None if n is None else _i32(n),
                    extra=None if extra is None else _i32(extra),
                    fresh=None if fresh is None else torch.as_tensor(fresh, device=DEV), prompt=prompt, workspace=ws)
        want = ref.seen_add(want, V, tokens, n, extra, fresh, prompt)
        assert np.array_equal(table.cpu().numpy(), want)
    assert ds.check(ws) == 0


def test_counts_end_at_their_largest():
    V = 100
    for fresh in (True, False):
        table = ds.seen_table(2, V)
        tokens = torch.full((2, 40000), 3, dtype=torch.int32, device=DEV)
        tokens[1, ::2] = 4
        ds.seen_add(table, tokens, V=V, fresh=torch.full((2,), int(fresh), dtype=torch.uint8, device=DEV))
        assert table[0, 3] == 32767 and table[1, 3] == 20000 and table[1, 4] == 20000 and int((table != 0).sum()) == 3
        ds.seen_add(table, tokens[:, :1], V=V, prompt=True)
        assert table[0, 3] == -1 and table[1, 3] == 20000 and table[1, 4] == 20000 - 32768
        ds.seen_add(table, tokens[:, :1], V=V)
        assert table[0, 3] == -1 and table[1, 4] == 20001 - 32768


def test_table_tokens_that_are_none():
    """Recorded and skipped, in rows that are fresh and in others; counts of tokens are clamped."""
    V = 50
    for fresh in (0, 1):
        for bad in (-1, V, 55, 1 << 30, -(1 << 31)):
            table = ds.seen_table(2, V)
            ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
            ds.seen_add(table, _i32([[1, bad], [2, 2]]), V=V, fresh=torch.full((2,), fresh, dtype=torch.uint8, device=DEV),
                        workspace=ws)
            assert ds.check(ws) == ds.ERR_DEVICE_INPUT
            assert table[0, 1] == 1 and table[1, 2] == 2 and int((table != 0).sum()) == 2
        for n, rows in ((-1, 0), (3, 2)):
            table = ds.seen_table(2, V)
            ds.seen_add(table, _i32([[1, 4], [2, 5]]), V=V, n=_i32([n, 2]), workspace=ws,
                        fresh=torch.full((2,), fresh, dtype=torch.uint8, device=DEV))
            assert ds.check(ws) == ds.ERR_DEVICE_INPUT
            assert int((table[0] != 0).sum()) == rows and int((table[1] != 0).sum()) == 2


def test_table_rows_of_wider_tables():
    table = torch.zeros((3, 80), dtype=torch.int16, device=DEV)
    tokens = torch.arange(12, dtype=torch.int32, device=DEV).view(3, 4)
    ds.seen_add(table[:, :40], tokens[:, 1:3], V=33)
    want = np.zeros((3, 80), np.int16)
    for r in range(3):
        want[r, [4 * r + 1, 4 * r + 2]] = 1
    assert np.array_equal(table.cpu().numpy(), want)
    with pytest.raises(ds.DsparkError):
        ds.seen_add(table[:, 1:40], tokens, V=33)       # off a 16-byte boundary
    with pytest.raises(ValueError):
        ds.seen_add(table, tokens, V=81)


# ------------------------------------------------------------------ the logits

def _ask(R, S, V, rng, biases=True, masks=True):
    a = {"rep": np.where(rng.random(R) < .3, 1.0, np.exp(.3 * rng.standard_normal(R))).astype(np.float32),
         "pres": np.where(rng.random(R) < .3, 0.0, rng.standard_normal(R)).astype(np.float32),
         "freq": np.where(rng.random(R) < .3, 0.0, rng.standard_normal(R)).astype(np.float32)}
    seen = np.zeros((R, -(-V // 8) * 8), np.int16)
    seen[:, :V] = np.where(rng.random((R, V)) < .1, rng.integers(1, 40, (R, V)), 0)
    seen[:, :V] |= np.where(rng.random((R, V)) < .1, -32768, 0).astype(np.int16)
    a["seen"] = seen
    a["tokens"] = rng.integers(0, V, (R, S - 1)).astype(np.int32)
    if S > 3:
        a["tokens"][:, 1] = a["tokens"][:, 0]           # the same token twice
    a["biases"] = [[(int(v), float(np.float32(x))) for v, x in zip(rng.integers(0, V, n), 5 * rng.standard_normal(n))]
                   for n in rng.integers(0, 9, R)] if biases else None
    if biases and V > 4:
        a["biases"][0] += [(3, 1.5), (3, -0.25), (V - 1, -np.inf)]
    a["mask"] = rng.random((5, V)) < np.array([0, .01, .5, .99, 1.])[:, None] if masks else None
    a["mask_row"] = rng.integers(-1, 5, (R, S)).astype(np.int32) if masks else None
    a["keep"] = rng.integers(0, S, R).astype(np.int32)
    return a


def _args(a):
    kw = dict(seen=torch.as_tensor(a["seen"], device=DEV), repetition=_f32(a["rep"]), presence=_f32(a["pres"]),
              frequency=_f32(a["freq"]), tokens=_i32(a["tokens"]), keep=_i32(a["keep"]))
    if a["biases"] is not None:
        flat = [e for b in a["biases"] for e in b]
        kw.update(bias_offsets=_i32(np.concatenate([[0], np.cumsum([len(b) for b in a["biases"]])])),
                  bias_token=_i32([e[0] for e in flat]), bias_value=_f32([e[1] for e in flat]))
    if a["mask"] is not None:
        kw.update(mask=torch.as_tensor(ref.pack_bits(a["mask"]), device=DEV), mask_row=_i32(a["mask_row"]))
    return kw


def _compare(got, logits, a, bf16):
    with np.errstate(invalid="ignore"):
        want, mag = ref.adjust(logits.astype(np.float64), a["seen"], a["rep"], a["pres"], a["freq"], a["tokens"], a["biases"],
                               a["mask"], a["mask_row"], a["keep"])
    live = np.arange(logits.shape[1]) <= a["keep"][:, None]
    got, want, mag = got[live], want[live], mag[live]
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    # quotient or product, the frequency's step, the presence's, the bias': one rounding each, and a bias' own sums
    with np.errstate(invalid="ignore"):
        near = np.abs(got - want) <= 8 * 2.0 ** -24 * mag + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(want)
    assert np.all(same | near)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("R,S,V", [(1, 1, 1), (2, 1, 7), (4, 5, 64), (4, 5, 1003), (3, 17, 2048), (2, 33, 2056), (9, 2, 4100),
                                   (5, 6, 10000), (3, 4, 6147)])
def test_logits_against_the_definition(R, S, V, bf16):
    rng = np.random.default_rng(R + S * 10 + V)
    a = _ask(R, S, V, rng)
    logits = ref.rows(3 * rng.standard_normal((R, S, V)), bf16)
    logits[rng.random(logits.shape) < .01] = -np.inf
    logits[rng.random(logits.shape) < .01] = 0
    dev = torch.as_tensor(logits).to(torch.bfloat16 if bf16 else torch.float32).to(DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out = torch.full_like(dev, 123.0)
    ds.adjust_logits(dev, **_args(a), out={"out": out}, workspace=ws)
    assert ds.check(ws) == 0
    _compare(out.double().cpu().numpy(), logits, a, bf16)
    live = torch.as_tensor(np.arange(S) <= a["keep"][:, None], device=DEV)
    assert bool((out[~live] == 123).all())
    assert np.array_equal(dev.float().cpu().numpy(), logits)
    # in place: the same, and the rows behind the last as they were
    mine = dev.clone()
    ds.adjust_logits(mine, **_args(a), out={"out": mine}, workspace=ws)
    assert torch.equal(mine[live], out[live]) and torch.equal(mine[~live], dev[~live])


@pytest.mark.parametrize("V", [4096, 1001])
def test_each_alone_and_none(V):
    rng = np.random.default_rng(V)
    R, S = 3, 4
    a = _ask(R, S, V, rng)
    logits = rng.standard_normal((R, S, V)).astype(np.float32)
    dev = torch.as_tensor(logits, device=DEV)
    full = _args(a)
    assert torch.equal(ds.adjust_logits(dev)["out"], dev)
    none = dict(rep=None, pres=None, freq=None, seen=None, tokens=None, biases=None, mask=None, mask_row=None,
                keep=np.full(R, S - 1, np.int32))
    for names, parts in ((("seen", "repetition"), ("seen", "rep")), (("seen", "frequency"), ("seen", "freq")),
                         (("tokens", "presence"), ("tokens", "pres")), (("bias_offsets", "bias_token", "bias_value"), ("biases",)),
                         (("mask", "mask_row"), ("mask", "mask_row")), (("seen", "tokens"), ("seen", "tokens"))):
        out = ds.adjust_logits(dev, **{n: full[n] for n in names})["out"].double().cpu().numpy()
        _compare(out, logits, dict(none, **{n: a[n] for n in parts}), False)
    # a mask row for every row of logits
    mask = rng.random((R * S, V)) < .5
    out = ds.adjust_logits(dev, mask=torch.as_tensor(ref.pack_bits(mask), device=DEV))["out"].double().cpu().numpy()
    _compare(out, logits, dict(none, mask=mask), False)


@pytest.mark.parametrize("V", [2048, 515])
def test_what_a_mask_hides_is_not_looked_at(V):
    """NaN and infinities in masked places, a mask that leaves nothing, the type's lowest values."""
    for dt in (torch.float32, torch.bfloat16):
        x = torch.randn((1, 3, V), device=DEV).to(dt)
        allowed = np.zeros((2, V), bool)
        allowed[1, ::3] = True
        x[0, :, 1::3], x[0, 1, 2::3], x[0, 0, ::3] = float("nan"), float("inf"), torch.finfo(dt).min
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        out = ds.adjust_logits(x, mask=torch.as_tensor(ref.pack_bits(allowed), device=DEV), mask_row=_i32([[1, 1, 0]]),
                               repetition=_f32([1.0]), workspace=ws)["out"]
        assert ds.check(ws) == 0
        assert torch.equal(out[0, :2, ::3], x[0, :2, ::3])
        hidden = torch.as_tensor(~allowed[1], device=DEV)
        assert bool((out[0, :2, hidden] == -float("inf")).all()) and bool((out[0, 2] == -float("inf")).all())


def test_inputs_that_are_none():
    R, S, V = 3, 3, 300
    x = torch.randn((R, S, V), device=DEV)
    seen = torch.ones((R, 304), dtype=torch.int16, device=DEV)
    bad = [dict(seen=seen, repetition=_f32([1, v, 1])) for v in (0.0, -1.0, np.nan, np.inf)]
    bad += [dict(seen=seen, presence=_f32([0, v, 0])) for v in (np.nan, np.inf)]
    bad += [dict(seen=seen, frequency=_f32([0, v, 0])) for v in (np.nan, -np.inf)]
    bad += [dict(bias_offsets=_i32(o), bias_token=_i32([5, 6]), bias_value=_f32([0, 0]))
            for o in ([0, 0, -1, -1], [0, 2, 1, 1], [0, 0, 3, 3])]
    bad += [dict(bias_offsets=_i32([0, 1, 2, 2]), bias_token=_i32([t, 6]), bias_value=_f32([7, 0])) for t in (-1, V, 1 << 30)]
    bad += [dict(presence=_f32([0, 0, 0]), tokens=_i32([[1, 2], [V, 1], [1, 1]]))]
    bad += [dict(mask=torch.zeros((2, 10), dtype=torch.int32, device=DEV), mask_row=_i32([[-1, 2, -1]] * R))]
    for kw in bad:
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        out = ds.adjust_logits(x, workspace=ws, **kw)["out"]
        assert ds.check(ws) == ds.ERR_DEVICE_INPUT, kw
        assert torch.equal(out, x)
    for keep, rows in ((-1, 1), (S, S)):
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        out = torch.zeros_like(x)
        ds.adjust_logits(x, keep=_i32([keep, 0, 1]), workspace=ws, out={"out": out})
        assert ds.check(ws) == ds.ERR_DEVICE_INPUT
        assert torch.equal(out[0, :rows], x[0, :rows]) and not out[0, rows:].any() and not out[1, 1:].any()
    with pytest.raises(ValueError):
        ds.adjust_logits(x, mask_row=_i32([[0] * S] * R))
    with pytest.raises(ValueError):
        ds.adjust_logits(x, mask=torch.zeros((9, 9), dtype=torch.int32, device=DEV))
    with pytest.raises(ds.DsparkError):
        ds.adjust_logits(x, mask=torch.zeros((8, 10), dtype=torch.int32, device=DEV))
    with pytest.raises(ds.DsparkError):
        ds.adjust_logits(x, mask=torch.zeros((1, 10), dtype=torch.int32, device=DEV).expand(9, 10))
    with pytest.raises(TypeError):
        ds.adjust_logits(x.half())


def test_many_biases_of_one_token_add_up_in_order():
    V = 3000
    rng = np.random.default_rng(4)
    n = 1000
    value = rng.standard_normal(n).astype(np.float32)
    token = np.where(rng.random(n) < .5, 2500, rng.integers(0, V, n)).astype(np.int32)
    x = torch.zeros((1, 1, V), device=DEV)
    args = dict(bias_offsets=_i32([0, n]), bias_token=_i32(token), bias_value=_f32(value))
    out = ds.adjust_logits(x, **args)["out"].cpu().numpy()[0, 0]
    want = np.zeros(V, np.float32)
    for t, v in zip(token, value):
        want[t] = np.float32(want[t] + v)
    assert np.array_equal(out, want)


def test_fresh_rows_end_with_their_words():
    """Clearing the rows of a view leaves what lies between them, before the first and behind the last as it was."""
    wide = torch.full((5, 96), 7, dtype=torch.int16, device=DEV)
    view = wide[1:4, 40:80]
    ds.seen_add(view, _i32([[3], [32], [0]]), V=33, fresh=torch.ones(3, dtype=torch.uint8, device=DEV))
    want = np.full((5, 96), 7, np.int16)
    want[1:4, 40:80] = 0
    want[[1, 2, 3], [43, 72, 40]] = 1
    assert np.array_equal(wide.cpu().numpy(), want)
    with pytest.raises(ds.DsparkError):
        ds.seen_add(wide[:, 40:76], None, V=33)
