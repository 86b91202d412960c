"""add_norm_quant's codes next to a half and its scales next to fp32's end, against whole numbers of any length."""
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_draft_round_gb300 as ds

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _codes(s, g):
    """The nearest whole number to 127 p / max|p| of a row, ties to even, in exact arithmetic."""
    p = [Fraction(float(a)) * Fraction(float(b)) for a, b in zip(s, g)]
    top = max(abs(x) for x in p)
    return np.array([round(127 * x / top) for x in p])       # Fraction rounds ties to even


def _quantised(s, g, bf16=False, norm=True):
    x = torch.as_tensor(np.ascontiguousarray(s), device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    got = ds.add_norm_quant(x.bfloat16() if bf16 else x, gain=None if g is None else torch.as_tensor(g, device=DEV),
                            norm=norm, eps=0.0, workspace=ws)
    assert ds.check(ws) == 0
    return got["codes"].cpu().numpy().astype(np.int64), got["scale"].cpu().numpy()


@pytest.mark.parametrize("N", [256, 2048, 77])
@pytest.mark.parametrize("gained", [False, True])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -60, 2.0 ** -110, 2.0 ** 100])
def test_the_nearest_values_on_both_sides_of_a_half(N, gained, size):
    """Quotients as near to k + 1/2 as fp32 elements allow, and an ulp beside that. (Sizes out of fp32's range for the
    squares go through 64 bits.)"""
    rng = np.random.default_rng(N)
    T = 12
    g = (1 + rng.random(N)).astype(np.float32) if gained else np.ones(N, np.float32)
    s = np.empty((T, N), np.float32)
    s[:, 0] = ((2 + rng.random(T)) * size).astype(np.float32)
    top = s[:, 0].astype(np.float64) * float(g[0])
    k = rng.integers(0, 126, (T, N - 1))
    near = ((k + 0.5) / 127 * top[:, None] / g[1:]).astype(np.float32)
    near = np.where(rng.random(near.shape) < .3, np.nextafter(near, np.float32(np.inf)), near)
    s[:, 1:] = near * rng.choice([-1, 1], near.shape)
    codes, _ = _quantised(s, g if gained else None)
    for t in range(T):
        assert np.array_equal(codes[t], _codes(s[t], g))


@pytest.mark.parametrize("N", [64, 2048, 77])
def test_rows_in_bf16_next_to_a_half(N):
    """Elements of 8 bits, gains of 24: the gain brings the quotient next to the half."""
    rng = np.random.default_rng(N)
    for _ in range(6):
        s = (1 + rng.integers(0, 128, N) / 128).astype(np.float32)
        g = np.empty(N, np.float32)
        g[0] = 2 + rng.random()
        top = float(s[0]) * float(g[0])
        g[1:] = (rng.integers(0, 120, N - 1) + 0.5) / 127 * top / s[1:]
        codes, _ = _quantised(s[None], g, bf16=True)
        assert np.array_equal(codes[0], _codes(s, g))


# s, g, the largest element and its gain, all of 24 bits: 127 s g / 128 and the product of the others are whole numbers and
# 1/128 apart, so that the quotient is next to 1/2 by less than 64 bits of floating point hold
NEAR = [(15652751, 9918353, 12350715, 12471879), (16756431, 9875153, 12658865, 12969533),
        (11865523, 14839045, 12684132, 13772914), (14687705, 13442327, 13376829, 14644312),
        (15280753, 11557615, 11426133, 15335836), (13947433, 14094233, 13558418, 14385351)]


@pytest.mark.parametrize("N", [64, 2048, 33])
@pytest.mark.parametrize("size", [2.0 ** -24, 2.0 ** -90])
def test_quotients_that_64_bits_do_not_tell_from_a_half(N, size):
    for a, b, c, d in NEAR:
        s, g = np.zeros(N, np.float32), np.ones(N, np.float32)
        s[:4] = [c * size, a / 256 * size, -a / 256 * size, c * size / 3]
        g[:4] = [d * 2.0 ** -24, b * 2.0 ** -24, b * 2.0 ** -24, 1.0]
        want = _codes(s, g)
        assert abs(want[1]) == int(127 * a * b > 128 * c * d)
        for sign in (1, -1):
            codes, _ = _quantised((sign * s)[None], g)
            assert np.array_equal(codes[0], sign * want)


@pytest.mark.parametrize("N", [1024, 8192, 999])
def test_scales_whose_largest_value_leaves_fp32(N):
    """The largest |y| is past fp32's end and its 127th part is not."""
    s, g = np.zeros((2, N), np.float32), np.ones(N, np.float32)
    s[0, 3], s[1, 3], s[1, 5] = 1e-9, -1e-9, 3e-10
    g[3] = 3e38
    codes, scale = _quantised(s, g)
    for t in range(2):
        assert np.array_equal(codes[t], _codes(s[t], g))
        p = s[t].astype(np.float64) * g
        want = np.abs(p).max() / np.sqrt((s[t].astype(np.float64) ** 2).mean()) / 127
        assert want > 2.0 ** 128 / 127 and want < 2.0 ** 128
        # the sum's and the other steps' roundings: fewer than 2^7 of 2^-24
        assert abs(scale[t] - want) <= 2.0 ** -17 * want
