"""The target layer's attention written out in numpy, 64 bits, for the tests: head norms and rotation, the
4-bit cache's format, and attention over it. Shares nothing with the CUDA path; loops, not speed."""
import math

import numpy as np

GROUP = 32


def bf16_round(x):
    """fp32 values rounded to bf16 (nearest even), as fp32."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32)


def scales_of(x):
    """The stored scale of each group of rows x [..., D] (finite), as float64 [..., D / 32]."""
    g = np.abs(np.asarray(x, np.float32)).reshape(*x.shape[:-1], -1, GROUP).max(-1)
    s = bf16_round(g * (np.float32(1) / np.float32(7)))
    return np.minimum(s, np.float32(9344)).astype(np.float16).astype(np.float64)


def codes_of(x, s):
    """The codes -7 .. 7 of rows x for scales s; np.rint rounds half to even."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, GROUP)
    safe = np.where(s > 0, s, 1.0)[..., None]
    c = np.where(s[..., None] > 0, np.rint(g / safe), 0.0)
    return np.clip(c, -7, 7).reshape(x.shape)


def stored(x):
    """What the cache holds of rows x."""
    s = scales_of(x)
    return codes_of(x, s) * np.repeat(s, GROUP, -1)


def block_parts(page, D):
    """Byte offsets of V codes, K scales, V scales and the block's end."""
    return page * D // 2, page * D, page * D + page * D // 16, page * D * 9 // 8


def block_row(block, slot, page, D, half):
    """The values of token `slot` in one block (uint8 vector): half 0 = K, 1 = V."""
    v, ks, vs, _ = block_parts(page, D)
    base = (0 if half == 0 else v) + slot * (D // 2)
    u = block[base:base + D // 2].astype(np.int64)
    c = np.empty(D)
    c[0::2], c[1::2] = (u & 15) - 8, (u >> 4) - 8
    s = np.empty(D // GROUP)
    for g in range(D // GROUP):
        at = ks + 2 * (slot * (D // GROUP) + g) if half == 0 else \
            vs + 2 * (((slot // 16) * (D // GROUP) + g) * 16 + slot % 16)
        s[g] = block[at:at + 2].copy().view(np.float16)[0]
    return c * np.repeat(s, GROUP)


def norm_rope(x, gain, pos, freq, norm, eps, interleaved):
    """x [T][H][D] normed and turned; freq: Python ints in units of 2^-64 turns."""
    y = np.asarray(x, np.float64)
    D = y.shape[-1]
    if norm:
        y = y / np.sqrt((y * y).sum(-1, keepdims=True) / D + eps)
    if norm and gain is not None:
        y = y * np.asarray(gain, np.float64)
    elif gain is not None:
        y = y * np.asarray(gain, np.float64)
    out = y.copy()
    half = len(freq)
    for t, p in enumerate(pos):
        for i, f in enumerate(freq):
            phi = 2 * math.pi * (((int(f) * int(p)) % (1 << 64)) / 2.0 ** 64)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = math.cos(phi), math.sin(phi)
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, a] * s + y[t, :, b] * c
    return out


def visible(p, n, window, sinks):
    i = np.arange(n)
    see = i <= p
    if window:
        see &= (i > p - window) | (i < sinks)
    return see


def attend(q, keys, values, ctx, offsets, scale, window, sinks):
    """q [T][Hq][D]; keys, values: per request [n][Hkv][D] (n = ctx + rows). Returns out, lse and, per row and
    head, the largest sum over channels of |q k| scale, which bounds the rounding of its products."""
    T, Hq, D = q.shape
    out = np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    mag = np.zeros((T, Hq))
    for r in range(len(ctx)):
        Hkv = keys[r].shape[1]
        G = Hq // Hkv
        for t in range(offsets[r], offsets[r + 1]):
            p = ctx[r] + t - offsets[r]
            see = visible(p, keys[r].shape[0], window, sinks)
            if not see.any():
                continue
            for h in range(Hq):
                k, v = keys[r][see, h // G], values[r][see, h // G]
                x = q[t, h].astype(np.float64)
                z = (k @ x) * scale
                mag[t, h] = (np.abs(k) @ np.abs(x)).max() * scale
                top = z.max()
                e = np.exp(z - top)
                out[t, h] = (e / e.sum()) @ v
                lse[t, h] = top + math.log(e.sum())
    return out, lse, mag
