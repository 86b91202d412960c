"""The rest of the target's pass written out in numpy, 64 bits, for the tests: norms and 8-bit codes, 8-bit products,
the table of seen tokens and the adjustment of logits. Shares nothing with the CUDA path."""
import numpy as np

from layer_ref import bf16_round


def rows(x, bf16):
    """Values that the type holds, as float32."""
    x = np.asarray(x, np.float32)
    return bf16_round(x) if bf16 else x


def norm_quant(x, residual, gain, norm, eps, bf16):
    """sum (float32), y, codes and scale of finite rows."""
    s = x if residual is None else rows(x + residual, bf16)
    p = s.astype(np.float64) * (1.0 if gain is None else gain.astype(np.float64))
    inv = 1.0 / np.sqrt((s.astype(np.float64) ** 2).mean(-1, keepdims=True) + eps) if norm else np.ones((len(x), 1))
    top = np.abs(p).max(-1, keepdims=True)
    safe = np.where(top > 0, top, 1.0)
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.where(top > 0, p * inv, 0.0)
        scale = np.where(top > 0, top * inv / 127, 0.0)[:, 0]
    return s, y, np.rint(p * 127 / safe).astype(np.int64), scale


def linear(x, xs, w, ws, bias):
    """The values, the magnitude that roundings go by, and the largest sum of |products|."""
    x, w = x.astype(np.int64), w.astype(np.int64)
    scale = xs.astype(np.float64)[:, None] * ws.astype(np.float64)
    v = (x @ w.T) * scale
    b = np.zeros(len(w)) if bias is None else bias.astype(np.float64)
    most = np.abs(x) @ np.abs(w).T
    return v + b, np.abs(v) + np.abs(b), most


def seen_add(table, V, tokens, n, extra, fresh, prompt):
    """The new table (int16) as the definition has it, one token at a time."""
    t = table.copy()
    u = t.view(np.uint16)
    for r in range(len(t)):
        if fresh is not None and fresh[r]:
            u[r] = 0
        ids = [] if tokens is None else list(tokens[r][:len(tokens[r]) if n is None else n[r]])
        if extra is not None:
            ids.append(extra[r])
        for v in ids:
            if not 0 <= v < V:
                continue
            if prompt:
                u[r, v] |= 0x8000
            elif u[r, v] & 0x7FFF < 0x7FFF:
                u[r, v] += 1
    return t


def adjust(logits, seen, rep, pres, freq, tokens, biases, mask, mask_row, keep):
    """logits [R][S][V] float64; biases: per request a list of (token, value); mask: bool [M][V]. Returns the adjusted
    rows (others NaN) and the magnitude that roundings go by."""
    R, S, V = logits.shape
    out, mag = np.full(logits.shape, np.nan), np.zeros(logits.shape)
    for r in range(R):
        a, b, f = (float(x[r]) if x is not None else d for x, d in ((rep, 1.0), (pres, 0.0), (freq, 0.0)))
        n = np.zeros(V)
        known = np.zeros(V, bool)
        if seen is not None:
            word = seen[r, :V].view(np.uint16).astype(np.int64)
            n, known = (word & 0x7FFF).astype(np.float64), word >= 0x8000
        add, size = np.zeros(V), np.zeros(V)
        for v, x in (biases[r] if biases is not None else []):
            if 0 <= v < V:
                add[v] += x
                size[v] += abs(x) + abs(add[v])
        for j in range((S - 1 if keep is None else keep[r]) + 1):
            if j > 0 and tokens is not None and 0 <= tokens[r][j - 1] < V:
                n[tokens[r][j - 1]] += 1
            z = logits[r, j].copy()
            hit = known | (n > 0)
            z = np.where(hit, np.where(z > 0, z / a, z * a), z)
            with np.errstate(invalid="ignore"):
                mag[r, j] = np.abs(np.where(np.isfinite(z), z, 0)) + abs(f) * n + abs(b) * (n > 0) + size
            z = z - f * n - b * (n > 0) + add
            if mask is not None:
                m = r * S + j if mask_row is None else mask_row[r][j]
                if 0 <= m < len(mask):
                    z = np.where(mask[m], z, -np.inf)
            out[r, j] = z
    return out, mag


def pack_bits(allowed):
    """bool [M][V] as int32 words, bit v % 32 of word v / 32."""
    M, V = allowed.shape
    words = -(-V // 32)
    padded = np.zeros((M, words * 32), np.uint64)
    padded[:, :V] = allowed
    w = (padded.reshape(M, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)
