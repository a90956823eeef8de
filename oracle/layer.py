"""The operators around the experts in 64 bits (test infrastructure only): 8-bit
rows, RMS norm with the residual, the combine's gradient and the gated
feed-forward block, each from its definition and without the library."""

import numpy as np

from .numerics import bf16_to_f32, f32_to_bf16

# ------------------------------------------------------------------ 8-bit rows


def e4m3_table():
    """Value of each of the 256 e4m3 codes (sign, 4 exponent bits with bias 7, 3 mantissa bits; 0x7F is NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 0x7F) == 0x7F] = np.nan
    return np.where(c >= 128, -v, v)


def row_bytes(n):
    return (n + -(-n // 32) + 15) // 16 * 16


def block_exponent(a):
    """Smallest integer e with a <= 448 * 2^e, clamped to [-117, 120], for a block's largest finite magnitude."""
    if a == 0:
        return -117
    m, x = np.frexp(float(a))                      # a = m * 2^x
    return int(min(max(x - 9 if m <= 0.875 else x - 8, -117), 120))


def encode_e4m3(v):
    """Nearest code of values within +-448 (ties to even); NaN stays NaN (sign dropped)."""
    v = np.asarray(v, dtype=np.float64)
    out = np.full(v.shape, 0x7F, dtype=np.uint8)
    f = np.isfinite(v)
    a = np.abs(v[f])
    x = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    k = np.rint(a / 2.0 ** (x - 3))                # np.rint: ties to even
    up = k == 16                                   # rounded up into the next binade
    x, k = np.where(up, x + 1, x), np.where(up, 8, k)
    code = np.where(k >= 8, (x + 7) * 8 + (k - 8), k).astype(np.int64)
    out[f] = code + 128 * np.signbit(v[f])
    return out


def pack8(rows):
    """fp64 rows [T, n] -> uint8 [T, row_bytes(n)]."""
    T, n = rows.shape
    nb = -(-n // 32)
    out = np.zeros((T, row_bytes(n)), dtype=np.uint8)
    for t in range(T):
        for b in range(nb):
            v = rows[t, 32 * b:32 * b + 32]
            fin = np.isfinite(v)
            e = block_exponent(np.abs(v[fin]).max() if fin.any() else 0.0)
            out[t, 32 * b:32 * b + len(v)] = encode_e4m3(np.where(fin, v * 2.0 ** -e, np.nan))
            out[t, n + b] = e + 127
    return out


def unpack8(packed, n):
    """The values 8-bit rows stand for, fp64 [T, n]."""
    nb = -(-n // 32)
    s = 2.0 ** (packed[:, n:n + nb].astype(np.float64) - 127)
    return e4m3_table()[packed[:, :n]] * np.repeat(s, 32, axis=1)[:, :n]


# ------------------------------------------------------------------ norm

def stored_sum(x, residual, dtype):
    """x + residual as the row type stores it (fp32 addition, one rounding); bit patterns for bf16."""
    if dtype == "bf16":
        return f32_to_bf16((bf16_to_f32(x) + bf16_to_f32(residual)).astype(np.float32))
    return (x + residual).astype(np.float32)


def rms_norm(s, w, eps):
    s, w = np.asarray(s, np.float64), np.asarray(w, np.float64)
    r = 1 / np.sqrt((s * s).mean(1) + eps)
    return s * r[:, None] * w, r


def rms_norm_backward(dy, s, w, r, dsum=None):
    dy, s, w = (np.asarray(a, np.float64) for a in (dy, s, w))
    r = np.asarray(r, np.float64)[:, None]
    n, d = s * r, dy * w
    dx = r * (d - n * (d * n).mean(1, keepdims=True))
    return dx + (0 if dsum is None else np.asarray(dsum, np.float64)), (dy * n).sum(0)


# ------------------------------------------------------------------ experts

def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def dsilu(g):
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g))
    return s * (1 + g * (1 - s))


def ffn(x, wg, wu, wd):
    """One expert: (gate, up, h, y), all fp64."""
    g, u = x @ wg.T, x @ wu.T
    h = silu(g) * u
    return g, u, h, h @ wd.T


def ffn_backward(dy, x, g, u, wg, wu, wd):
    """One expert: dict of dh, dg, du, h, dx and the weight gradients, all fp64."""
    dh = dy @ wd
    dg, du, h = dh * u * dsilu(g), dh * silu(g), silu(g) * u
    return {"dh": dh, "dg": dg, "du": du, "h": h, "dx": dg @ wg + du @ wu, "dwg": dg.T @ x, "dwu": du.T @ x,
            "dwd": dy.T @ h}


def blocks(splits, rows):
    """(rank, expert, first row, rows) of every expert block: splits [N][N][E], rows of each rank's buffer."""
    N, _, E = splits.shape
    out = []
    for d in range(N):
        at = 0
        for e in range(E):
            n = int(np.maximum(splits[:, d, e], 0).sum())
            n = max(0, min(n, rows[d] - at))
            out.append((d, e, at, n))
            at += n
    return out
