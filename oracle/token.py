"""Oracle of the two ends of a training step in 64 bits: token embedding and its
gradient, dropout with its counter-based generator, and the log probabilities of
given tokens with entropy, alternatives and gradient.  Arrays are numpy, values
float64; the formulas follow the operators' definitions, not their kernels."""

import numpy as np

M32 = np.uint64(0xFFFFFFFF)


# ------------------------------------------------------------------ embedding

def embedding(weight, tokens, scale=1.0):
    """Rows of weight [V, H] for tokens [T], times scale; zeros for tokens outside [0, V)."""
    out = np.zeros((len(tokens), weight.shape[1]))
    ok = (tokens >= 0) & (tokens < weight.shape[0])
    out[ok] = weight[tokens[ok]] * scale
    return out


def embedding_backward(dout, tokens, vocab, scale=1.0):
    """(gradient [V, H], the same sums of magnitudes, number of terms of each row)."""
    g, mag = np.zeros((vocab, dout.shape[1])), np.zeros((vocab, dout.shape[1]))
    n = np.zeros(vocab, dtype=np.int64)
    ok = (tokens >= 0) & (tokens < vocab)
    np.add.at(g, tokens[ok], dout[ok] * scale)
    np.add.at(mag, tokens[ok], np.abs(dout[ok] * scale))
    np.add.at(n, tokens[ok], 1)
    return g, mag, n


# ------------------------------------------------------------------ dropout

def philox4x32(counter, key, rounds=10):
    """The generator of Salmon et al. (SC 2011): counter [..., 4] and key (2) as 32-bit values in uint64."""
    c = [np.asarray(counter[..., i], dtype=np.uint64) for i in range(4)]
    k0, k1 = np.uint64(key[0]), np.uint64(key[1])
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ k0, b & M32, (a >> np.uint64(32)) ^ c[3] ^ k1, a & M32]
        k0, k1 = (k0 + np.uint64(0x9E3779B9)) & M32, (k1 + np.uint64(0xBB67AE85)) & M32
    return np.stack(c, axis=-1)


def drop_steps(p):
    """p in steps of 2^-16."""
    return int(np.floor(np.float64(np.float32(p)) * 65536 + 0.5))


def keep(n, rank, p, seed, at):
    """Which of a rank's n elements stay; at = offset + step."""
    b = np.arange((n + 7) // 8, dtype=np.uint64)
    at = np.uint64(at % (1 << 64))
    counter = np.stack([b & M32, (b >> np.uint64(32)) | np.uint64(rank << 8), np.full_like(b, at & M32),
                        np.full_like(b, at >> np.uint64(32))], axis=-1)
    words = philox4x32(counter, (seed & 0xFFFFFFFF, seed >> 32))
    halves = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], axis=-1).reshape(-1)
    return halves[:n] >= np.uint64(drop_steps(p))


def dropout(x, rank, p, seed, at, residual=None):
    d = drop_steps(p)
    y = np.where(keep(x.size, rank, p, seed, at).reshape(x.shape), x * (65536.0 / (65536 - d) if d < 65536 else 0.0), 0.0)
    return y if residual is None else y + residual


# ------------------------------------------------------------------ log probabilities

def log_softmax(x, scale=1.0):
    """(log p [T, V], lse [T]) of scale * x; a row of -inf gives -inf everywhere, NaN or +inf a row of NaN."""
    with np.errstate(all="ignore"):
        z = x * scale
        m = np.max(z, axis=1, keepdims=True)
        base = np.where(np.isneginf(m), 0.0, m)
        s = np.exp(z - base).sum(1, keepdims=True)
        log_s = np.log(s)
        lse = base + log_s
        return np.where(np.isneginf(lse), -np.inf, z - base - log_s), lse[:, 0]   # lse would round log_s beside a large base


def entropy(lp):
    with np.errstate(all="ignore"):
        p = np.exp(lp)
        return -np.where(p > 0, p * lp, np.where(np.isnan(p), np.nan, 0.0)).sum(1)


def token_logprob(lp, targets):
    T, V = lp.shape
    ok = (targets >= 0) & (targets < V)
    return np.where(ok, lp[np.arange(T), np.where(ok, targets, 0)], 0.0)


def alternatives(x, lp, k):
    """Tokens of the k largest logits per row (equal values: lowest token first; NaN never, -1 where none is left)
    and their log probabilities."""
    ids = np.full((x.shape[0], k), -1, dtype=np.int64)
    val = np.full((x.shape[0], k), -np.inf)
    for r, row in enumerate(x):
        some = np.nonzero(~np.isnan(row))[0]
        order = some[np.argsort(-row[some], kind="stable")][:k]
        ids[r, :len(order)] = order
        val[r, :len(order)] = lp[r, order]
        if np.isnan(lp[r]).any():
            val[r] = np.nan
    return ids, val


def token_logprob_backward(x, targets, lse, dlogprob, scale=1.0, ent=None, dentropy=None):
    """Gradient of the logits from a given lse (and entropy)."""
    T, V = x.shape
    with np.errstate(all="ignore"):
        d = x * scale - lse[:, None]
        some = ~np.isneginf(lse)
        p = np.where(some[:, None], np.exp(d), 0.0)
        ok = (targets >= 0) & (targets < V) & some
        g = np.where(ok, dlogprob, 0.0)
        dz = -g[:, None] * p
        dz[np.arange(T), np.where(ok, targets, 0)] += g
        if dentropy is not None:
            dz -= dentropy[:, None] * np.where(p == 0, 0.0, p * (d + ent[:, None]))
        return dz * scale
