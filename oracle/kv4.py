"""The 4-bit key/value cache and the log probabilities, written as their definitions in float64.

ORACLE -- test infrastructure only; shares no code with the library.

A page's block of one head (64 tokens, head size D) is described value by
value: where the code and the scale of token t, position d lie.
"""

import numpy as np

from .formats import e2m1_decode, e2m1_encode, e4m3_decode, e4m3_encode

PAGE = 64


def kv_quantize(x, g):
    """x [..., D] -> (codes [..., D] of 0..15, scales [..., D / 16] bytes)."""
    w = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], -1, 16)
    amax = np.abs(w).max(-1)
    nan = np.isnan(w).any(-1)
    scales = e4m3_encode(np.minimum(np.where(nan, 0.0, amax) / (6.0 * float(g)), 448.0))
    unit = (e4m3_decode(scales) * float(g))[..., None]
    ok = (unit > 0) & ~nan[..., None]
    with np.errstate(invalid="ignore", over="ignore"):
        ratio = np.where(ok, w / np.where(ok, unit, 1.0), 0.0)
    ratio = np.clip(ratio, -6.0, 6.0)
    codes = np.where(ok, e2m1_encode(ratio), 0).astype(np.uint8)
    return codes.reshape(np.shape(x)), np.where(nan, 0x7F, scales).astype(np.uint8)


def kv_places(D):
    """For [64, D]: (K byte, V byte, nibble, K scale byte, V scale byte) of every value of a block."""
    t, d = np.arange(PAGE)[:, None], np.arange(D)[None, :]
    q, i = d // (D // 4), d % (D // 4)
    run = t // 16 * (D // 8) + i // 2
    k = run // 16 * 1024 + q * 256 + t % 16 * 16 + run % 16
    ks = 32 * D + (q * 16 + t % 16) * (D // 16) + t // 16 * (D // 64) + i // 16
    c, i = d // (D // 16), d % (D // 16)
    o = t // 16 * 4 + t % 4
    run = o * (D // 32) + i // 2
    v = 36 * D + run // 16 * 1024 + t % 16 // 4 * 256 + c * 16 + run % 16
    vs = 68 * D + d // 16 * 64 + t % 16 // 4 * 16 + o
    return k, v, np.broadcast_to(d % 2, (PAGE, D)), ks, vs


def kv_values(block, D, gk, gv):
    """K and V [64, D] of a block [72 * D]."""
    k, v, nib, ks, vs = kv_places(D)
    with np.errstate(invalid="ignore"):
        return tuple(e2m1_decode(block[at] >> (4 * nib) & 15) * e4m3_decode(block[sc]) * float(g)
                     for at, sc, g in ((k, ks, gk), (v, vs, gv)))


def kv_put(block, t, kcodes, kscales, vcodes, vscales):
    """Writes token t's codes [D] and scales [D / 16] into a block in place."""
    D = len(kcodes)
    k, v, nib, ks, vs = kv_places(D)
    for at, codes in ((k[t], kcodes), (v[t], vcodes)):
        for d in range(D):
            block[at[d]] = (block[at[d]] & (0xF0 if nib[t, d] == 0 else 0x0F)) | (codes[d] << (4 * nib[t, d]))
    block[ks[t][::16]] = kscales
    block[vs[t][::16]] = vscales


def kv_held(cache, row, n, h, D, gk=1.0, gv=1.0):
    """(K, V [n, D], held [n]) of the first n slots of a sequence whose table row is `row`."""
    ks, vs, held = [], [], []
    for p in row[:-(-n // PAGE)]:
        good = 0 <= p < len(cache)
        k, v = kv_values(cache[p, h], D, gk, gv) if good else (np.zeros((PAGE, D)), np.zeros((PAGE, D)))
        ks.append(k), vs.append(v), held.append(np.full(PAGE, good))
    if not ks:
        return np.zeros((0, D)), np.zeros((0, D)), np.zeros(0, bool)
    return np.concatenate(ks)[:n], np.concatenate(vs)[:n], np.concatenate(held)[:n]


def kv_attend(q, k, v, held, limit, scale):
    """One row: (out, lse, weights [n], sum of p|v| / sum p) over the held slots below limit."""
    n = len(k)
    see = held & (np.arange(n) < limit)
    p = np.zeros(n)
    if not see.any():
        return np.zeros(len(q)), -np.inf, p, np.zeros(len(q))
    x = scale * (k[see] @ q)
    m = x.max()
    e = np.exp(x - m)
    p[see] = e / e.sum()
    return p[see] @ v[see], m + np.log(e.sum()), p, p[see] @ np.abs(v[see])


def kv_evict(acc, n, keep, sinks, recent):
    """The slots kept of n, in order."""
    if n <= keep:
        return np.arange(n)
    w = np.where(np.isnan(acc[:n]), -np.inf, acc[:n].astype(np.float64))
    nan = np.isnan(acc[:n])
    sure = (np.arange(n) < sinks) | (np.arange(n) >= n - recent)
    order = sorted(range(n), key=lambda s: (not sure[s], nan[s], -w[s], s))
    return np.array(sorted(order[:keep]))


def logprobs(x, token, k):
    """One row of float64 logits: (logprob, entropy, top ids, top logprobs).

    Everything is taken about the maximum: x - m stays exact where m + log S would swallow log S."""
    x = np.asarray(x, np.float64)
    ids = sorted(range(len(x)), key=lambda i: (np.isnan(x[i]), -x[i] if x[i] == x[i] else 0, i))
    ids = [i for i in ids[:k] if x[i] == x[i]]
    ids += [-1] * (k - len(ids))
    m, log, entropy = 0.0, 0.0, 0.0
    if np.isnan(x).any() or (x == np.inf).any():
        log = entropy = np.nan
    elif (x > -np.inf).any():
        m = x.max()
        e = np.exp(x - m)
        log = np.log(e.sum())
        p = e / e.sum()
        entropy = -(p[p > 0] * (x[p > 0] - m - log)).sum()
    lp = x[token] - m - log if 0 <= token < len(x) else np.nan
    return lp, entropy, np.array(ids), np.array([x[i] - m - log if i >= 0 else np.nan for i in ids])
