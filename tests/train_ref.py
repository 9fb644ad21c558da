"""Plain implementations, in 64 bits, of what include/sdm_train.h defines: a route's
balance and its gradient, lookups with dropout, and the gradients to a bank; with
bounds on what float32 arithmetic may be off by."""

from __future__ import annotations

import numpy as np

from memory_ref import clean, live

U = 2.0 ** -24  # half a step of float32, relative

# ------------------------------------------------------------------ balance


def sequences(tokens, chunk, valid=None, chunk_valid=None, per_chunk=False):
    """For each sequence, its live tokens."""
    alive = np.flatnonzero(live(tokens, chunk, valid, chunk_valid))
    if not per_chunk:
        return [alive]
    return [alive[alive // chunk == g] for g in range(tokens // chunk)]


def shares(x, score):
    """A clean row's p, 1 - s (1 for a softmax), and how far a float32 p may be off, relative to it.

    An exponential of a is within (4 + 2 |a|) u of its value, and a itself, a difference, within |a| u. The
    row's sum adds at most 90 more in its additions (64 terms a lane, 6 steps over a wavefront, 16
    wavefronts with an exponential each), and of its terms' own errors their mean, weighted with p: |a| has
    the mean ln(1/p_max) + entropy <= 2 ln 65536 < 23. A sigmoid is one addition and a reciprocal (2 u) more.
    """
    if not (x > -np.inf).any():
        return np.zeros_like(x), np.ones_like(x), np.zeros_like(x)
    most = x.max()
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "softmax" or most <= -64:
            a = x - most
            e = np.exp(a)
            if score != "softmax":  # exp(most) is out of every s
                e = e / (1 + np.exp(x))
        else:
            a = np.minimum(x, 0)
            e = 1 / (1 + np.exp(-x))
        rest = 1 / (1 + np.exp(x)) if score == "sigmoid" else np.ones_like(x)
    a = np.where(x > -np.inf, np.abs(a), 0.0)
    return e / e.sum(), rest, (4 + 3 * np.minimum(a, 200) + 90 + 4 + 3 * 23 + 8) * U


def balance(logits, keys_of, *, score="softmax", chunk=None, valid=None, chunk_valid=None, per_chunk=False, scale=1.0):
    """(loss, counts, mean, coef), and the bounds of loss and mean. keys_of [T, k]: chosen keys (outside: none)."""
    X = clean(logits)
    T, N = X.shape
    k = keys_of.shape[1]
    runs = sequences(T, chunk or max(T, 1), valid, chunk_valid, per_chunk)
    some = sum(len(r) > 0 for r in runs)
    counts = np.zeros((len(runs), N), np.int64)
    mean, off = np.zeros((len(runs), N)), np.zeros((len(runs), N))
    coef = np.zeros(len(runs))
    loss = far = 0.0
    for g, run in enumerate(runs):
        for t in run:
            j = keys_of[t][(keys_of[t] >= 0) & (keys_of[t] < N)]
            np.add.at(counts[g], j, 1)
            p, _, rel = shares(X[t], score)
            mean[g] += p
            off[g] += p * (rel + 300 * U) + 2.0 ** -120  # 255 additions of a piece, and its rows' at its end
        if len(run):
            coef[g] = scale * N / (k * len(run) ** 2 * some)
            loss += coef[g] * (counts[g] * mean[g]).sum()
            far += abs(coef[g]) * (counts[g] * off[g]).sum()
            mean[g] /= len(run)
            off[g] = off[g] / len(run) + mean[g] * 2 * U
    return (loss, counts, mean, coef), (far + 2 * U * abs(loss), off)


def balance_backward(logits, counts, coef, *, dloss=1.0, score="softmax", chunk=None, valid=None, chunk_valid=None,
                     per_chunk=False):
    """(dlogits, bound). Counts are taken relative to their mean, or to that of a key with more than 4/5 of its row's
    share: what float32 sums of their products with the shares may be off by is relative to those differences."""
    X = clean(logits)
    T, N = X.shape
    out, off = np.zeros_like(X), np.zeros_like(X)
    for g, run in enumerate(sequences(T, chunk or max(T, 1), valid, chunk_valid, per_chunk)):
        f = dloss * float(coef[g])
        whole = counts[g].astype(np.float64)
        for t in run:
            x = X[t]
            p, rest, rel = shares(x, score)
            if not p.any():
                continue
            mean, top = np.trunc(whole.sum() / N), whole[x == x.max()].max()
            d = (whole - top) - (p * (whole - top)).sum()
            out[t] = p * rest * d * f
            with np.errstate(invalid="ignore"):
                more = rel + 12 * U + (np.minimum(np.where(x > -np.inf, np.abs(x), 0), 200) * 2 * U if score == "sigmoid" else 0)
            for c, there in ((whole - mean, p.max() < 0.81), (whole - top, p.max() > 0.79)):
                if there:
                    sums = (p * np.abs(c) * (rel + 110 * U)).sum()
                    size = np.abs(f) * p * rest * (np.abs(d) * more + sums + 4 * U * np.abs(c))
                    off[t] = np.maximum(off[t], size + np.abs(f) * (np.abs(d) + np.abs(c).max()) * 2.0 ** -120)
    return out, off


# ------------------------------------------------------------------ lookups


def philox(counter, key):
    """Philox4x32-10 of one counter, in Python's integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xffffffff, (a >> 32) ^ c[3] ^ k[1], a & 0xffffffff]
        k = [(k[0] + 0x9E3779B9) & 0xffffffff, (k[1] + 0xBB67AE85) & 0xffffffff]
    return c


def threshold(dropout):
    return int(np.rint(float(np.float32(dropout)) * 65536))


def factor(scale, dropout):
    """What a kept value is multiplied by, as float32."""
    return np.float32(float(np.float32(scale)) * 65536 / (65536 - threshold(dropout)))


def kept(n, head_dim, dropout, rng):
    """[n, head_dim] truth values."""
    t = threshold(dropout)
    out = np.ones((n, head_dim), bool)
    if t == 0:
        return out
    seed, offset = (int(v) & 0xffffffffffffffff for v in rng)
    key, high = (seed & 0xffffffff, seed >> 32), (offset & 0xffffffff, offset >> 32)
    for i in range(n):
        for o in range(-(-head_dim // 8)):
            words = philox((o, i) + high, key)
            for j in range(min(8, head_dim - 8 * o)):
                out[i, 8 * o + j] = (words[j // 2] >> (16 * (j % 2))) & 0xffff >= t
    return out


def lookup(values, idx, scale=1.0, mask=None, dropout=0.0):
    """float32 [n, head_dim] of float32 values: one product, rounded."""
    idx = np.asarray(idx, np.int64)
    ok = (idx >= 0) & (idx < len(values))
    with np.errstate(over="ignore", invalid="ignore"):
        rows = values[np.where(ok, idx, 0)].astype(np.float32) * factor(scale, dropout)
    keep = ok[:, None] if mask is None else ok[:, None] & mask
    return np.where(keep, rows, np.float32(0))


def bank_grad(num_slots, slots, terms, head_dim):
    """(sums, sums of magnitudes, terms of each slot) of terms(i) [head_dim] for entry i; slots outside: none."""
    out, size = np.zeros((num_slots, head_dim)), np.zeros((num_slots, head_dim))
    count = np.zeros(num_slots, np.int64)
    at = np.flatnonzero((slots >= 0) & (slots < num_slots))
    for a in range(0, len(at), 4096):
        e = at[a:a + 4096]
        v = terms(e)
        np.add.at(out, slots[e], v)
        np.add.at(size, slots[e], np.abs(v))
        np.add.at(count, slots[e], 1)
    return out, size, count
