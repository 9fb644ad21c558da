"""Plain implementations, in 64 bits, of what include/sdm_memory.h defines: the
route and its gradient, packing, and a gather with its weights' gradient."""

from __future__ import annotations

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)
BLOCK = 32

# ------------------------------------------------------------------ route


def clean(logits) -> np.ndarray:
    x = np.asarray(logits, dtype=np.float64)
    return np.minimum(np.where(np.isnan(x), -np.inf, x), FLT_MAX)


def _eligible(x, bias):
    ok = x > -np.inf
    return ok if bias is None else ok & (np.asarray(bias, dtype=np.float64) > -np.inf)  # NaN: False


def scores(x: np.ndarray, score: str) -> np.ndarray:
    """Scores of one row of clean logits."""
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-x))
    top = max(float(x.max()), -FLT_MAX)
    e = np.exp(x - top)
    return e / e.sum() if e.sum() > 0 else np.zeros_like(x)


def _top(values, keys, k):
    """The k keys of largest value, descending, the lowest key first among equals."""
    order = sorted(range(len(keys)), key=lambda i: (-values[i], keys[i]))
    return [keys[i] for i in order[:k]]


def _weights(x, s, ok, chosen, score, normalise):
    """u_j / U (or u_j) of the chosen keys of one row, and U's place taken by 1 where it is 0."""
    ok = ok[chosen]
    if not normalise:
        return np.where(ok, s[chosen], 0.0)
    if score == "softmax":  # up to the row's factor, from the chosen keys' own largest
        at = np.where(ok, x[chosen], -np.inf)
        u = np.exp(at - max(float(at.max()), -FLT_MAX))
    else:
        u = np.where(ok, s[chosen], 0.0)
    return u / u.sum() if u.sum() > 0 else np.zeros_like(u)


def route(logits, k, *, score="softmax", bias=None, groups=1, kept=None, top=1, normalise=False, scale=1.0):
    """(keys [T, k], weights [T, k])."""
    X = clean(logits)
    kept = groups if kept is None else kept
    N = X.shape[1]
    size = N // groups
    out_k, out_w = [], []
    for x in X:
        ok, s = _eligible(x, bias), scores(x, score)
        c = np.where(ok, s if bias is None else s + np.nan_to_num(np.asarray(bias, np.float64), nan=0.0,
                                                                posinf=np.inf, neginf=-np.inf), -np.inf)
        keys = range(N)
        if groups > 1:
            worth = []
            for g in range(groups):
                best = np.sort(c[g * size:(g + 1) * size])[::-1][:top]
                best = best[best > -np.inf]
                worth.append(best.sum() if len(best) else -np.inf)
            keep = set(_top(worth, list(range(groups)), kept))
            keys = [i for i in range(N) if i // size in keep]
        v = np.where(ok, x, -np.inf) if bias is None else c
        chosen = _top(list(v[list(keys)]), list(keys), k)
        out_k.append(chosen)
        out_w.append(scale * _weights(x, s, ok, chosen, score, normalise))
    return np.array(out_k).reshape(len(X), k), np.array(out_w).reshape(len(X), k)


def route_backward(logits, keys, dw, *, score="softmax", bias=None, normalise=False, scale=1.0):
    """(dlogits [T, N], the size of the terms that its cancellations leave [T, N])."""
    X = clean(logits)
    out, size = np.zeros_like(X), np.zeros_like(X)
    for t, x in enumerate(X):
        ok, s = _eligible(x, bias), scores(x, score)
        j = [(i, key) for i, key in enumerate(keys[t]) if 0 <= key < len(x) and ok[key]]
        at, d = [key for _, key in j], np.array([float(dw[t][i]) for i, _ in j])
        if not j:
            continue
        if normalise:
            w = _weights(x, s, ok, at, score, True)
            f = scale * w
            if score == "sigmoid":  # 1 - s
                f = scale * w * scores(-x[at], "sigmoid")
            np.add.at(out[t], at, f * (d - (d * w).sum()))
            np.add.at(size[t], at, f * (np.abs(d) + np.abs(d * w).sum()))
        elif score == "sigmoid":
            f = scale * s[at] * scores(-x[at], "sigmoid")
            np.add.at(out[t], at, f * d)
            np.add.at(size[t], at, np.abs(f * d))
        else:
            du, mag = np.zeros_like(x), np.zeros_like(x)
            np.add.at(du, at, scale * d)
            np.add.at(mag, at, abs(scale) * np.abs(d))
            out[t] = s * (du - (scale * d * s[at]).sum())
            size[t] = s * (mag + (abs(scale) * np.abs(d) * s[at]).sum())
    return out, size


# ------------------------------------------------------------------ packed rows

E4M3 = [(b % 8 / 8 + (b // 8 > 0)) * 2.0 ** (max(b // 8, 1) - 7) for b in range(127)]
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def row_bytes(head_dim, kind):
    n = head_dim if kind == "mx8" else (head_dim + 1) // 2
    return (n + 15) // 16 * 16


def scale_bytes(head_dim):
    return ((head_dim + BLOCK - 1) // BLOCK + 3) // 4 * 4


def nearest(a: np.ndarray, table) -> np.ndarray:
    """The index of the table's nearest value to each a >= 0 (at most its largest), ties to even indexes."""
    t = np.array(table)
    low = np.clip(np.searchsorted(t, a, side="right") - 1, 0, len(t) - 2)
    below, above = a - t[low], t[low + 1] - a
    return low + ((above < below) | ((above == below) & (low % 2 == 1)))


def pack(rows: np.ndarray, kind: str):
    """(codes [n, row_bytes], scales [n, scale_bytes]) of float32 rows."""
    n, hd = rows.shape
    table, most = (E4M3, 448.0) if kind == "mx8" else (E2M1, 6.0)
    codes = np.zeros((n, row_bytes(hd, kind)), np.uint8)
    scales = np.zeros((n, scale_bytes(hd)), np.uint8)
    half = np.zeros((n, hd + hd % 2), np.uint8)
    for b in range(0, hd, BLOCK):
        x = rows[:, b:b + BLOCK].astype(np.float64)
        fin = np.isfinite(x)
        a = np.where(fin, np.abs(x), 0.0)
        top = a.max(1)
        e = np.full(n, -127)
        for i in range(n):
            while e[i] < 127 and top[i] > most * 2.0 ** int(e[i]):
                e[i] += 1
        code = nearest(a / np.exp2(e.astype(np.float64))[:, None], table).astype(np.uint8)
        neg = np.signbit(x)
        if kind == "mx8":
            codes[:, b:b + x.shape[1]] = np.where(fin, code | (neg.astype(np.uint8) << 7), 0x7f)
            scales[:, b // BLOCK] = e + 127
        else:
            whole = fin.all(1)
            half[:, b:b + x.shape[1]] = np.where(whole[:, None], code | (neg.astype(np.uint8) << 3), 0)
            scales[:, b // BLOCK] = np.where(whole, e + 127, 255)
    if kind == "mx4":
        both = half[:, 0::2] | (half[:, 1::2] << 4)
        codes[:, :both.shape[1]] = both
    return codes, scales


def unpack(codes: np.ndarray, scales: np.ndarray, head_dim: int, kind: str) -> np.ndarray:
    """float64 values [n, head_dim]."""
    if kind == "mx8":
        v = np.array(E4M3 + [np.nan] + [-a for a in E4M3] + [np.nan])[codes[:, :head_dim]]
    else:
        c = np.arange(head_dim)
        v = np.array(E2M1 + [-a for a in E2M1])[(codes[:, c // 2] >> (c % 2 * 4).astype(np.uint8)) & 15]
    s = scales[:, np.arange(head_dim) // BLOCK].astype(np.float64)
    return np.ascontiguousarray(v * np.where(s == 255, np.nan, np.exp2(s - 127)))


# ------------------------------------------------------------------ gather


def live(tokens, chunk, valid=None, chunk_valid=None) -> np.ndarray:
    t = np.arange(tokens)
    return t % chunk < (np.asarray(chunk_valid)[t // chunk] if chunk_valid is not None else
                        chunk if valid is None else valid)


def weight_grad(bank: np.ndarray, idx, dout, alive):
    """(dw, sum of the terms' magnitudes), [tokens, width], in float64."""
    dw = np.zeros(idx.shape)
    size = np.zeros(idx.shape)
    for t in np.flatnonzero(alive):
        terms = bank[idx[t]] * np.asarray(dout[t], np.float64)[None]
        dw[t], size[t] = terms.sum(1), np.abs(terms).sum(1)
    return dw, size
