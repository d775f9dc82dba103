"""fp64 oracles of the router's balance loss and of 4-bit MX matrices, in plain
NumPy from the definitions; they share no code with the GPU path."""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


# ------------------------------------------------------------------ balance loss

def counted(logits, mask=None):
    """Rows that count: not masked, at least one logit above -infinity (NaN counts as one)."""
    keep = ~np.all(np.isneginf(logits), axis=1)
    return keep if mask is None else keep & (np.asarray(mask) != 0)


def balance(logits, idx, mask=None):
    """(stats [4], counts [E], prob [E]) in fp64."""
    T, E = logits.shape
    k = idx.shape[1]
    rows = np.nonzero(counted(logits, mask))[0]
    n = rows.size
    counts = np.zeros(E, dtype=np.int64)
    if n == 0:
        return np.zeros(4), counts, np.zeros(E)
    ok = idx[rows].reshape(-1)
    ok = ok[(ok >= 0) & (ok < E)]
    np.add.at(counts, ok, 1)
    l = logits[rows].astype(np.float64)
    m = l.max(1, keepdims=True)
    ex = np.exp(l - m)
    s = ex.sum(1, keepdims=True)
    prob = (ex / s).sum(0) / n
    lse = (m + np.log(s))[:, 0]
    f = counts * E / (k * n)
    return np.array([(f * prob).sum(), (lse ** 2).sum() / n, n, f.max()]), counts, prob


def balance_grad(logits, idx, gate, mask, d_loss, d_gate, renorm):
    """d_logits [T, E] by the formula, and the magnitude its terms have (for error bounds)."""
    T, E = logits.shape
    k = idx.shape[1]
    _, counts, _ = balance(logits, idx, mask)
    keep = counted(logits, mask)
    n = keep.sum()
    out = np.zeros((T, E))
    size = np.zeros((T, E))
    for t in np.nonzero(keep)[0]:
        l = logits[t].astype(np.float64)
        m = l.max()
        p = np.exp(l - m)
        s = p.sum()
        p /= s
        a = d_loss[0] * E / (k * n * n)
        z = d_loss[1] * 2 / n * (m + np.log(s))
        out[t] = p * (a * (counts - (counts * p).sum()) + z)
        size[t] = p * (abs(a) * (counts + (counts * p).sum()) + abs(z))
        if d_gate is not None:
            g, dg = gate[t].astype(np.float64), d_gate[t].astype(np.float64)
            ok = (idx[t] >= 0) & (idx[t] < E)  # a choice that names no expert takes no part
            mean = (g * dg)[ok].sum()
            mag = (g * abs(dg))[ok].sum()
            if not renorm:
                out[t] -= p * mean
                size[t] += p * mag
            for j in range(k):
                e = idx[t, j]
                if 0 <= e < E:
                    out[t, e] += g[j] * (dg[j] - (mean if renorm else 0))
                    size[t, e] += g[j] * (abs(dg[j]) + mag)
    return out, size


def balance_total(logits, idx, mask, d_loss, d_gate, renorm):
    """The scalar that balance_grad differentiates, the counts held fixed."""
    stats, _, _ = balance(logits, idx, mask)
    total = d_loss[0] * stats[0] + d_loss[1] * stats[1]
    if d_gate is not None:
        for t in np.nonzero(counted(logits, mask))[0]:
            l = logits[t].astype(np.float64)
            e = np.exp(l - l.max())
            g = e[idx[t]] / (e[idx[t]].sum() if renorm else e.sum())
            total += (g * d_gate[t]).sum()
    return total


# ------------------------------------------------------------------ MX matrices

def pitch(cols):
    return -(-(cols // 32) // 16) * 16


def mx4_quantize(x):
    """x [rows, cols] (any float type) -> codes [rows, cols/2], scales [rows, pitch] (uint8)."""
    rows, cols = x.shape
    with np.errstate(invalid="ignore"):  # signalling NaN
        v = np.asarray(x, dtype=np.float64).reshape(rows, cols // 32, 32)
    q = np.zeros(v.shape, dtype=np.uint8)
    sc = np.zeros((rows, pitch(cols)), dtype=np.uint8)
    for r in range(rows):
        for b in range(cols // 32):
            blk = v[r, b]
            if not np.all(np.isfinite(blk)):
                sc[r, b] = 255
                continue
            top = np.abs(blk).max()
            e = -127 if top == 0 else int(np.clip(np.frexp(top)[1] - 1 - 2, -127, 127))
            sc[r, b] = e + 127
            a = np.ldexp(np.abs(blk), -e)
            d = np.abs(a[:, None] - LEVELS[None, :])
            near = d == d.min(1, keepdims=True)
            # of two equally near levels the one with an even code
            best = np.array([min((i for i in range(8) if near[j, i]), key=lambda i: (i & 1, i)) for j in range(32)])
            q[r, b] = best | (np.signbit(blk).astype(np.uint8) << 3)
    q = q.reshape(rows, cols)
    return q[:, 0::2] | (q[:, 1::2] << 4), sc


def mx4_values(codes, scales):
    """The fp64 values of codes [rows, cols/2] and scales."""
    rows, half = codes.shape
    q = np.empty((rows, 2 * half), dtype=np.uint8)
    q[:, 0::2] = codes & 15
    q[:, 1::2] = codes >> 4
    v = LEVELS[q & 7] * np.where(q & 8, -1.0, 1.0)
    s = scales[:, :2 * half // 32].astype(np.float64)
    f = np.where(s == 255, np.nan, np.exp2(s - 127))
    return v * np.repeat(f, 32, axis=1)
