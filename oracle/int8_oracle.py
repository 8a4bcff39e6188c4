"""Float64 definitions of routing with scores and of the int8 expert products (numpy, one
row or one expert at a time).  Test infrastructure only."""
from __future__ import annotations

import numpy as np


def route(logits, k, score="softmax", bias=None, n_groups=1, top_groups=1, group_rank="max", renormalize=True,
          scale=1.0):
    """ids [T][k] int32 and weights [T][k] float64 of logits [T][E].  Scores that decide
    are doubles; weights are taken from scores in long double, whose exponents reach
    further, unless the chosen doubles sum to 0."""
    l = np.array(logits, dtype=np.float64)
    l[np.isnan(l)] = -np.inf
    T, E = l.shape
    size = E // n_groups
    ids = np.zeros((T, k), np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        row = l[t]
        with np.errstate(over="ignore", invalid="ignore"):
            wide = row.astype(np.longdouble)
            if score == "sigmoid":
                s = np.where(row < -700, np.exp(row), 1.0 / (1.0 + np.exp(-row)))
                wide = 1 / (1 + np.exp(-wide))
            elif np.all(row == -np.inf):
                s = wide = np.zeros(E)
            else:
                z = np.where(row == row.max(), 1.0, np.exp(row - row.max()))
                s = z / z.sum()
                wide = np.where(row == row.max(), np.longdouble(1), np.exp(wide - wide.max()))
                wide = wide / wide.sum()
            c = row.copy() if bias is None else s + np.asarray(bias, np.float64)
        c[np.isnan(c)] = -np.inf
        chosen = []
        for g in range(n_groups):
            part = c[g * size:(g + 1) * size] if bias is not None or group_rank == "max" else s[g * size:(g + 1) * size]
            two = sorted(part, reverse=True)[:2]
            with np.errstate(invalid="ignore"):
                v = sum(two) if group_rank == "top2" else two[0]
            chosen.append((-np.inf if np.isnan(v) else v, -g))
        kept = {-g for _, g in sorted(chosen, reverse=True)[:top_groups]}
        allowed = [e for e in range(E) if e // size in kept]
        order = sorted(allowed, key=lambda e: (-c[e], e))[:k]
        ids[t] = order
        w[t] = wide[order]
        if renormalize:
            w[t] = wide[order] / wide[order].sum() if s[order].sum() > 0 else 0.0
    return ids, w * float(np.float32(scale))


def quantize(v):
    """Codes (int64) and float32 scales of the last axis of v."""
    v = np.asarray(v, np.float64)
    flat = v.reshape(-1, v.shape[-1])
    q = np.zeros(flat.shape, np.int64)
    s = np.ones(flat.shape[0], np.float32)
    for r, row in enumerate(flat):
        if not np.all(np.isfinite(row)):
            s[r] = np.nan
            continue
        a = np.float32(np.abs(row).max()) * (np.float32(1.0) / np.float32(127.0))
        s[r] = a if a > 0 else np.float32(1.0)
        q[r] = np.clip(np.rint(row / np.float64(s[r])), -127, 127).astype(np.int64)
    return q.reshape(v.shape), s.reshape(v.shape[:-1])


def group_expert(g, E, nseg):
    return g % E if g < nseg * E else E + g - nseg * E


def _dot(q, w):
    """Sums of products of codes (exact: integers below 2^53)."""
    return np.asarray(q, np.float64) @ np.asarray(w, np.float64).T


def grouped_linear(xq, xs, rows, offs, E, nseg, w, ws):
    """y [N][O] float64; rows of no group are NaN."""
    y = np.full((len(rows), w.shape[1]), np.nan)
    for g in range(len(offs) - 1):
        r = np.asarray(rows[offs[g]:offs[g + 1]], np.int64)
        if len(r):
            e = group_expert(g, E, nseg)
            y[offs[g]:offs[g + 1]] = _dot(xq[r], w[e]) * xs[r].astype(np.float64)[:, None] * ws[e].astype(np.float64)
    return y


def grouped_ffn(x, rows, offs, E, nseg, wg, sg, wu, su, wd, sd, block=128, margin=0.0):
    """h [N][d] float64 of token rows x [T][d], and what it can move by if every
    code whose quotient lies within `margin` of a border between two codes falls on
    the other side.  Rows of no group are NaN."""
    xq, xs = quantize(x)
    h = np.full((len(rows), wd.shape[1]), np.nan)
    slack = np.zeros_like(h)
    I = wg.shape[1]
    for g in range(len(offs) - 1):
        e = group_expert(g, E, nseg)
        r = np.asarray(rows[offs[g]:offs[g + 1]], np.int64)
        if not len(r):
            continue
        sx = xs[r].astype(np.float64)[:, None]
        gate = _dot(xq[r], wg[e]) * sx * sg[e].astype(np.float64)
        up = _dot(xq[r], wu[e]) * sx * su[e].astype(np.float64)
        with np.errstate(over="ignore", invalid="ignore"):
            a = gate / (1.0 + np.exp(-gate)) * up
        acc = np.zeros((len(r), wd.shape[1]))
        loose = np.zeros_like(acc)
        for b in range(0, I, block):
            q, s = quantize(a[:, b:b + block])
            s = s.astype(np.float64)[:, None]
            acc += _dot(q, wd[e][:, b:b + block]) * s
            v = np.abs(a[:, b:b + block] / s)
            near = np.abs(v - np.floor(v) - 0.5) < margin
            loose += _dot(near, np.abs(wd[e][:, b:b + block].astype(np.float64))) * s
        h[offs[g]:offs[g + 1]] = acc * sd[e].astype(np.float64)
        slack[offs[g]:offs[g + 1]] = loose * sd[e].astype(np.float64)
    return h, slack


def grouped_ffn_magnitude(x, rows, offs, E, nseg, wg, sg, wu, su, wd, sd, block=128):
    """The sums that grouped_ffn's outputs are made of, with every term's magnitude."""
    xq, xs = quantize(x)
    m = np.full((len(rows), wd.shape[1]), np.nan)
    for g in range(len(offs) - 1):
        e = group_expert(g, E, nseg)
        r = np.asarray(rows[offs[g]:offs[g + 1]], np.int64)
        if len(r):
            sx = xs[r].astype(np.float64)[:, None]
            gate, up = _dot(xq[r], wg[e]) * sx * sg[e], _dot(xq[r], wu[e]) * sx * su[e]
            with np.errstate(over="ignore", invalid="ignore"):
                a = np.abs(gate / (1.0 + np.exp(-gate)) * up)
            m[offs[g]:offs[g + 1]] = _dot(a, np.abs(wd[e].astype(np.float64))) * sd[e]
    return m
