"""Float64 definitions of the root-mean-square norm and of the block-scaled E4M3 products (numpy, one
row or one expert at a time).  Codes appear as the values they stand for.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

from .int8_oracle import group_expert
from .moe_oracle import bf16_bits_to_f64, f64_to_bf16_bits

BLOCK = 128
F32 = np.float32


def e4m3_step(v):
    """Distance of the E4M3 values around |v|: 2^(e - 3) in [2^e, 2^(e + 1)), 2^-9 below 2^-6."""
    e = np.frexp(np.asarray(v, np.float64))[1] - 1
    return np.ldexp(1.0, np.maximum(e, -6) - 3)


def e4m3(v):
    """The nearest E4M3 value, halves to the even code; |v| <= 448."""
    v = np.asarray(v, np.float64)
    step = e4m3_step(v)
    return np.rint(v / step) * step


def quantize_blocks(v):
    """Code values [..][d] and float32 scales [..][ceil(d / 128)] of fp32 values v [..][d]."""
    v = np.asarray(v, F32)
    d = v.shape[-1]
    flat = v.reshape(-1, d)
    nb = -(-d // BLOCK)
    q = np.zeros(flat.shape)
    s = np.ones((flat.shape[0], nb), F32)
    c = F32(1.0) / F32(448.0)
    for r, row in enumerate(flat):
        for b in range(nb):
            part = row[b * BLOCK:(b + 1) * BLOCK]
            if not np.all(np.isfinite(part)):
                s[r, b] = np.nan
                continue
            a = np.abs(part).max() * c
            if a >= F32(2.0 ** -100):
                s[r, b] = a
            quotient = (part.astype(np.float64) / np.float64(s[r, b])).astype(F32)
            q[r, b * BLOCK:(b + 1) * BLOCK] = e4m3(quotient)
    return q.reshape(v.shape), s.reshape(*v.shape[:-1], nb)


def residual_sum(x, residual, bf16):
    """x + residual in fp32, rounded to the residual's type; inputs as fp32 values, fp32 values out."""
    with np.errstate(over="ignore", invalid="ignore"):
        r = np.asarray(x, F32) + np.asarray(residual, F32)
    return bf16_bits_to_f64(f64_to_bf16_bits(r)).astype(F32) if bf16 else r


def rmsnorm(r, w, eps):
    """1 / sqrt(mean r^2 + eps) [T] and r * w [T][d] as fp32 products, of fp32 rows and weights."""
    r, w = np.asarray(r, F32), np.asarray(w, F32)
    out = np.zeros(len(r))
    with np.errstate(over="ignore", invalid="ignore"):
        for t, row in enumerate(r.astype(np.float64)):
            m = np.sum(row * row)
            out[t] = 1.0 / np.sqrt(m / r.shape[1] + float(F32(eps))) if m < 2.0 ** 128 else np.nan
        return out, r * w


def rows_i8(p):
    """int8 codes and the base scale of fp32 rows p."""
    q, s = np.zeros(p.shape, np.int64), np.ones(len(p), F32)
    for t, row in enumerate(p):
        if not np.all(np.isfinite(row)):
            s[t] = np.nan
            continue
        a = np.abs(row).max() * (F32(1.0) / F32(127.0))
        s[t] = a if a > 0 else F32(1.0)
        q[t] = np.clip(np.rint(row.astype(np.float64) / np.float64(s[t])), -127, 127).astype(np.int64)
    return q, s


def wide_rows(q, s):
    """Code values [n][K] times their scales [n][blocks]."""
    return q * np.repeat(s.astype(np.float64), BLOCK, axis=1)[:, :q.shape[1]]


def wide_matrix(q, s):
    """Code values [R][K] times their scales [ceil(R / 128)][ceil(K / 128)]."""
    return wide_rows(q, np.repeat(s, BLOCK, axis=0)[:q.shape[0]])


def grouped_linear(xq, xs, rows, offs, E, nseg, w, ws):
    """y [N][O] and the sums of the terms' magnitudes; rows of no group are NaN."""
    x = wide_rows(xq, xs)
    y = np.full((len(rows), w.shape[1]), np.nan)
    mag = np.full_like(y, np.nan)
    for g in range(len(offs) - 1):
        r = np.asarray(rows[offs[g]:offs[g + 1]], np.int64)
        if len(r):
            e = group_expert(g, E, nseg)
            m = wide_matrix(w[e], ws[e])
            y[offs[g]:offs[g + 1]] = x[r] @ m.T
            mag[offs[g]:offs[g + 1]] = np.abs(x[r]) @ np.abs(m).T
    return y, mag


def sum_error(K):
    """Bound of the error of a sum of K products taken in blocks of 128, relative to the sum of magnitudes:
    a block's 128 terms in any order with steps that round down (2^-23 each), the product of the scales and its
    fma, and the sums over the blocks (2^-24 each)."""
    return BLOCK * 2.0 ** -23 + (-(-K // BLOCK) + 3) * 2.0 ** -24


def cut(x, w):
    """Bound of what the FP8 matrix instructions leave out of x [n][K] . w [O][K]^T (wide values).  Of each 8
    neighbouring columns they cut the products toward zero to multiples of 2^(e - 13), e the sum of the factors' exponents
    of the largest product, so that each of the other seven loses less than c = 2^-13 of the largest, with its
    own sign.  Signs are independent and even in the tests' data, so by Hoeffding's inequality the sum of the losses
    passes 8 sqrt(sum of c^2) once in 4e13 values."""
    pad = -x.shape[1] % 8
    big = lambda v: np.pad(np.abs(v), ((0, 0), (0, pad))).reshape(len(v), -1, 8).max(2) ** 2
    return 8 * 2.0 ** -13 * np.sqrt(7 * (big(x) @ big(w).T))


def linear_cut(xq, xs, rows, offs, E, nseg, w, ws):
    """cut() of grouped_linear."""
    x = wide_rows(xq, xs)
    out = np.full((len(rows), w.shape[1]), np.nan)
    for g in range(len(offs) - 1):
        r = np.asarray(rows[offs[g]:offs[g + 1]], np.int64)
        if len(r):
            e = group_expert(g, E, nseg)
            out[offs[g]:offs[g + 1]] = cut(x[r], wide_matrix(w[e], ws[e]))
    return out


def grouped_ffn(xq, xs, rows, offs, E, nseg, wg, sg, wu, su, wd, sd, on_codes=(False, False)):
    """h [N][d], the bound of its fp32 steps, and what it can move by if every code of the SwiGLU product whose
    quotient can reach the other side of a border does.  on_codes: which of the two products run on the FP8
    matrix instructions (cut).  Rows of no group are NaN."""
    x = wide_rows(xq, xs)
    d, I = wd.shape[1], wg.shape[1]
    h = np.full((len(rows), d), np.nan)
    err, slack = np.full_like(h, np.nan), np.full_like(h, np.nan)
    for g in range(len(offs) - 1):
        r = np.asarray(rows[offs[g]:offs[g + 1]], np.int64)
        if not len(r):
            continue
        e = group_expert(g, E, nseg)
        mg, mu = wide_matrix(wg[e], sg[e]), wide_matrix(wu[e], su[e])
        gate, up = x[r] @ mg.T, x[r] @ mu.T
        with np.errstate(over="ignore", invalid="ignore"):
            sig = 1.0 / (1.0 + np.exp(-gate))
            a = gate * sig * up
            # gate and up within their sums' errors; |silu'| <= 1.1; 12 + 5 |gate| half steps for silu and the products
            dg = (np.abs(x[r]) @ np.abs(mg).T) * sum_error(x.shape[1])
            du = (np.abs(x[r]) @ np.abs(mu).T) * sum_error(x.shape[1])
            if on_codes[0]:
                dg, du = dg + cut(x[r], mg), du + cut(x[r], mu)
            da = 1.1 * np.abs(up) * dg + np.abs(gate * sig) * du + 1.1 * dg * du + (12 + 5 * np.abs(gate)) * 2.0 ** -24 * np.abs(a)
        acc, moved, mag = np.zeros((len(r), d)), np.zeros((len(r), d)), np.zeros((len(r), d))
        md = wide_matrix(wd[e], sd[e])
        for b in range(0, I, BLOCK):
            part, dp, m = a[:, b:b + BLOCK], da[:, b:b + BLOCK], md[:, b:b + BLOCK]
            q, s = quantize_blocks(part.astype(F32))
            s = s.astype(np.float64)
            quotient = np.abs(part) / s
            # the scale is that of the largest value, so it is within that one's error; three more steps for the quotient
            top = np.abs(part).argmax(1)
            ds = dp[np.arange(len(r)), top] / np.maximum(np.abs(part).max(1), 1e-300) + 3 * 2.0 ** -24
            reach = dp / s + quotient * ds[:, None]
            step = e4m3_step(quotient)
            near = np.abs(quotient / step - np.floor(quotient / step) - 0.5) * step <= reach
            # a code next to a border moves by at most a step (twice that where the border is a power of two's)
            acc += (q * s) @ m.T
            moved += (near * 2 * step * s) @ np.abs(m).T
            mag += (np.abs(q) * s * (1 + ds[:, None])) @ np.abs(m).T
            moved += (np.abs(q) * s * ds[:, None]) @ np.abs(m).T
        if on_codes[1]:
            q, s = quantize_blocks(np.pad(a, ((0, 0), (0, -I % BLOCK))).astype(F32))
            moved += cut(wide_rows(q, s)[:, :I], md)
        h[offs[g]:offs[g + 1]] = acc
        slack[offs[g]:offs[g + 1]] = moved
        err[offs[g]:offs[g + 1]] = mag * sum_error(I)
    return h, err, slack
