"""The float64 definitions of the norm and of the block-scaled E4M3 products, pinned by hand and against torch."""
import numpy as np
import torch

from oracle import fp8_oracle as Q


def test_e4m3_values_match_torch():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    values = codes[torch.isfinite(codes)].double().numpy()
    np.testing.assert_array_equal(Q.e4m3(values), values)
    v = np.sort(values)
    mid = (v[1:] + v[:-1]) / 2                           # halves: torch rounds to even too
    np.testing.assert_array_equal(Q.e4m3(mid), torch.from_numpy(mid).float().to(torch.float8_e4m3fn).double().numpy())
    x = np.random.default_rng(0).uniform(-448, 448, 20000) * np.exp2(np.random.default_rng(1).integers(-20, 1, 20000))
    x = x.astype(np.float32)
    np.testing.assert_array_equal(Q.e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_quantize_blocks_by_hand():
    v = np.zeros((1, 136), np.float32)
    v[0, :3] = [896.0, -2.0, 1e-3]
    v[0, 128:131] = [7.0, -7.0, 0.25]
    q, s = Q.quantize_blocks(v)
    np.testing.assert_allclose(s, [[2.0, 7 / 448]], rtol=2e-7)
    assert q[0, 0] == 448 and q[0, 1] == -1 and q[0, 2] == 0
    assert q[0, 128] == 448 and q[0, 129] == -448 and q[0, 130] == 16
    assert not q[0, 3:128].any()
    q, s = Q.quantize_blocks(np.array([[0.0] * 8, [1e-37] * 8, [1.0, np.inf] + [0.0] * 6, [np.nan] + [1.0] * 7], np.float32))
    assert s[0, 0] == 1 and s[1, 0] == 1 and np.isnan(s[2:]).all() and not q.any()


def test_rmsnorm_by_hand():
    rstd, p = Q.rmsnorm(np.array([[3.0, 4.0]]), np.array([2.0, -1.0]), 0.5)
    np.testing.assert_allclose(rstd, [1 / np.sqrt(12.5 + 0.5)], rtol=1e-12)
    np.testing.assert_array_equal(p, [[6, -4]])
    rstd, _ = Q.rmsnorm(np.array([[1e20, 0.0], [np.nan, 0], [0, 0]], np.float32), np.ones(2), 1e-6)
    assert np.isnan(rstd[:2]).all() and abs(rstd[2] - 1e3) < 1e-3


def test_residual_sum_rounds_once_to_its_type():
    r = Q.residual_sum([1.0, 1.0], [2.0 ** -8, 2.0 ** -7], True)
    np.testing.assert_array_equal(r, np.array([1.0, 1.0 + 2.0 ** -7], np.float32))
    np.testing.assert_array_equal(Q.residual_sum([1.0], [2.0 ** -8], False), np.array([1.0 + 2.0 ** -8], np.float32))


def test_rows_i8_by_hand():
    q, s = Q.rows_i8(np.array([[254.0, -2.0, 1.0, 3.0], [0, 0, 0, 0], [1, np.inf, 0, 0]], np.float32))
    np.testing.assert_allclose(s[:2], [2, 1], rtol=1e-7)
    assert q[0].tolist() == [127, -1, 0, 2] or q[0].tolist() == [127, -1, 1, 2]
    assert np.isnan(s[2]) and not q[1:].any()


def test_linear_scales_by_block_and_expert():
    g = np.random.default_rng(2)
    K, O, E = 192, 256, 2
    xq, w = g.integers(-8, 9, (3, K)).astype(float), g.integers(-8, 9, (E, O, K)).astype(float)
    xs, ws = g.random((3, 2)).astype(np.float32), g.random((E, 2, 2)).astype(np.float32)
    y, mag = Q.grouped_linear(xq, xs, [2, 0], [0, 1, 2], E, 1, w, ws)
    for n, (r, e) in enumerate(((2, 0), (0, 1))):
        for o in (0, 127, 128, 255):
            want = sum(float(xs[r, b]) * float(ws[e, o // 128, b]) * (xq[r, b * 128:b * 128 + 128] @ w[e, o, b * 128:b * 128 + 128])
                       for b in (0, 1))
            np.testing.assert_allclose(y[n, o], want, rtol=1e-12)
            assert mag[n, o] >= abs(want)


def test_ffn_against_plain_torch():
    """Against quantisation and products spelled in torch double, on values far from a border or within the slack."""
    g = torch.Generator().manual_seed(3)
    d, I, E = 192, 320, 2
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.float8_e4m3fn).double()
    xq, wg, wu, wd = rnd(5, d), rnd(E, I, d), rnd(E, I, d), rnd(E, d, I)
    sc = lambda *s: torch.rand(s, generator=g) * 0.1 + 0.05
    xs, sg, su, sd = sc(5, 2), sc(E, 3, 2), sc(E, 3, 2), sc(E, 2, 3)
    h, err, slack = Q.grouped_ffn(*[t.numpy() for t in (xq, xs)], [0, 3, 4, 1], [0, 2, 4], E, 1,
                                  *[t.numpy() for t in (wg, sg, wu, su, wd, sd)])
    wide = lambda q, s: q * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:q.shape[0], :q.shape[1]]
    x = xq * xs.double().repeat_interleave(128, 1)[:, :d]
    for n, (r, e) in enumerate(((0, 0), (3, 0), (4, 1), (1, 1))):
        gate, up = wide(wg[e], sg[e]) @ x[r], wide(wu[e], su[e]) @ x[r]
        a = torch.nn.functional.silu(gate) * up
        want = torch.zeros(d, dtype=torch.float64)
        for b in range(0, I, 128):
            s = a[b:b + 128].abs().max() / 448
            want += wide(wd[e], sd[e])[:, b:b + 128] @ ((a[b:b + 128] / s).float().to(torch.float8_e4m3fn).double() * s)
        assert np.all(np.abs(h[n] - want.numpy()) <= err[n] + slack[n])
    assert np.median(err + slack) < 0.05 * np.median(np.abs(h))


def test_cut_bounds_products_cut_one_by_one():
    """Products of each eight columns cut toward zero to a multiple of 2^(E - 13), E the exponent sum of the largest
    product's factors: the sums lose no more than cut() allows, and something."""
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: (torch.randn(s, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    x, w = rnd(24, 261), rnd(40, 261)
    lost = np.zeros((24, 40))
    for k in range(0, 261, 8):
        p = x[:, None, k:k + 8] * w[None, :, k:k + 8]
        e = np.floor(np.log2(np.maximum(np.abs(x[:, None, k:k + 8]), 2.0 ** -20))) + np.floor(np.log2(np.maximum(np.abs(w[None, :, k:k + 8]), 2.0 ** -20)))
        at = np.abs(p).argmax(2)[:, :, None]
        step = np.exp2(np.take_along_axis(e, at, 2) - 13)
        lost += (p - np.trunc(p / step) * step).sum(2)
    bound = Q.cut(x, w)
    assert np.all(np.abs(lost) <= bound) and np.abs(lost).max() > 0
    np.testing.assert_allclose(np.linalg.norm(lost) / np.linalg.norm(x @ w.T), 3e-5, rtol=0.7)
