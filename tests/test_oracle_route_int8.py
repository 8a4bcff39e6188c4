"""Pins of the float64 definitions of routing with scores and of the int8 products."""
import numpy as np
import pytest
import torch

from oracle import int8_oracle as Q
from oracle import moe_oracle as O


def test_route_without_extras_is_the_gate():
    g = np.random.default_rng(1)
    l = g.standard_normal((40, 16)).astype(np.float32)
    for renorm in (True, False):
        ids, w = Q.route(l, 4, renormalize=renorm)
        ids0, w0 = O.gate(l, 4, renorm)
        np.testing.assert_array_equal(ids, ids0)
        # the gate's oracle rounds its weights to fp32: half a step, 2^-24 of the value, apart
        assert np.all(np.abs(w - w0) <= 2.0 ** -24 * np.abs(w) * (1 + 1e-6))


def test_route_by_hand():
    # four experts in two groups: sigmoid scores .5 .88 .73 .27
    l = np.array([[0.0, 2.0, 1.0, -1.0]])
    ids, w = Q.route(l, 2, "sigmoid", None, 2, 1, "max", False, 2.0)
    assert ids.tolist() == [[1, 0]]                                # group 0 holds the best
    np.testing.assert_allclose(w, [[2 / (1 + np.exp(-2.0)), 1.0]])
    ids, _ = Q.route(l, 2, "sigmoid", np.array([0, 0, 0.5, 0.5]), 2, 1, "top2", False)
    assert ids.tolist() == [[2, 3]]                                # 0.5 + 0.88 < 1.23 + 0.77
    ids, w = Q.route(l, 1, "sigmoid", np.array([5.0, 0, 0, 0]), renormalize=False)
    assert ids.tolist() == [[0]] and w[0, 0] == 0.5                # the bias selects, the score weighs
    ids, _ = Q.route(np.zeros((1, 8)), 3, "softmax", None, 4, 2)
    assert ids.tolist() == [[0, 1, 2]]                             # ties: lower group, lower expert
    ids, w = Q.route(np.full((1, 4), -np.inf), 2)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]
    ids, w = Q.route(np.array([[np.nan, np.inf, 0.0, np.inf]]), 2, renormalize=False)
    assert ids.tolist() == [[1, 3]] and w.tolist() == [[0.5, 0.5]]


def test_quantize_by_hand():
    q, s = Q.quantize(np.array([[127.0, 0.5, 1.5, -2.5, 63.4999]]))
    assert s.tolist() == [1.0] and q.tolist() == [[127, 0, 2, -2, 63]]
    q, s = Q.quantize(np.array([[0.0, 0.0], [1.0, np.inf], [np.nan, 2.0]]))
    assert s[0] == 1.0 and np.isnan(s[1:]).all() and not q.any()


def test_linear_is_a_matrix_product():
    g = np.random.default_rng(2)
    xq, w = g.integers(-127, 128, (5, 64)), g.integers(-127, 128, (1, 64, 64))
    xs, ws = g.random(5).astype(np.float32), g.random((1, 64)).astype(np.float32)
    y = Q.grouped_linear(xq, xs, np.arange(5), [0, 5], 1, 1, w, ws)
    ref = torch.from_numpy(xq * xs[:, None].astype(np.float64)) @ torch.from_numpy(w[0] * ws[0][:, None].astype(np.float64)).T
    np.testing.assert_allclose(y, ref.numpy(), rtol=1e-12)


def test_ffn_is_near_the_plain_ffn():
    """Every step of 1/254 of a row's or block's largest value: the result is within a few per cent of the
    unquantised FFN of the dequantised weights."""
    g = np.random.default_rng(3)
    E, d, I, T = 2, 128, 192, 6
    x = g.standard_normal((T, d))
    ws = [g.integers(-127, 128, (E, *sh)) for sh in ((I, d), (I, d), (d, I))]
    ss = [(g.random((E, sh)) * 1e-3 + 1e-3).astype(np.float32) for sh in (I, I, d)]
    rows, offs = np.arange(T), [0, 4, 6]
    h, slack = Q.grouped_ffn(x, rows, offs, E, 1, ws[0], ss[0], ws[1], ss[1], ws[2], ss[2], margin=1e-6)
    full = [w * s[:, :, None].astype(np.float64) for w, s in zip(ws, ss)]
    for e in range(E):
        r = slice(offs[e], offs[e + 1])
        gate = x[r] @ full[0][e].T
        ref = (gate / (1 + np.exp(-gate)) * (x[r] @ full[1][e].T)) @ full[2][e].T
        assert np.linalg.norm(h[r] - ref) < 0.05 * np.linalg.norm(ref)
    assert slack.max() < 0.05 * np.abs(h).max()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_against_torch(score):
    g = torch.Generator().manual_seed(4)
    l = torch.randn((64, 32), generator=g, dtype=torch.float64)
    b = torch.randn(32, generator=g, dtype=torch.float64).float()
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    c = s + b.double()
    v = c.view(64, 4, 8).topk(2, 2).values.sum(2)
    keep = torch.zeros(64, 4, dtype=torch.bool).scatter_(1, v.topk(2, 1).indices, True)
    ref = c.masked_fill(~keep.repeat_interleave(8, 1), -9e9).topk(5, 1).indices
    ids, w = Q.route(l.numpy(), 5, score, b.numpy(), 4, 2, "top2", True, 2.5)
    np.testing.assert_array_equal(ids, ref.numpy())
    sel = s.gather(1, ref)
    np.testing.assert_allclose(w, (2.5 * sel / sel.sum(1, keepdim=True)).numpy(), rtol=1e-12)


def test_planted_mistakes_are_seen(monkeypatch):
    """The pins fail on wrong definitions: a bias that weighs, codes rounded down, one scale for the whole row."""
    l = np.array([[0.0, 2.0, 1.0, -1.0]])
    real = Q.route
    monkeypatch.setattr(Q, "route", lambda l, k, *a, **kw: tuple(v * 2 for v in real(l, k, *a, **kw)))
    with pytest.raises(AssertionError):
        test_route_by_hand()
    monkeypatch.setattr(Q, "route", real)
    real_q = Q.quantize
    monkeypatch.setattr(Q, "quantize", lambda v: (np.floor(np.nan_to_num(np.asarray(v) / 1.0)).astype(np.int64), real_q(v)[1]))
    with pytest.raises(AssertionError):
        test_quantize_by_hand()
    with pytest.raises(AssertionError):
        test_ffn_is_near_the_plain_ffn()
    assert real(l, 1)[0][0, 0] == 1
