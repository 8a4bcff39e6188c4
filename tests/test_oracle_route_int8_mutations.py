"""Plant one-line mistakes in the float64 definitions of routing with scores and of the int8 products (on the CPU) and
check that a pin sees each."""
import inspect
import textwrap

import numpy as np
import pytest

from oracle import int8_oracle as Q
import test_oracle_route_int8 as P


# ------------------------------------------------------------------ further pins
def pin_weights_by_hand():
    # shares of the chosen scores, not of all; the bias selects and does not weigh; the scale multiplies
    l = np.log([[1.0, 3.0, 4.0, 8.0]])
    ids, w = Q.route(l, 2, "softmax", np.array([0, 0, 0, -5.0]), renormalize=True, scale=2.0)
    assert ids.tolist() == [[2, 1]]
    np.testing.assert_allclose(w, [[8 / 7, 6 / 7]], rtol=1e-12)
    ids, w = Q.route(l, 2, "softmax", np.array([0, 0.9, 0, 0]), renormalize=False, scale=0.5)
    assert ids.tolist() == [[1, 3]]
    np.testing.assert_allclose(w, [[1.5 / 16, 4 / 16]], rtol=1e-12)
    # a sum of next to nothing still has shares (the sigmoid of -720 is below the smallest normal double)
    ids, w = Q.route(np.full((1, 4), -720.0), 2, "sigmoid", scale=3.0)
    np.testing.assert_allclose(w, [[1.5, 1.5]], rtol=1e-12)


def pin_groups_by_hand():
    s = np.array([[0.1, 0.1, 0.3, 0.0, 0.2, 0.25, 0.05, 0.0]])
    ids, _ = Q.route(np.log(np.maximum(s, 1e-9)), 2, "softmax", None, 4, 1, "top2")
    assert ids.tolist() == [[5, 4]]                         # .45 over .30
    ids, _ = Q.route(np.log(np.maximum(s, 1e-9)), 1, "softmax", None, 4, 1, "max")
    assert ids.tolist() == [[2]]


def pin_experts_of_groups():
    assert [Q.group_expert(g, 3, 2) for g in range(8)] == [0, 1, 2, 0, 1, 2, 3, 4]
    g = np.random.default_rng(5)
    xq, w = g.integers(-127, 128, (4, 64)), g.integers(-127, 128, (2, 64, 64))
    xs, ws = g.random(4).astype(np.float32), g.random((2, 64)).astype(np.float32)
    y = Q.grouped_linear(xq, xs, [3, 0, 1], [0, 1, 3], 2, 1, w, ws)
    for n, (r, e) in enumerate(((3, 0), (0, 1), (1, 1))):
        np.testing.assert_allclose(y[n], (w[e] @ xq[r]) * (xs[r].astype(np.float64) * ws[e].astype(np.float64)), rtol=1e-12)


def pin_blocks_have_their_own_scale():
    """The second 128 columns of the SwiGLU product are a ten-thousandth of the first: with a scale of their own they
    are within half a step of their largest, with the row's they would all be 0.  And silu, gate and up by hand."""
    d, I = 64, 256
    x = np.zeros((1, d))
    x[0, 0] = 127.0                                          # scale 1, code 127
    wg, wu, wd = np.zeros((1, I, d), int), np.zeros((1, I, d), int), np.zeros((1, d, I), int)
    wg[0, :, 0], wu[0, :, 0] = 1, np.arange(1, I + 1) % 100 + 27
    wd[0, :, 128:192] = np.eye(d, dtype=int)
    sg = np.full((1, I), -1 / 127, np.float32)               # gates of about -1
    su = np.where(np.arange(I) < 128, 1.0, 1e-4).astype(np.float32)[None]
    sd = np.full((1, d), 2.0, np.float32)
    h, _ = Q.grouped_ffn(x, [0], [0, 1], 1, 1, wg, sg, wu, su, wd, sd)
    gate = 127.0 * np.float64(sg[0, 0])
    a = gate / (1 + np.exp(-gate)) * 127.0 * wu[0, :, 0] * su[0].astype(np.float64)
    step = np.abs(a[128:]).max() / 127
    assert np.abs(h[0] - 2.0 * a[128:192]).max() <= 2.0 * 0.51 * step


PINS = [P.test_route_by_hand, P.test_route_without_extras_is_the_gate, lambda: P.test_route_against_torch("softmax"),
        lambda: P.test_route_against_torch("sigmoid"), P.test_quantize_by_hand, P.test_linear_is_a_matrix_product,
        P.test_ffn_is_near_the_plain_ffn, pin_weights_by_hand, pin_groups_by_hand, pin_experts_of_groups,
        pin_blocks_have_their_own_scale]


@pytest.mark.parametrize("pin", [pin_weights_by_hand, pin_groups_by_hand, pin_experts_of_groups, pin_blocks_have_their_own_scale])
def test_pins(pin):
    pin()


MISTAKES = [
    ("route", "w[t] = wide[order]\n", "w[t] = (wide if bias is None else wide + np.asarray(bias))[order]\n"),   # a bias that weighs
    ("route", "wide[order] / wide[order].sum()", "wide[order] / wide.sum()"),
    ("route", "if s[order].sum() > 0 else 0.0", "if s[order].sum() > 1e-300 else 0.0"),
    ("route", "if renormalize:", "if not renormalize:"),
    ("route", "return ids, w * float(np.float32(scale))", "return ids, w"),
    ("route", "(-c[e], e)", "(-c[e], -e)"),                                                 # ties to the higher expert
    ("route", "-np.inf if np.isnan(v) else v, -g", "-np.inf if np.isnan(v) else v, g % 1 - (n_groups - g)"),   # and group
    ("route", "l[np.isnan(l)] = -np.inf", "l[np.isnan(l)] = np.inf"),
    ("route", "sum(two) if group_rank", "two[0] if group_rank"),
    ("route", "s + np.asarray(bias, np.float64)", "row + np.asarray(bias, np.float64)"),
    ("route", "-np.inf if np.isnan(v) else v", "v * 0"),                                    # groups not valued
    ("quantize", "np.rint(", "np.floor("),                                                  # codes rounded down
    ("quantize", "np.rint(row / np.float64(s[r]))", "np.sign(row) * np.floor(np.abs(row) / np.float64(s[r]) + 0.5)"),
    ("quantize", "np.float32(127.0)", "np.float32(128.0)"),
    ("quantize", "a if a > 0 else np.float32(1.0)", "a"),
    ("quantize", "s[r] = np.nan", "s[r] = 1.0"),
    ("group_expert", "g % E", "g"),
    ("group_expert", "g - nseg * E", "g - E"),
    ("grouped_linear", "_dot(xq[r], w[e])", "_dot(xq[r], w[0])"),
    ("grouped_linear", "xs[r]", "xs[:len(r)]"),
    ("grouped_linear", "ws[e]", "ws[0]"),
    ("grouped_ffn", "q, s = quantize(a[:, b:b + block])",
     "q, s = quantize(a)\n            q = q[:, b:b + block]"),                              # one scale for the whole row
    ("grouped_ffn", "np.exp(-gate)", "np.exp(gate)"),
    ("grouped_ffn", "gate / (1.0 + np.exp(-gate)) * up", "up / (1.0 + np.exp(-up)) * gate"),
    ("grouped_ffn", "acc * sd[e]", "acc * sd[0] * 0 + acc"),
    ("grouped_ffn", "_dot(xq[r], wu[e]) * sx", "_dot(xq[r], wu[e])"),
]


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("name,right,wrong", MISTAKES)
def test_planted_mistake_is_seen(monkeypatch, name, right, wrong):
    text = textwrap.dedent(inspect.getsource(getattr(Q, name)))
    assert right in text
    space = dict(vars(Q))
    exec(text.replace(right, wrong, 1), space)               # the rest of the module as it is
    monkeypatch.setattr(Q, name, space[name])
    seen = 0
    for pin in PINS:
        try:
            pin()
        except (AssertionError, ValueError, IndexError):
            seen += 1
    assert seen > 0
