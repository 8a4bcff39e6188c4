"""Plant one-line mistakes in the float64 definitions of the norm and of the block-scaled E4M3 products (on the CPU) and
check that a pin sees each."""
import inspect
import textwrap

import numpy as np
import pytest

from oracle import fp8_oracle as Q
import test_oracle_norm_fp8 as P


# ------------------------------------------------------------------ further pins
def pin_codes_of_a_row():
    # quotients are rounded to fp32 and then to E4M3, halves to even; each block has its own scale
    q, s = Q.quantize_blocks(np.array([[448.0, 17.0, 19.0, -17.0] + [0.0] * 124 + [-44.8, 1.7] + [0.0] * 6], np.float32))
    assert q[0, :4].tolist() == [448, 16, 20, -16]
    np.testing.assert_allclose(s, [[1, 0.1]], rtol=3e-7)
    assert q[0, 128] == -448 and q[0, 129] in (16, 18)


def pin_rows_of_experts():
    g = np.random.default_rng(5)
    xq, w = g.integers(-8, 9, (4, 64)).astype(float), g.integers(-8, 9, (3, 64, 64)).astype(float)
    xs, ws = g.random((4, 1)).astype(np.float32), g.random((3, 1, 1)).astype(np.float32)
    y, mag = Q.grouped_linear(xq, xs, [3, 0, 1, 2], [0, 1, 2, 3, 3, 4], 2, 2, w, ws)     # 2 + 2 groups and a shared one
    for n, (r, e) in enumerate(((3, 0), (0, 1), (1, 0), (2, 2))):
        np.testing.assert_allclose(y[n], w[e] @ xq[r] * (float(xs[r, 0]) * float(ws[e, 0, 0])), rtol=1e-12)
        np.testing.assert_allclose(mag[n], np.abs(w[e]) @ np.abs(xq[r]) * (float(xs[r, 0]) * float(ws[e, 0, 0])), rtol=1e-12)


def pin_blocks_have_their_own_scale():
    """The second 128 columns of the SwiGLU product are a ten-thousandth of the first: with a scale of their own they are
    within half a step of their size."""
    d, I = 64, 256
    x = np.zeros((1, d))
    x[0, 0] = 4.0
    wg, wu, wd = np.zeros((1, I, d)), np.zeros((1, I, d)), np.zeros((1, d, I))
    wg[0, :, 0], wu[0, :, 0] = -0.25, np.arange(I) % 7 + 1                  # gates of -1
    wd[0, :, 128:192] = np.eye(d)
    one = np.ones((1, 1, 1), np.float32)
    su = np.array([[[1.0], [1e-4]]], np.float32)
    sd = np.array([[[1.0, 2.0]]], np.float32)
    h, err, slack = Q.grouped_ffn(x, np.ones((1, 1), np.float32), [0], [0, 1], 1, 1, wg, np.repeat(one, 2, 1), wu, su, wd, sd)
    a = -1.0 / (1 + np.e) * 4.0 * wu[0, :, 0] * np.repeat(su[0, :, 0].astype(np.float64), 128)
    assert np.all(np.abs(h[0] - 2.0 * a[128:192]) <= 2.0 * np.abs(a[128:192]) * (2.0 ** -4 + 1e-6))
    assert np.all(err >= 0) and err.max() > 0 and np.all(slack >= 0) and np.isfinite(slack).all()


def pin_cut_is_counted_where_asked():
    g = np.random.default_rng(6)
    rnd = lambda *s: Q.e4m3(g.normal(size=s))
    args = (rnd(2, 128), np.ones((2, 1), np.float32), [0, 1], [0, 2], 1, 1, rnd(1, 128, 128), np.ones((1, 1, 1), np.float32),
            rnd(1, 128, 128), np.ones((1, 1, 1), np.float32), rnd(1, 128, 128), np.ones((1, 1, 1), np.float32))
    none, up, down = (Q.grouped_ffn(*args, on_codes=c)[2] for c in ((False, False), (True, False), (False, True)))
    assert up.sum() > none.sum() and np.all(down > none)


MORE = [pin_codes_of_a_row, pin_rows_of_experts, pin_blocks_have_their_own_scale, pin_cut_is_counted_where_asked]
PINS = [f for name, f in sorted(vars(P).items()) if name.startswith("test_")] + MORE


@pytest.mark.parametrize("pin", MORE)
def test_pins(pin):
    pin()


MISTAKES = [
    ("e4m3_step", "np.maximum(e, -6)", "e"),                                        # no subnormals
    ("e4m3_step", "np.maximum(e, -6) - 3", "np.maximum(e, -6) - 4"),                # a bit more of mantissa
    ("e4m3", "np.rint(v / step)", "np.floor(v / step + 0.5)"),
    ("quantize_blocks", "F32(448.0)", "F32(256.0)"),
    ("quantize_blocks", "F32(2.0 ** -100)", "F32(2.0 ** -149)"),
    ("quantize_blocks", "s[r, b] = np.nan", "s[r, b] = 1.0"),
    ("quantize_blocks", "np.abs(part).max()", "np.abs(row).max()"),                 # one scale for the whole row
    ("quantize_blocks", "np.abs(part).max()", "part.max()"),
    ("residual_sum", "if bf16 else r", "if not bf16 else r"),
    ("rmsnorm", "m / r.shape[1]", "m"),
    ("rmsnorm", "+ float(F32(eps))", ""),
    ("rmsnorm", "return out, r * w", "return out, r"),
    ("rmsnorm", "if m < 2.0 ** 128 else np.nan", ""),
    ("rows_i8", "F32(127.0)", "F32(128.0)"),
    ("rows_i8", "a if a > 0 else F32(1.0)", "a"),
    ("rows_i8", "s[t] = np.nan", "s[t] = 1"),
    ("wide_rows", "np.repeat(s.astype(np.float64), BLOCK, axis=1)", "np.tile(s.astype(np.float64), (1, BLOCK))"),
    ("wide_matrix", "np.repeat(s, BLOCK, axis=0)", "np.tile(s, (BLOCK, 1))"),
    ("grouped_linear", "x[r] @ m.T", "x[:len(r)] @ m.T"),
    ("grouped_linear", "wide_matrix(w[e], ws[e])", "wide_matrix(w[e], ws[0])"),
    ("grouped_linear", "np.abs(x[r]) @ np.abs(m).T", "np.abs(x[r] @ m.T)"),
    ("cut", "2.0 ** -13", "2.0 ** -24"),
    ("cut", "reshape(len(v), -1, 8).max(2)", "reshape(len(v), -1, 8).min(2)"),
    ("grouped_ffn", "np.exp(-gate)", "np.exp(gate)"),
    ("grouped_ffn", "a = gate * sig * up", "a = up * sig * gate * gate"),
    ("grouped_ffn", "wide_matrix(wd[e], sd[e])", "wide_matrix(wd[e], sd[e] * 0 + 1)"),
    ("grouped_ffn", "wide_matrix(wu[e], su[e])", "wide_matrix(wu[e], sg[e])"),
    ("grouped_ffn", "if on_codes[0]:", "if False:"),
    ("grouped_ffn", "if on_codes[1]:", "if False:"),
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
