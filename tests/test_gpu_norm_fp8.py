"""GPU parity of the norm and of the block-scaled FP8 calls against their float64 definitions.

Tolerances, from the arithmetic of the calls (u = 2^-24, half an fp32 step):
  residual sums, codes  equal
  y, scales of the norm the sum of d squares: a thread adds at most n = max(64, d / 32) of them one after the other, then 9 steps
                        join them, all terms positive, so within (n + 9) u; its mean, the sum with eps, root and
                        reciprocal within half of that and 4 u more; two products: (n / 2 + 10) u, and the rounding of y
  scales of quantize    equal
  linear                sum_error(K) of the sum of magnitudes, and the output's rounding; with bf16 out, where groups are
                        large enough for the FP8 matrix instructions (fp8_plan), what those cut (fp8_oracle.cut)
  ffn                   the same for its second product, what the codes of the SwiGLU product may move, and the rounding
"""
import numpy as np
import pytest
import torch

import fp8_plan
from oracle import fp8_oracle as Q
from helpers import announce, f64_of, np_of, require_gpu

import top_expert_routing_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _dt(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _rows(g, T, d, dtype):
    x = torch.randn((T, d), generator=g) * torch.exp(torch.randn((T, 1), generator=g))
    return x.to(_dt(dtype))


def _f32(t):
    return t.float().cpu().numpy()


# ------------------------------------------------------------------ norm
NORM = [
    # T, d, x, residual, weight, y, codes
    (1, 8, "f32", None, "f32", "f32", None),
    (3, 40, "bf16", "bf16", "bf16", "bf16", "fp8"),
    (5, 128, "bf16", None, "f32", "bf16", "fp8"),
    (2, 136, "f32", "bf16", "bf16", None, "fp8"),
    (9, 504, "bf16", "f32", "bf16", "f32", "i8"),
    (6, 512, "bf16", "bf16", "bf16", None, "i8"),
    (7, 520, "f32", "f32", "f32", "f32", "i8"),
    (16, 2048, "bf16", "bf16", "bf16", "bf16", "fp8"),
    (4, 2056, "bf16", "f32", "bf16", "bf16", "fp8"),
    (131, 2880, "bf16", "bf16", "bf16", "bf16", "fp8"),
    (17, 4096, "f32", None, "bf16", "bf16", "i8"),
    (3, 4104, "f32", "f32", "bf16", None, "fp8"),
    (2, 8200, "bf16", "bf16", "bf16", "bf16", "fp8"),
    (3, 16384, "bf16", "bf16", "f32", "f32", "i8"),
    (3, 16392, "bf16", "bf16", "bf16", "bf16", "fp8"),
    (2, 20000, "f32", "bf16", "bf16", "bf16", "i8"),
    (1, 33000, "bf16", None, "bf16", "f32", "fp8"),
    (2, 16400, "f32", "f32", "f32", "bf16", None),
]


def _norm_check(x, res, w, eps, y, codes, out, q, s):
    d = x.shape[1]
    r = _f32(x)
    if res is not None:
        with np.errstate(over="ignore"):
            r = Q.residual_sum(r, _f32(res), res.dtype == torch.bfloat16)
        np.testing.assert_array_equal(_f32(out), r)
    with np.errstate(over="ignore", invalid="ignore"):
        rstd, p = Q.rmsnorm(r, _f32(w), eps)
        rel = (max(64, d / 32) / 2 + 10) * 2.0 ** -24
        if y is not None:
            ref = p.astype(np.float64) * rstd[:, None]
            got = f64_of(y)
            tol = (rel + torch.finfo(y.dtype).eps / 2) * (1 + 1e-6) * np.abs(ref) + 1e-37
            assert np.array_equal(np.isnan(got), np.isnan(ref))
            fine = ~np.isnan(ref)
            assert np.all(np.abs(got - ref)[fine] <= tol[fine]), np.abs(got - ref)[fine].max()
        if codes == "fp8":
            qr, base = Q.quantize_blocks(p)
            np.testing.assert_array_equal(f64_of(q), qr)
            sr = base.astype(np.float64) * rstd[:, None]
        elif codes == "i8":
            qr, base = Q.rows_i8(p)
            np.testing.assert_array_equal(np_of(q), qr)
            sr = base.astype(np.float64) * rstd
        if codes:
            np.testing.assert_allclose(f64_of(s), sr, rtol=rel)


@pytest.mark.parametrize("case", NORM)
def test_norm_parity(case):
    announce(f"norm {case}")
    T, d, xt, rt, wt, yt, codes = case
    g = _gen(T * 7 + d)
    x = _rows(g, T, d, xt)
    res = None if rt is None else (3 * _rows(g, T, d, rt)).to(_dt(rt))
    w = (1 + 0.3 * torch.randn((d,), generator=g)).to(_dt(wt))
    y = None if yt is None else torch.full((T, d), 7.0, dtype=_dt(yt), device=DEV)
    out = None if res is None else torch.full((T, d), 7.0, dtype=res.dtype, device=DEV)
    rd = None if res is None else res.to(DEV)
    got, q, s = moe.rmsnorm(x.to(DEV), w.to(DEV), 1e-5, rd, out, y, codes, want_y=yt is not None)
    torch.cuda.synchronize()
    assert got is y
    if res is not None:
        assert torch.equal(rd.cpu(), res)
    _norm_check(x, res, w, 1e-5, y, codes, out, q, s)
    # in place, outputs made by the call, the same bits
    if res is not None:
        y2, q2, s2 = moe.rmsnorm(x.to(DEV), w.to(DEV), 1e-5, rd, codes=codes, y=None if y is None else torch.empty_like(y),
                                 want_y=y is not None)
        assert torch.equal(rd, out)
        for a, b in ((y, y2), (q, q2), (s, s2)):
            assert (a is None) == (b is None)
            if a is not None:
                assert torch.equal(a.view(torch.uint8) if a.dtype == F8 else a, b.view(torch.uint8) if b.dtype == F8 else b)


@pytest.mark.parametrize("d", [48, 2880, 17000])
@pytest.mark.parametrize("codes", ["fp8", "i8"])
@pytest.mark.parametrize("rt", [None, "bf16", "f32"])
def test_norm_special_rows(d, codes, rt):
    announce(f"norm special {d} {codes} {rt}")
    g = _gen(d)
    x = torch.randn((12, d), generator=g)
    x[0] = 0
    x[1, 5] = np.nan
    x[2, d - 1] = np.inf
    x[3] = -np.inf
    x[4] *= 1e25                     # squares pass fp32
    x[5] *= 1e-30                    # squares vanish: eps alone
    x[6] *= 1e-42                    # subnormal
    x[7, 0] = 3e18                   # one value far above the others
    x[8] = torch.finfo(torch.float32).max
    x[9, ::2] = 0
    x[10] *= 1e15
    res = None if rt is None else torch.zeros((12, d), dtype=_dt(rt))
    w = torch.randn((d,), generator=g)
    out = None if res is None else torch.empty((12, d), dtype=res.dtype, device=DEV)
    rd = None if res is None else res.to(DEV)
    y, q, s = moe.rmsnorm(x.to(DEV), w.to(DEV), 1e-6, rd, out, codes=codes)
    torch.cuda.synchronize()
    _norm_check(x, res, w, 1e-6, y, codes, out, q, s)
    assert torch.isnan(y[1]).all() and torch.isnan(s[1]).all() and torch.isnan(y[4]).all()
    assert not y[0].any() and not y[9, ::2].any()


def test_norm_codes_stand_for_y():
    """Codes times scales are the row that y holds, within half a step of the codes."""
    announce("norm codes and y")
    g = _gen(2)
    x, w = _rows(g, 50, 640, "bf16").to(DEV), (1 + 0.2 * torch.randn((640,), generator=g)).to(DEV)
    y, q, s = moe.rmsnorm(x, w, codes="fp8", y=torch.empty((50, 640), device=DEV))
    wide = s.repeat_interleave(128, 1)
    err = (q.float() * wide - y).abs()
    assert torch.all(err <= 2.0 ** -4 * y.abs() * (1 + 1e-5) + 2.0 ** -10 * wide)
    y2, q, s = moe.rmsnorm(x, w, codes="i8", y=torch.empty_like(y))
    assert torch.equal(y, y2)
    assert torch.all((q.float() * s[:, None] - y).abs() <= 0.5 * (1 + 1e-4) * s[:, None])


def test_norm_shapes_and_refusals():
    x = torch.randn((2, 3, 64), generator=_gen(9)).to(DEV)
    w = torch.ones(64, device=DEV)
    y, q, s = moe.rmsnorm(x, w, codes="fp8")
    assert y.shape == x.shape and q.shape == x.shape and q.dtype == F8 and s.shape == (2, 3, 1)
    y2, q2, s2 = moe.rmsnorm(x.view(6, 64), w, codes="fp8")
    assert torch.equal(y.view(6, 64), y2) and torch.equal(s.view(6, 1), s2)
    assert moe.rmsnorm(x, w, codes="i8")[2].shape == (2, 3)
    assert moe.rmsnorm(x, w)[1:] == (None, None)
    y, q, s = moe.rmsnorm(torch.empty((0, 64), device=DEV), w, codes="fp8")
    assert y.shape == (0, 64) and s.shape == (0, 1)
    half = x.half()
    for a, kw in (((half, w), {}), ((x[..., ::2], w[::2].contiguous()), {}), ((x.cpu(), w), {}), ((x, w[:32]), {}), ((x, w.half()), {}),
                  ((x, w.cpu()), {}), ((x, w), dict(residual=half)), ((x, w), dict(residual=x[0])), ((x, w), dict(residual_out=x)),
                  ((x, w), dict(residual=x, residual_out=x.bfloat16())), ((x, w), dict(codes="fp4")), ((x, w), dict(want_y=False)),
                  ((x, w), dict(q=torch.empty_like(x, dtype=torch.int8))), ((x, w), dict(codes="i8", q=torch.empty_like(x, dtype=F8))),
                  ((x, w), dict(codes="fp8", s=torch.empty((2, 3), device=DEV))), ((x, w), dict(y=x[0])), ((x, w), dict(y=half))):
        with pytest.raises((TypeError, ValueError)):
            moe.rmsnorm(*a, **kw)
    for kw in (dict(eps=0.0), dict(eps=float("nan"))):
        with pytest.raises(moe.MoeError):
            moe.rmsnorm(x, w, **kw)
    with pytest.raises(moe.MoeError):
        moe.rmsnorm(torch.zeros((2, 12), device=DEV), torch.ones(12, device=DEV))


# ------------------------------------------------------------------ quantize
@pytest.mark.parametrize("T,d,dtype", [(1, 8, "bf16"), (3, 120, "f32"), (5, 128, "bf16"), (7, 136, "f32"), (19, 2880, "bf16"),
                                       (130, 2048, "f32"), (2, 40000, "bf16"), (257, 264, "bf16")])
def test_quantize_parity(T, d, dtype):
    announce(f"quantize {T} {d} {dtype}")
    x = _rows(_gen(T + d), T, d, dtype)
    x[0, : d // 2] = 0
    q, s = moe.quantize_blocks_fp8(x.to(DEV))
    qr, sr = Q.quantize_blocks(_f32(x))
    np.testing.assert_array_equal(f64_of(q), qr)
    np.testing.assert_array_equal(np_of(s), sr)


def test_quantize_borders():
    """Every midpoint of two E4M3 values and its fp32 neighbours, at scales that are no powers of two."""
    announce("quantize borders")
    v = torch.arange(128, dtype=torch.uint8).view(F8).float()
    v = v[torch.isfinite(v)].sort().values
    mid = (v[1:] + v[:-1]) / 2
    rows = []
    for scale in (1.0, 0.37, 1.7e-20, 3.3e22):
        for m in (mid, torch.nextafter(mid, torch.tensor(1e9)), torch.nextafter(mid, torch.tensor(0.0))):
            r = torch.zeros(128)
            r[:126] = m * scale
            r[127] = -448.0 * scale
            rows.append(r)
    x = torch.stack(rows)
    q, s = moe.quantize_blocks_fp8(x.to(DEV))
    qr, sr = Q.quantize_blocks(x.numpy())
    np.testing.assert_array_equal(np_of(s), sr)
    np.testing.assert_array_equal(f64_of(q), qr)


def test_quantize_special_values():
    x = torch.zeros((8, 256))
    x[1, 3] = np.nan
    x[2, 200] = -np.inf
    x[3] = 1e-38
    x[4, :128] = 2.0 ** -92
    x[5] = torch.finfo(torch.float32).max
    x[6, 0], x[6, 1] = 1e30, 1e-30
    x[7, 128:] = 1e-45
    for dt in (torch.float32, torch.bfloat16):
        q, s = moe.quantize_blocks_fp8(x.to(dt).to(DEV))
        qr, sr = Q.quantize_blocks(_f32(x.to(dt)))
        np.testing.assert_array_equal(np_of(s), sr)
        np.testing.assert_array_equal(f64_of(q), qr)
    assert torch.equal(moe.quantize_blocks_fp8(torch.empty((0, 64), device=DEV))[1], torch.empty((0, 1), device=DEV))
    q, s = moe.quantize_blocks_fp8(x.view(2, 4, 256).to(DEV))
    assert q.shape == (2, 4, 256) and s.shape == (2, 4, 2)
    for bad in (x.half().to(DEV), x.to(DEV)[:, ::2], x):
        with pytest.raises((TypeError, ValueError)):
            moe.quantize_blocks_fp8(bad)


def test_more_rows_than_one_launch_and_elements_past_int32():
    announce("norm and quantize past int32")
    x = torch.randn((4096, 8), generator=_gen(19)).bfloat16().to(DEV)
    w = torch.linspace(0.5, 2, 8).to(DEV)
    T = 2 ** 25 + 77
    big = x.repeat(8193, 1)[:T].contiguous()
    y0, q0, s0 = moe.rmsnorm(x, w, codes="fp8")
    y, q, s = moe.rmsnorm(big, w, codes="fp8")
    bits = lambda t: t.view(torch.uint8)
    assert torch.equal(y, y0.repeat(8193, 1)[:T]) and torch.equal(s, s0.repeat(8193, 1)[:T])
    assert torch.equal(bits(q), bits(q0).repeat(8193, 1)[:T])
    q1, s1 = moe.quantize_blocks_fp8(x)
    q, s = moe.quantize_blocks_fp8(big)
    assert torch.equal(bits(q), bits(q1).repeat(8193, 1)[:T]) and torch.equal(s, s1.repeat(8193, 1)[:T])
    del y, q, s, big
    # 2^31 values and more
    d, T = 2048, 2 ** 20 + 5
    x = torch.randn((1024, d), generator=_gen(20)).bfloat16().to(DEV)
    w = torch.rand((d,), generator=_gen(21)).to(DEV)
    big = x.repeat(1025, 1)[:T].contiguous()
    y, q, s = moe.rmsnorm(big, w, codes="fp8")
    y0, q0, s0 = moe.rmsnorm(x, w, codes="fp8")
    tail = slice(T - 700, T)
    at = torch.arange(T - 700, T, device=DEV) % 1024
    assert torch.equal(y[tail], y0[at]) and torch.equal(bits(q)[tail], bits(q0)[at]) and torch.equal(s[tail], s0[at])
    q, s = moe.quantize_blocks_fp8(big)
    q0, s0 = moe.quantize_blocks_fp8(x)
    assert torch.equal(bits(q)[tail], bits(q0)[at]) and torch.equal(s[tail], s0[at])


# ------------------------------------------------------------------ batches
def _batch(g, sizes, T, prio_sizes=None, shared=0):
    """Sorted rows of given group sizes (prio_sizes: the priority segment's), each of a random token, the shared
    experts' groups of T rows.  Returns rows, offsets, E, nseg."""
    E = len(sizes)
    groups = (list(prio_sizes) if prio_sizes is not None else []) + list(sizes) + [T] * shared
    n = sum(groups)
    rows = torch.randint(0, T, (n,), generator=g, dtype=torch.int32)
    if shared:
        rows[n - T * shared:] = torch.arange(T, dtype=torch.int32).repeat(shared)
    offs = torch.zeros(len(groups) + 1, dtype=torch.int32)
    offs[1:] = torch.tensor(groups, dtype=torch.int32).cumsum(0)
    return rows, offs, E, 2 if prio_sizes is not None else 1


def _nb(n):
    return -(-n // 128)


def _codes(g, *shape):
    return (torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(F8)


def _scales(g, *shape):
    return torch.exp(torch.randn(shape, generator=g)) * 0.01


BATCHES = {
    "one_row": dict(sizes=[1], T=1),
    "one_group": dict(sizes=[70], T=70),
    "tiny_groups": dict(sizes=[1, 0, 3, 16, 0, 17, 2, 0], T=9),
    "medium_groups": dict(sizes=[40, 0, 61, 5, 33, 20], T=37),
    "large_groups": dict(sizes=[300, 1, 130, 257, 0, 90], T=150),
    "hot_expert": dict(sizes=[0, 700, 0, 0], T=90),
    "shared": dict(sizes=[5, 0, 12, 30], T=21, shared=2),
    "priority": dict(sizes=[20, 33, 0, 4], T=30, prio_sizes=[3, 0, 5, 20]),
    "priority_large": dict(sizes=[270, 33, 0, 140], T=64, prio_sizes=[3, 130, 5, 0], shared=1),
}


def _linear_case(g, b, K, O):
    rows, offs, E, nseg = _batch(g, **b)
    S = b.get("shared", 0)
    return (rows, offs, E, nseg, S, _codes(g, b["T"], K), _scales(g, b["T"], _nb(K)), _codes(g, E + S, O, K),
            _scales(g, E + S, _nb(O), _nb(K)))


def _linear_check(y, case):
    rows, offs, E, nseg, S, xq, xs, w, ws = case
    ref, mag = Q.grouped_linear(f64_of(xq), xs.numpy(), rows.numpy(), offs.tolist(), E, nseg, f64_of(w), ws.numpy())
    got = f64_of(y)
    tol = Q.sum_error(xq.shape[1]) * mag
    if fp8_plan.on_codes(fp8_plan.linear(len(rows), E, S, nseg, xq.shape[1], w.shape[1], y.dtype == torch.float32)):
        tol = tol + Q.linear_cut(f64_of(xq), xs.numpy(), rows.numpy(), offs.tolist(), E, nseg, f64_of(w), ws.numpy())
    tol = tol + torch.finfo(y.dtype).eps / 2 * (1 + 1e-6) * (np.abs(ref) + tol)
    assert np.all(np.abs(got - ref) <= tol), (np.abs(got - ref) / tol).max()
    _norms(got, ref, y.dtype)


def _norms(got, ref, dtype, row=0.0):
    """Errors of single values are far below their bounds: in the 2-norm a result, and each row of it, is its
    rounding off and little more (row: and that for single rows)."""
    step = torch.finfo(dtype).eps / 2
    off = np.linalg.norm(got - ref, axis=1)
    size = np.linalg.norm(ref, axis=1)
    assert np.linalg.norm(off) <= (step + 100 * 2.0 ** -24) * np.linalg.norm(size)
    assert np.all(off <= (row + 4 * step + 400 * 2.0 ** -24) * size), (off / size).max()


@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("K,O,dtype", [(64, 64, "f32"), (192, 320, "bf16"), (256, 128, "f32"), (704, 448, "bf16")])
def test_linear_parity(name, K, O, dtype):
    announce(f"linear fp8 {name} {K} {O} {dtype}")
    g = _gen(K + O + len(name))
    case = rows, offs, E, nseg, S, xq, xs, w, ws = _linear_case(g, BATCHES[name], K, O)
    dt = _dt(dtype)
    y = torch.full((len(rows), O), 7.0, dtype=dt, device=DEV)
    wp = moe.pack_fp8_codes(w).to(DEV)
    moe.grouped_linear_fp8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, S, nseg, wp, ws.to(DEV), y, x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _linear_check(y, case)
    # without a row list: rows in sorted order, the same bits
    at = rows.long()
    y2 = moe.grouped_linear_fp8(xq.view(torch.uint8)[at].view(F8).to(DEV), xs[at].to(DEV), offs.to(DEV), E, S, nseg, wp, ws.to(DEV),
                                out_dtype=dt)
    assert torch.equal(y, y2)


def test_linear_sums_are_those_of_fp32():
    """Well below the worst case that the other tests allow for: a dense product's error in the 2-norm is that of
    fp32 sums (a hundred half steps of the typical magnitude, not 128 * 2^-23 of all magnitudes together)."""
    announce("linear fp8 fp32 sums")
    g = _gen(5)
    rows, K, O = 200, 2048, 256
    xq, xs, w, ws = _codes(g, rows, K), _scales(g, rows, 16), _codes(g, 1, O, K), _scales(g, 1, 2, 16)
    offs = torch.tensor([0, rows], dtype=torch.int32)
    y = moe.grouped_linear_fp8(xq.to(DEV), xs.to(DEV), offs.to(DEV), 1, 0, 1, moe.pack_fp8_codes(w).to(DEV), ws.to(DEV),
                               out_dtype=torch.float32)
    ref, _ = Q.grouped_linear(f64_of(xq), xs.numpy(), np.arange(rows), [0, rows], 1, 1, f64_of(w), ws.numpy())
    rel = np.linalg.norm(f64_of(y) - ref) / np.linalg.norm(ref)
    assert rel <= 100 * 2.0 ** -24, rel


def test_linear_weights_past_two_gib():
    """Expert matrices whose offsets pass 2^31 bytes."""
    E, O, K = 40, 8192, 8192
    w = torch.zeros((E, O, K), dtype=torch.uint8, device=DEV).view(F8)
    g = _gen(11)
    last = _codes(g, O, K)
    w[E - 1].view(torch.uint8).copy_(moe.pack_fp8_codes(last.to(DEV)).view(torch.uint8))
    xq, xs, ws = _codes(g, 5, K), _scales(g, 5, 64), _scales(g, E, 64, 64)
    offs = torch.zeros(E + 1, dtype=torch.int32)
    offs[E] = 5
    y = moe.grouped_linear_fp8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, 0, 1, w, ws.to(DEV), out_dtype=torch.float32)
    ref, mag = Q.grouped_linear(f64_of(xq), xs.numpy(), np.arange(5), [0, 5], 1, 1, f64_of(last)[None], ws[E - 1:].numpy())
    assert np.all(np.abs(f64_of(y) - ref) <= (Q.sum_error(K) + 2.0 ** -24) * mag)


def test_rows_outside_the_groups_stay():
    g = _gen(12)
    xq, w = _codes(g, 20, 128).to(DEV), moe.pack_fp8_codes(_codes(g, 2, 64, 128)).to(DEV)
    one = torch.ones((20, 1), device=DEV)
    for offs in ([4, 9, 12], [0, 0, 0], [3, 3, 20], [20, 20, 20]):
        o = torch.tensor(offs, dtype=torch.int32, device=DEV)
        y = torch.full((20, 64), 3.0, device=DEV)
        moe.grouped_linear_fp8(xq, one, o, 2, 0, 1, w, torch.ones((2, 1, 1), device=DEV), y)
        assert (y[:offs[0]] == 3).all() and (y[offs[-1]:] == 3).all()
        if offs[-1] > offs[0]:
            assert not (y[offs[0]:offs[-1]] == 3).all(1).any()


# ------------------------------------------------------------------ ffn
def _ffn_case(g, b, d, I):
    rows, offs, E, nseg = _batch(g, **b)
    S = b.get("shared", 0)
    x = torch.randn((b["T"], d), generator=g) * torch.exp(0.5 * torch.randn((b["T"], 1), generator=g))
    q, s = Q.quantize_blocks(x.numpy())
    ws = [_codes(g, E + S, *sh) for sh in ((I, d), (I, d), (d, I))]
    ss = [_scales(g, E + S, _nb(r), _nb(c)) * 0.02 for r, c in ((I, d), (I, d), (d, I))]
    return rows, offs, E, nseg, S, torch.from_numpy(q).float().to(F8), torch.from_numpy(s), ws, ss


def _ffn_args(ws, ss):
    return [t for w, s in zip(ws, ss) for t in (moe.pack_fp8_codes(w).to(DEV), s.to(DEV))]


def _ffn_check(got, case):
    rows, offs, E, nseg, S, xq, xs, ws, ss = case
    ref, err, slack = Q.grouped_ffn(f64_of(xq), xs.numpy(), rows.numpy(), offs.tolist(), E, nseg,
                                    *[t for w, s in zip(ws, ss) for t in (f64_of(w), s.numpy())],
                                    on_codes=[fp8_plan.on_codes(k) for k in fp8_plan.ffn(len(rows), E, S, nseg, xq.shape[1], ws[0].shape[1])])
    tol = err + slack
    tol = tol + 2.0 ** -8 * (1 + 1e-6) * (np.abs(ref) + tol)
    off = np.abs(f64_of(got) - ref)
    assert np.all(off <= tol), (off / tol).max()
    # A row's SwiGLU product can be one large value, and its code next to a border: neighbours are up to 2^-3 apart.
    _norms(f64_of(got), ref, torch.bfloat16, row=2.0 ** -3)


@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("d,I", [(64, 64), (192, 192), (256, 320), (512, 256)])
def test_ffn_parity(name, d, I):
    announce(f"ffn fp8 {name} {d} {I}")
    g = _gen(d + I + len(name))
    case = rows, offs, E, nseg, S, xq, xs, ws, ss = _ffn_case(g, BATCHES[name], d, I)
    args = _ffn_args(ws, ss)
    h = torch.full((len(rows), d), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.grouped_ffn_fp8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, S, nseg, *args, h, x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _ffn_check(h, case)
    at = rows.long()
    h2 = moe.grouped_ffn_fp8(xq.view(torch.uint8)[at].view(F8).to(DEV), xs[at].to(DEV), offs.to(DEV), E, S, nseg, *args)
    assert torch.equal(h, h2)


# sizes at which the calls have several full tiles per block, and partial ones
LARGE = {
    "ragged": dict(sizes=[1, 0, 255, 256, 257, 129, 700, 40, 2000, 16, 1500, 33], T=900),
    "many": dict(sizes=[100 + 7 * (i % 13) for i in range(44)], T=700),
    "hot": dict(sizes=[0, 13100, 0, 300], T=2048),
    "priority": dict(sizes=[600, 0, 1, 900, 1300], T=800, prio_sizes=[64, 3, 0, 130, 1000], shared=1),
}


@pytest.mark.parametrize("name", LARGE)
@pytest.mark.parametrize("K,O,dtype", [(256, 1344, "f32"), (320, 1344, "bf16"), (704, 1280, "bf16"), (448, 1280, "f32")])
def test_linear_large(name, K, O, dtype):
    announce(f"linear fp8 large {name} {K} {O} {dtype}")
    g = _gen(K + O + len(name))
    case = rows, offs, E, nseg, S, xq, xs, w, ws = _linear_case(g, LARGE[name], K, O)
    args = [xq.to(DEV), xs.to(DEV), offs.to(DEV), E, S, nseg, moe.pack_fp8_codes(w).to(DEV), ws.to(DEV)]
    if K > 256:
        assert fp8_plan.linear(len(rows), E, S, nseg, K, O, dtype == "f32").startswith("tile")
    y = moe.grouped_linear_fp8(*args, x_rows=rows.to(DEV), out_dtype=_dt(dtype))
    torch.cuda.synchronize()
    _linear_check(y, case)
    assert torch.equal(y, moe.grouped_linear_fp8(*args, x_rows=rows.to(DEV), out_dtype=_dt(dtype)))


@pytest.mark.parametrize("name", LARGE)
@pytest.mark.parametrize("d,I", [(1344, 960), (960, 1088)])
def test_ffn_large(name, d, I):
    announce(f"ffn fp8 large {name} {d} {I}")
    g = _gen(d + I + len(name))
    case = rows, offs, E, nseg, S, xq, xs, ws, ss = _ffn_case(g, LARGE[name], d, I)
    args = _ffn_args(ws, ss)
    assert all(k.startswith("tile") for k in fp8_plan.ffn(len(rows), E, S, nseg, d, I))
    h = moe.grouped_ffn_fp8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, S, nseg, *args, x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _ffn_check(h, case)
    assert torch.equal(h, moe.grouped_ffn_fp8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, S, nseg, *args, x_rows=rows.to(DEV)))


def test_few_hundred_groups():
    g = _gen(15)
    for E, nseg in ((512, 1), (512, 2)):
        sizes = torch.randint(40, 80, (E,), generator=g).tolist()
        b = dict(sizes=sizes, T=300, **({"prio_sizes": torch.randint(0, 60, (E,), generator=g).tolist()} if nseg == 2 else {}))
        case = rows, offs, E, nseg, S, xq, xs, w, ws = _linear_case(g, b, 256, 256)
        y = moe.grouped_linear_fp8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, 0, nseg, moe.pack_fp8_codes(w).to(DEV), ws.to(DEV),
                                   x_rows=rows.to(DEV), out_dtype=torch.float32)
        _linear_check(y, case)


@pytest.mark.parametrize("rows,K,O", [(9, 8192, 64), (16, 2240, 192), (100, 64, 1024), (33, 1984, 512)])
def test_linear_few_rows_long_and_short_sums(rows, K, O):
    announce(f"linear fp8 few rows {rows} {K} {O}")
    g = _gen(rows + K)
    case = _linear_case(g, dict(sizes=[rows], T=rows), K, O)
    list_, offs, E, nseg, S, xq, xs, w, ws = case
    y = moe.grouped_linear_fp8(xq.to(DEV), xs.to(DEV), offs.to(DEV), 1, 0, 1, moe.pack_fp8_codes(w).to(DEV), ws.to(DEV),
                               x_rows=list_.to(DEV), out_dtype=torch.float32)
    _linear_check(y, case)


@pytest.mark.parametrize("d,I", [(64, 64), (4160, 192), (192, 2624), (1088, 1088)])
def test_ffn_few_rows_long_and_short_sums(d, I):
    announce(f"ffn fp8 few rows {d} {I}")
    g = _gen(d + I)
    case = rows, offs, E, nseg, S, xq, xs, ws, ss = _ffn_case(g, dict(sizes=[1, 0, 2, 0, 1], T=3), d, I)
    h = moe.grouped_ffn_fp8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, S, nseg, *_ffn_args(ws, ss), x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _ffn_check(h, case)


@pytest.mark.parametrize("name,d,I", [("tiny_groups", 256, 192), ("medium_groups", 320, 192), ("ragged", 960, 1088)])
def test_bad_rows_stay_in_their_rows(name, d, I):
    """A NaN scale, as the quantisers give it, makes a token's outputs NaN and no others; codes that are NaN likewise; a
    list entry out of range reaches no memory outside the tokens (it is held to the last token)."""
    announce(f"ffn fp8 bad rows {name}")
    g = _gen(13)
    rows, offs, E, nseg, S, xq, xs, ws, ss = _ffn_case(g, {**BATCHES, **LARGE}[name], d, I)
    args = _ffn_args(ws, ss)
    xd, sd, od, rd = xq.to(DEV), xs.to(DEV), offs.to(DEV), rows.to(DEV)
    call = lambda q=xd, s=sd, r=rd: moe.grouped_ffn_fp8(q, s, od, E, S, nseg, *args, x_rows=r)
    good = call()
    assert torch.isfinite(good).all()
    bad_s, bad_q = sd.clone(), xd.clone()
    bad_s[3, _nb(d) - 1] = np.nan
    bad_q.view(torch.uint8)[5, d - 1] = 0x7f
    bad = call(bad_q, bad_s)
    hit = (rd == 3) | (rd == 5)
    assert bool(hit.any()) and torch.isnan(bad[hit]).all() and torch.equal(bad[~hit], good[~hit])
    bad_q = xd.clone()                          # the code after a row's last one is the next row's first
    bad_q.view(torch.uint8)[:, 0][4] = 0xff
    hit = rd == 4
    bad = call(bad_q)
    assert torch.isnan(bad[hit]).all() and torch.equal(bad[~hit], good[~hit])
    r2 = rd.clone()
    r2[0], r2[1] = -5, 10 ** 6
    h = call(r=r2)
    r2[0], r2[1] = 0, xd.shape[0] - 1
    assert torch.equal(h, call(r=r2))
    assert not call(torch.zeros_like(xd.view(torch.uint8)).view(F8)).any()


def _captured(step, outs, change):
    """step() captured; each replay after change() is what step() gives eagerly."""
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        change()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name,d,I", [("tiny_groups", 256, 320), ("priority_large", 256, 320), ("ragged", 960, 1088)])
def test_norm_to_ffn_graph_and_streams(name, d, I):
    """The calls as they are used together (norm, then the FFN on its codes), captured and replayed with new inputs, on
    another stream, and twice at once with workspaces of their own."""
    announce(f"norm to ffn {name}")
    g = _gen(14)
    b = {**BATCHES, **LARGE}[name]
    rows, offs, E, nseg, S, xq, xs, ws, ss = _ffn_case(g, b, d, I)
    args = _ffn_args(ws, ss)
    T = b["T"]
    x, res, w = _rows(g, T, d, "bf16").to(DEV), _rows(g, T, d, "f32").to(DEV), torch.rand((d,), generator=g).to(DEV)
    out, y = torch.empty_like(res), torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
    q, s = torch.empty((T, d), dtype=torch.uint8, device=DEV).view(F8), torch.empty((T, _nb(d)), device=DEV)
    od, rd = offs.to(DEV), rows.to(DEV)
    h = torch.zeros((len(rows), d), dtype=torch.bfloat16, device=DEV)
    wk = torch.empty(moe.ffn_fp8_workspace_bytes(len(rows), I), dtype=torch.uint8, device=DEV)

    def step():
        moe.rmsnorm(x, w, 1e-6, res, out, y, "fp8", q, s)
        moe.grouped_ffn_fp8(q, s, od, E, S, nseg, *args, h, wk, x_rows=rd)

    def change():
        x.copy_(_rows(g, T, d, "bf16").to(DEV))
        res.copy_(_rows(g, T, d, "f32").to(DEV))
    _captured(step, [out, y, q.view(torch.uint8), s, h], change)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    for st in (s1, s2):
        with torch.cuda.stream(st):
            outs.append(moe.grouped_ffn_fp8(q, s, od, E, S, nseg, *args, x_rows=rd))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], h) and torch.equal(outs[1], h)


def test_norm_to_int8_linear():
    """int8 codes of the norm are rows of grouped_linear_i8."""
    announce("norm to int8 linear")
    g = _gen(17)
    x, w = _rows(g, 40, 256, "bf16").to(DEV), torch.rand((256,), generator=g).to(DEV)
    m = torch.randn((1, 128, 256), generator=g).to(DEV) * 0.05
    mq, ms = moe.quantize_rows_i8(m)
    y, q, s = moe.rmsnorm(x, w, codes="i8", y=torch.empty((40, 256), device=DEV))
    offs = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    got = moe.grouped_linear_i8(q, s, offs, 1, 0, 1, moe.pack_i8_codes(mq), ms, out_dtype=torch.float32)
    want = (q.double() * s.double()[:, None]) @ (mq[0].double() * ms[0].double()[:, None]).T.contiguous()
    assert (got.double() - want).abs().max() <= 4 * 2.0 ** -24 * want.abs().max()
    assert (got.double() - y.double() @ m[0].double().T.contiguous()).norm() <= 0.02 * want.norm()


def test_bindings_refuse_mismatches():
    z8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV).view(F8)
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=DEV)
    offs = z(3, dt=torch.int32)
    ok = dict(xq=z8(4, 192), x_scale=z(4, 2), group_offsets=offs, E=2, n_shared=0, nseg=1, w=z8(2, 64, 192), w_scale=z(2, 1, 2))
    for k, v in (("xq", z(4, 192)), ("xq", z(4, 192, dt=torch.uint8)), ("x_scale", z(4)), ("x_scale", z(4, 1)), ("x_scale", z(5, 2)),
                 ("group_offsets", z(4, dt=torch.int32)), ("w", z8(3, 64, 192)), ("w", z8(2, 64, 128)), ("w_scale", z(2, 2, 2)),
                 ("w_scale", z(2, 64)), ("E", 3), ("nseg", 2), ("x_scale", z(4, 2).cpu())):
        with pytest.raises((TypeError, ValueError)):
            moe.grouped_linear_fp8(**{**ok, k: v})
    with pytest.raises(TypeError):
        moe.grouped_linear_fp8(**ok, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.grouped_linear_fp8(**ok, y=z(3, 64))
    with pytest.raises(moe.MoeError):
        moe.grouped_linear_fp8(**{**ok, "xq": z8(4, 32), "x_scale": z(4, 1), "w": z8(2, 64, 32), "w_scale": z(2, 1, 1)})
    good = [z8(4, 64), z(4, 1), offs, 2, 0, 1, z8(2, 192, 64), z(2, 2, 1), z8(2, 192, 64), z(2, 2, 1), z8(2, 64, 192), z(2, 1, 2)]
    for i, v in ((0, z(4, 64)), (1, z(4, 2)), (6, z8(2, 192, 32)), (7, z(2, 1, 1)), (8, z8(2, 64, 64)), (10, z8(2, 192, 64)),
                 (11, z(2, 2, 1)), (3, 3)):
        with pytest.raises((TypeError, ValueError)):
            moe.grouped_ffn_fp8(*[v if j == i else t for j, t in enumerate(good)])
    with pytest.raises(moe.MoeError):
        moe.grouped_ffn_fp8(*good, workspace=z(64, dt=torch.uint8))
    with pytest.raises(TypeError):
        moe.grouped_ffn_fp8(*good, h_sorted=z(4, 64))
    with pytest.raises(ValueError):
        moe.grouped_ffn_fp8(*good, h_sorted=z(4, 128, dt=torch.bfloat16))
    e = moe.grouped_ffn_fp8(z8(0, 64), z(0, 1), *good[2:])
    assert e.shape == (0, 64)


def test_ffn_most_groups():
    """512 experts in two segments and 256 shared ones, each group of a few tens of rows."""
    announce("ffn fp8 most groups")
    g = _gen(18)
    sizes = lambda: torch.randint(0, 140, (512,), generator=g).tolist()
    case = rows, offs, E, nseg, S, xq, xs, ws, ss = _ffn_case(g, dict(sizes=sizes(), prio_sizes=sizes(), T=53, shared=256), 256, 256)
    h = moe.grouped_ffn_fp8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, S, nseg, *_ffn_args(ws, ss), x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _ffn_check(h, case)
