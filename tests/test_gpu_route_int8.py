"""GPU parity of routing with scores and of the int8 calls against their float64 definitions.

Tolerances, from the arithmetic of the calls:
  ids, codes, scales   equal
  weights              1e-6 relative (the call's promise)
  linear               fl(float(sum) * fl(sx * sw)), sums below 2^31: the conversion, the two products and the
                       output's rounding are each half a step: 3 * 2^-24 + finfo(out).eps / 2
  ffn                  2^-8 (bf16) of the value; 2e-5 of the sum of magnitudes of the block terms for the fp32 steps
                       (each value of the SwiGLU product is within (|g| + 8) * 2^-23 of its exact value, |g| < 80 here,
                       its block's scale likewise, and the blocks are added in fp32); and every code whose exact quotient
                       lies within 127 * 2e-5 of a border may be the neighbour: the oracle's slack
"""
import numpy as np
import pytest
import torch

from oracle import int8_oracle as Q
from helpers import announce, f64_of, np_of, require_gpu

import top_expert_routing_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
MARGIN = 127 * 2e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ route
ROUTE = [
    # T, E, k, score, bias, groups, top_groups, rank, renorm, scale, dtype
    (1, 1, 1, "softmax", False, 1, 1, "max", True, 1.0, "f32"),
    (5, 3, 3, "sigmoid", True, 1, 1, "max", True, 2.5, "f32"),
    (1, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5, "f32"),
    (67, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5, "bf16"),
    (130, 160, 6, "softmax", False, 8, 3, "max", False, 16.0, "f32"),
    (33, 160, 6, "softmax", True, 8, 3, "top2", True, 1.0, "bf16"),
    (40, 64, 8, "softmax", False, 1, 1, "max", True, 1.0, "f32"),
    (40, 512, 16, "sigmoid", False, 64, 5, "top2", True, 1.0, "f32"),
    (21, 512, 512, "softmax", True, 1, 1, "max", False, 1.0, "f32"),
    (19, 64, 5, "sigmoid", True, 64, 9, "top2", False, -1.5, "f32"),   # groups of one expert
    (23, 99, 7, "sigmoid", False, 3, 1, "top2", True, 0.0, "bf16"),
    (300, 384, 8, "sigmoid", True, 1, 1, "max", True, 2.827, "f32"),
    (64, 72, 36, "softmax", True, 2, 1, "max", True, 1.0, "f32"),
]


def _route_check(l, k, score, bias, groups, top, rank, renorm, scale):
    ids, w = moe.route(l.to(DEV), k, score, None if bias is None else bias.to(DEV), groups, top, rank, renorm, scale)
    torch.cuda.synchronize()
    ref_ids, ref_w = Q.route(f64_of(l), k, score, None if bias is None else f64_of(bias), groups, top, rank, renorm, scale)
    np.testing.assert_array_equal(np_of(ids), ref_ids)
    got = np_of(w).astype(np.float64)
    assert np.all(np.abs(got - ref_w) <= 1e-6 * np.abs(ref_w) + 1e-37), np.abs(got - ref_w).max()


@pytest.mark.parametrize("case", ROUTE)
def test_route_parity(case):
    T, E, k, score, has_bias, groups, top, rank, renorm, scale, dtype = case
    announce(f"route {case}")
    g = _gen(T + E + k)
    l = torch.randn((T, E), generator=g) * 2
    if dtype == "bf16":
        l = l.bfloat16()
    bias = torch.randn(E, generator=g) * 0.2 if has_bias else None
    _route_check(l, k, score, bias, groups, top, rank, renorm, scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("has_bias", [False, True])
@pytest.mark.parametrize("rank", ["max", "top2"])
def test_route_ties(score, has_bias, rank):
    """Few distinct logits and biases: ties among experts and among groups everywhere."""
    announce(f"route ties {score} {has_bias} {rank}")
    g = _gen(3)
    l = torch.randint(-2, 3, (96, 64), generator=g).float()
    bias = torch.randint(0, 2, (64,), generator=g).float() * 0.5 if has_bias else None
    _route_check(l, 9, score, bias, 8, 3, rank, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("has_bias", [False, True])
def test_route_near_ties(score, has_bias):
    """Scores that differ by a few fp32 steps or less fall as double says."""
    announce(f"route near ties {score} {has_bias}")
    g = _gen(4)
    l = (1.0 + torch.randint(0, 6, (128, 128), generator=g).float() * 2.0 ** -23) * torch.randint(1, 3, (128, 1), generator=g)
    bias = 0.25 + torch.randint(0, 4, (128,), generator=g).float() * 2.0 ** -25 if has_bias else None
    _route_check(l, 12, score, bias, 4, 2, "top2", True, 1.0)
    # saturated sigmoids: distinct logits whose scores round to 1 even in double
    _route_check(30.0 + torch.randint(0, 60, (16, 128), generator=g).float(), 6, score, bias, 1, 1, "max", True, 1.0)


def test_route_special_values():
    g = _gen(5)
    l = torch.randn((12, 64), generator=g)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, 5:] = -np.inf                       # fewer finite experts than k
    l[3, 7] = np.inf
    l[4, [9, 3]] = np.inf
    l[5, ::2] = np.nan
    l[6] = torch.finfo(torch.float32).min
    l[7] = -800.0                            # sigmoids below the smallest double
    l[8] = 0.0
    l[8, ::3] = -0.0
    bias = torch.randn(64, generator=g) * 0.1
    bias[[2, 40]] = -np.inf
    bias[[11]] = np.nan
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            for groups, top, rank in ((1, 1, "max"), (8, 2, "max"), (8, 2, "top2")):
                for renorm in (True, False):
                    announce(f"route special {score} {b is not None} {groups} {rank} {renorm}")
                    _route_check(l, 8, score, b, groups, top, rank, renorm, 1.0)
    # fp64's exp of -800 is 0: sums of no mass give weight 0
    ids, w = moe.route(torch.full((1, 64), -np.inf).to(DEV), 4, "sigmoid")
    assert ids.tolist() == [[0, 1, 2, 3]] and w.tolist() == [[0.0] * 4]


def test_route_rows_do_not_depend_on_the_batch():
    g = _gen(6)
    l = torch.randn((500, 256), generator=g).to(DEV)
    b = (torch.randn(256, generator=g) * 0.1).to(DEV)
    ids, w = moe.route(l, 8, "sigmoid", b, 8, 4, "top2", True, 2.5)
    for t in (0, 3, 255, 499):
        i1, w1 = moe.route(l[t:t + 1], 8, "sigmoid", b, 8, 4, "top2", True, 2.5)
        assert torch.equal(i1[0], ids[t]) and torch.equal(w1[0], w[t])


# ------------------------------------------------------------------ quantize
def _quant_check(x):
    q, s = moe.quantize_rows_i8(x.to(DEV))
    torch.cuda.synchronize()
    rq, rs = Q.quantize(f64_of(x))
    np.testing.assert_array_equal(np_of(s), rs)
    np.testing.assert_array_equal(np_of(q), rq)


@pytest.mark.parametrize("T,d,dtype", [(1, 8, "bf16"), (7, 136, "f32"), (33, 2048, "bf16"), (5, 4104, "f32"),
                                       (3, 8200, "bf16"), (70, 2880, "f32"), (257, 512, "bf16")])
def test_quantize_parity(T, d, dtype):
    announce(f"quantize {T} {d} {dtype}")
    x = torch.randn((T, d), generator=_gen(T + d)) * torch.exp(torch.randn((T, 1), generator=_gen(d)))
    _quant_check(x.bfloat16() if dtype == "bf16" else x)


def test_quantize_borders():
    """Exact halves, their neighbours, every magnitude of scale, subnormals, zeros, infinities, NaN."""
    halves = torch.arange(-127, 128).float().clamp(-126.5, 126.5)
    halves = torch.cat([halves + 0.5, torch.tensor([127.0])]).clamp(-127, 127)          # scale 1: 256 values
    rows = []
    for e in (-120, -60, -3, 0, 5, 90):
        r = halves * 2.0 ** e
        rows += [r, torch.nextafter(r, torch.zeros(())), torch.nextafter(r, r * 4)]
    rows = [torch.cat([r[:255], torch.tensor([127.0 * 2.0 ** int(e)])]) for r, e in zip(rows, np.repeat((-120, -60, -3, 0, 5, 90), 3))]
    for e in (-149, -148, -145, -140, -133, -126):
        rows.append((torch.arange(256).float() - 100) * 2.0 ** e)
    for bad in (np.inf, -np.inf, np.nan):
        r = torch.ones(256)
        r[77] = bad
        rows.append(r)
    rows += [torch.zeros(256), torch.full((256,), 3.4e38), torch.full((256,), -1e-45)]
    # a third of a step and odd scales: quotients next to halves
    g = _gen(8)
    for _ in range(40):
        s = torch.rand((), generator=g) + 0.5
        r = (torch.randint(-127, 127, (256,), generator=g).float() + 0.5) * s
        r[0] = 127.0 * s
        rows.append(r)
    _quant_check(torch.stack(rows))
    _quant_check(torch.stack(rows).bfloat16())


def test_quantize_outputs_and_shapes():
    x = torch.randn((2, 3, 64), generator=_gen(9)).to(DEV)
    q, s = moe.quantize_rows_i8(x)
    assert q.shape == (2, 3, 64) and s.shape == (2, 3)
    q2, s2 = moe.quantize_rows_i8(x.view(6, 64))
    assert torch.equal(q.view(6, 64), q2) and torch.equal(s.view(6), s2)
    e = moe.quantize_rows_i8(torch.empty((0, 64), device=DEV))
    assert e[0].shape == (0, 64) and e[1].shape == (0,)
    for bad in (x.half(), x[..., ::2], x.cpu()):
        with pytest.raises((TypeError, ValueError)):
            moe.quantize_rows_i8(bad)
    with pytest.raises(moe.MoeError):
        moe.quantize_rows_i8(torch.zeros((2, 12), device=DEV))


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


def _codes(g, *shape):
    q = (torch.randn(shape, generator=g) * 40).round().clamp(-128, 127).to(torch.int8)
    return q


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


@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("K,O,dtype", [(64, 64, "f32"), (192, 320, "bf16"), (256, 128, "f32"), (704, 448, "bf16")])
def test_linear_parity(name, K, O, dtype):
    announce(f"linear {name} {K} {O} {dtype}")
    g = _gen(K + O + len(name))
    b = BATCHES[name]
    rows, offs, E, nseg = _batch(g, **b)
    S = b.get("shared", 0)
    xq, xs = _codes(g, b["T"], K), torch.rand(b["T"], generator=g) + 0.1
    w, ws = _codes(g, E + S, O, K), torch.rand((E + S, O), generator=g) + 0.1
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    y = torch.full((len(rows), O), 7.0, dtype=dt, device=DEV)
    moe.grouped_linear_i8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, S, nseg, moe.pack_i8_codes(w).to(DEV), ws.to(DEV), y,
                          x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    ref = Q.grouped_linear(xq.numpy(), xs.numpy(), rows.numpy(), offs.tolist(), E, nseg, w.numpy(), ws.numpy())
    got = f64_of(y)
    tol = (3 * 2.0 ** -24 + torch.finfo(dt).eps / 2) * (1 + 1e-6)
    assert np.all(np.abs(got - ref) <= tol * np.abs(ref)), (np.abs(got - ref) / np.maximum(np.abs(ref), 1e-9)).max()
    # without a row list: rows in sorted order, the same bits
    y2 = moe.grouped_linear_i8(xq[rows.long()].to(DEV), xs[rows.long()].to(DEV), offs.to(DEV), E, S, nseg,
                               moe.pack_i8_codes(w).to(DEV), ws.to(DEV), out_dtype=dt)
    assert torch.equal(y, y2)


def test_linear_largest_sums():
    """K = 131072 of the largest codes: 2^31 - 2^17 at most, still exact; and many K chunks."""
    K = 131072
    xq = torch.full((3, K), -127, dtype=torch.int8)
    w = torch.full((1, 64, K), -128, dtype=torch.int8)
    w[0, 1] = 127
    y = moe.grouped_linear_i8(xq.to(DEV), torch.ones(3, device=DEV), torch.tensor([0, 3], dtype=torch.int32, device=DEV), 1, 0, 1,
                              moe.pack_i8_codes(w).to(DEV), torch.ones((1, 64), device=DEV), out_dtype=torch.float32)
    ref = np.full((3, 64), 127.0 * 128 * K)
    ref[:, 1] = -127.0 * 127 * K
    assert np.all(np.abs(f64_of(y) - ref) <= 3 * 2.0 ** -24 * np.abs(ref))


def test_linear_weights_past_two_gib():
    """Expert matrices whose offsets pass 2^31 bytes."""
    E, O, K = 40, 8192, 8192
    w = torch.zeros((E, O, K), dtype=torch.int8, device=DEV)
    g = _gen(11)
    last = _codes(g, O, K)
    w[E - 1] = moe.pack_i8_codes(last.to(DEV))
    xq = _codes(g, 5, K)
    offs = torch.zeros(E + 1, dtype=torch.int32)
    offs[E] = 5
    ws = torch.ones((E, O))
    y = moe.grouped_linear_i8(xq.to(DEV), torch.ones(5, device=DEV), offs.to(DEV), E, 0, 1, w, ws.to(DEV), out_dtype=torch.float32)
    ref = xq.double() @ last.double().T
    assert np.all(np.abs(f64_of(y) - ref.numpy()) <= 3 * 2.0 ** -24 * np.abs(ref.numpy()))


def test_rows_outside_the_groups_stay():
    g = _gen(12)
    xq, w = _codes(g, 20, 128).to(DEV), moe.pack_i8_codes(_codes(g, 2, 64, 128)).to(DEV)
    for offs in ([4, 9, 12], [0, 0, 0], [3, 3, 20], [20, 20, 20]):
        o = torch.tensor(offs, dtype=torch.int32, device=DEV)
        y = torch.full((20, 64), 3.0, device=DEV)
        moe.grouped_linear_i8(xq, torch.ones(20, device=DEV), o, 2, 0, 1, w, torch.ones((2, 64), device=DEV), y)
        assert (y[:offs[0]] == 3).all() and (y[offs[-1]:] == 3).all()
        if offs[-1] > offs[0]:
            assert not (y[offs[0]:offs[-1]] == 3).all(1).any()


# ------------------------------------------------------------------ ffn
def _ffn_case(g, b, d, I):
    rows, offs, E, nseg = _batch(g, **b)
    S = b.get("shared", 0)
    x = (torch.randn((b["T"], d), generator=g) * torch.exp(0.5 * torch.randn((b["T"], 1), generator=g))).bfloat16()
    ws = [_codes(g, E + S, *sh) for sh in ((I, d), (I, d), (d, I))]
    ss = [(torch.rand((E + S, n), generator=g) + 0.5) * c for n, c in ((I, 0.02 / 40), (I, 0.02 / 40), (d, 0.02 / 40))]
    return rows, offs, E, nseg, S, x, ws, ss


def _ffn_args(ws, ss):
    return [t for w, s in zip(ws, ss) for t in (moe.pack_i8_codes(w).to(DEV), s.to(DEV))]


def _ffn_check(got, x, rows, offs, E, nseg, ws, ss):
    ref, slack = Q.grouped_ffn(f64_of(x), rows.numpy(), offs.tolist(), E, nseg, *[t.numpy() for w, s in zip(ws, ss) for t in (w, s)],
                               margin=MARGIN)
    # magnitudes of the block terms: |codes| with |weights|
    mag = Q.grouped_ffn_magnitude(f64_of(x), rows.numpy(), offs.tolist(), E, nseg, *[t.numpy() for w, s in zip(ws, ss) for t in (w, s)])
    err = np.abs(got - ref)
    ok = err <= 2.0 ** -8 * (1 + 1e-6) * (np.abs(ref) + slack) + 2e-5 * mag + slack
    assert ok.all(), (err.max(), np.abs(ref).max(), (~ok).sum())


@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("d,I", [(64, 64), (192, 192), (256, 320), (512, 256)])
def test_ffn_parity(name, d, I):
    announce(f"ffn {name} {d} {I}")
    g = _gen(d + I + len(name))
    rows, offs, E, nseg, S, x, ws, ss = _ffn_case(g, BATCHES[name], d, I)
    h = torch.full((len(rows), d), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *_ffn_args(ws, ss), h, x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _ffn_check(f64_of(h), x, rows, offs, E, nseg, ws, ss)
    h2 = moe.grouped_ffn_i8(x[rows.long()].to(DEV), offs.to(DEV), E, S, nseg, *_ffn_args(ws, ss))
    assert torch.equal(h, h2)


# sizes at which the calls run on the LDS-tiled kernels (several tiles per block, partial ones, 128- and 256-row tiles)
LARGE = {
    "ragged": dict(sizes=[1, 0, 255, 256, 257, 129, 700, 40, 2000, 16, 1500, 33], T=900),
    "many": dict(sizes=[100 + 7 * (i % 13) for i in range(44)], T=700),
    "hot": dict(sizes=[0, 13100, 0, 300], T=2048),
    "priority": dict(sizes=[600, 0, 1, 900, 1300], T=800, prio_sizes=[64, 3, 0, 130, 1000], shared=1),
}


@pytest.mark.parametrize("name", LARGE)
@pytest.mark.parametrize("K,O,dtype", [(256, 1344, "f32"), (320, 1344, "bf16"), (704, 1280, "bf16")])
def test_linear_large(name, K, O, dtype):
    announce(f"linear large {name} {K} {O} {dtype}")
    g = _gen(K + O + len(name))
    b = LARGE[name]
    rows, offs, E, nseg = _batch(g, **b)
    S = b.get("shared", 0)
    xq, xs = _codes(g, b["T"], K), torch.rand(b["T"], generator=g) + 0.1
    w, ws = _codes(g, E + S, O, K), torch.rand((E + S, O), generator=g) + 0.1
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    args = [t.to(DEV) for t in (xq, xs, offs)] + [E, S, nseg, moe.pack_i8_codes(w).to(DEV), ws.to(DEV)]
    y = moe.grouped_linear_i8(*args, x_rows=rows.to(DEV), out_dtype=dt)
    torch.cuda.synchronize()
    ref = Q.grouped_linear(xq.numpy(), xs.numpy(), rows.numpy(), offs.tolist(), E, nseg, w.numpy(), ws.numpy())
    tol = (3 * 2.0 ** -24 + torch.finfo(dt).eps / 2) * (1 + 1e-6)
    assert np.all(np.abs(f64_of(y) - ref) <= tol * np.abs(ref))
    again = moe.grouped_linear_i8(*args, x_rows=rows.to(DEV), out_dtype=dt)
    assert torch.equal(y, again)


@pytest.mark.parametrize("name", LARGE)
@pytest.mark.parametrize("d,I", [(320, 960), (1344, 704)])
def test_ffn_large(name, d, I):
    announce(f"ffn large {name} {d} {I}")
    g = _gen(d + I + len(name))
    rows, offs, E, nseg, S, x, ws, ss = _ffn_case(g, LARGE[name], d, I)
    args = _ffn_args(ws, ss)
    h = moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *args, x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _ffn_check(f64_of(h), x, rows, offs, E, nseg, ws, ss)
    again = moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *args, x_rows=rows.to(DEV))
    assert torch.equal(h, again)


def test_linear_few_hundred_groups():
    """More groups than the 128-row tiles' lists hold (the 256-row ones take them), and their largest number."""
    g = _gen(15)
    for E, nseg in ((512, 1), (512, 2)):
        sizes = torch.randint(40, 80, (E,), generator=g).tolist()
        b = dict(sizes=sizes, T=300, **({"prio_sizes": torch.randint(0, 60, (E,), generator=g).tolist()} if nseg == 2 else {}))
        rows, offs, E, nseg = _batch(g, **b)
        K, O = 256, 256
        xq, xs = _codes(g, 300, K), torch.rand(300, generator=g) + 0.1
        w, ws = _codes(g, E, O, K), torch.rand((E, O), generator=g) + 0.1
        y = moe.grouped_linear_i8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, 0, nseg, moe.pack_i8_codes(w).to(DEV), ws.to(DEV),
                                  x_rows=rows.to(DEV), out_dtype=torch.float32)
        ref = Q.grouped_linear(xq.numpy(), xs.numpy(), rows.numpy(), offs.tolist(), E, nseg, w.numpy(), ws.numpy())
        assert np.all(np.abs(f64_of(y) - ref) <= 4 * 2.0 ** -24 * np.abs(ref))


def test_ffn_bad_rows_stay_in_their_rows():
    """NaN and infinities in a token row make its outputs NaN and no others; so does a list entry out of range reach
    no memory outside the tokens (it is held to the last token)."""
    g = _gen(13)
    rows, offs, E, nseg, S, x, ws, ss = _ffn_case(g, BATCHES["medium_groups"], 256, 192)
    args = _ffn_args(ws, ss)
    good = moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *args, x_rows=rows.to(DEV))
    xb = x.clone()
    xb[3, 17] = np.nan
    xb[5, 0] = np.inf
    bad = moe.grouped_ffn_i8(xb.to(DEV), offs.to(DEV), E, S, nseg, *args, x_rows=rows.to(DEV))
    hit = ((rows == 3) | (rows == 5)).to(DEV)
    assert torch.isnan(bad[hit]).all() and torch.equal(bad[~hit], good[~hit]) and bool(hit.any())
    r2 = rows.clone()
    r2[0], r2[1] = -5, 10 ** 6
    h = moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *args, x_rows=r2.to(DEV))
    r2[0], r2[1] = 0, x.shape[0] - 1
    assert torch.equal(h, moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *args, x_rows=r2.to(DEV)))
    # all-zero tokens give zeros
    z = moe.grouped_ffn_i8(torch.zeros_like(x).to(DEV), offs.to(DEV), E, S, nseg, *args, x_rows=rows.to(DEV))
    assert not z.any()


@pytest.mark.parametrize("name", ["tiny_groups", "priority_large"])
def test_route_to_ffn_graph_and_streams(name):
    """The calls as they are used together (route, then the int8 FFN), captured and replayed with new inputs, on
    another stream, and twice at once with workspaces of their own."""
    g = _gen(14)
    rows, offs, E, nseg, S, x, ws, ss = _ffn_case(g, BATCHES[name], 256, 320)
    args = _ffn_args(ws, ss)
    T = x.shape[0]
    l = torch.randn((T, 64), generator=g).to(DEV)
    xd, od, rd = x.to(DEV), offs.to(DEV), rows.to(DEV)
    nb = moe.ffn_i8_workspace_bytes(len(rows), T, 256, 320)
    ids, w = torch.zeros((T, 4), dtype=torch.int32, device=DEV), torch.zeros((T, 4), device=DEV)
    h = torch.zeros((len(rows), 256), dtype=torch.bfloat16, device=DEV)
    wk = torch.empty(nb, dtype=torch.uint8, device=DEV)

    def step():
        moe.route(l, 4, "sigmoid", None, 8, 2, "top2", True, 2.5, ids, w)
        moe.grouped_ffn_i8(xd, od, E, S, nseg, *args, h, wk, x_rows=rd)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        xd.copy_(torch.randn((T, 256), generator=g).to(DEV))
        l.copy_(torch.randn((T, 64), generator=g).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = (ids.clone(), w.clone(), h.clone())
        ids.zero_(), w.zero_(), h.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (ids, w, h)):
            assert torch.equal(a, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    for s in (s1, s2):
        with torch.cuda.stream(s):
            outs.append(moe.grouped_ffn_i8(xd, od, E, S, nseg, *args, x_rows=rd))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], h) and torch.equal(outs[1], h)


@pytest.mark.parametrize("T,prio,S,fused", [(48, 0, 1, True), (300, 16, 0, True), (7, 0, 0, False)])
def test_layer_with_routing_and_int8_experts(T, prio, S, fused):
    """MoeLayer with both: its gate is route()'s, its FFN grouped_ffn_i8's, eagerly and through bound_calls."""
    import workloads
    wl = workloads.custom(T=T, E=16, k=4, d=256, I=192, dtype="bf16", S=S, n_priority=prio, seed=3, device=DEV)
    s = wl.spec
    q = []
    for w in (wl.w_gate, wl.w_up, wl.w_down):
        c, sc = moe.quantize_rows_i8(w)
        q += [moe.pack_i8_codes(c), sc]
    bias = (torch.randn(16, generator=_gen(16)) * 0.1).to(DEV)
    routing = dict(score="sigmoid", bias=bias, n_groups=4, top_groups=2, group_rank="top2", scale=2.5)
    layer = moe.MoeLayer(s.E, s.k, s.d, s.I, s.T, torch.bfloat16, None, None, None, n_shared=S, n_priority=prio, device=DEV,
                         fused_gather=fused, int8_weights=tuple(q), routing=routing)
    y = layer.forward(wl.logits, wl.x).clone()
    ids, w = Q.route(f64_of(wl.logits), 4, "sigmoid", f64_of(bias), 4, 2, "top2", True, 2.5)
    np.testing.assert_array_equal(np_of(layer.topk_ids), ids)
    p = moe.permute(layer.topk_ids, 16, S, prio)
    h = moe.grouped_ffn_i8(wl.x, p["group_offsets"], 16, S, 2 if prio else 1, *q, x_rows=p["sorted_token"])
    assert torch.equal(h, layer.h_sorted)
    assert torch.equal(y, moe.combine(h, p["flat_to_sorted"], layer.topk_w, S))
    # against the layer on the weights that the codes stand for: a few per cent (8-bit steps of rows and blocks)
    full = [(moe.quantize_rows_i8(t)[0].float() * moe.quantize_rows_i8(t)[1].unsqueeze(-1)).bfloat16() for t in (wl.w_gate, wl.w_up, wl.w_down)]
    h16 = moe.grouped_ffn(wl.x, p["group_offsets"], 16, S, 2 if prio else 1, *full, x_rows=p["sorted_token"])
    assert (h.float() - h16.float()).norm() < 0.05 * h16.float().norm()
    layer.y.zero_()
    for name, fn, a in layer.bound_calls(wl.logits, wl.x):
        assert fn(*a) == 0, name
    torch.cuda.synchronize()
    assert torch.equal(layer.y, y)
    for bad in (dict(routing=dict(scores="sigmoid")), dict(int8_weights=tuple(q), fused_combine=True)):
        with pytest.raises(ValueError):
            moe.MoeLayer(s.E, s.k, s.d, s.I, s.T, torch.bfloat16, None, None, None, device=DEV, **bad)


def test_bindings_refuse_mismatches():
    z = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt, device=DEV)
    f = torch.float32
    offs = z(3, dt=torch.int32)
    ok = dict(xq=z(4, 64), x_scale=z(4, dt=f), group_offsets=offs, E=2, n_shared=0, nseg=1, w=z(2, 64, 64), w_scale=z(2, 64, dt=f))
    for k, v in (("xq", z(4, 64, dt=f)), ("x_scale", z(5, dt=f)), ("group_offsets", z(4, dt=torch.int32)), ("w", z(3, 64, 64)),
                 ("w", z(2, 64, 128)), ("w_scale", z(2, 63, dt=f)), ("E", 3), ("nseg", 2), ("x_scale", z(4, dt=f).cpu())):
        with pytest.raises((TypeError, ValueError)):
            moe.grouped_linear_i8(**{**ok, k: v})
    with pytest.raises(TypeError):
        moe.grouped_linear_i8(**ok, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.grouped_linear_i8(**ok, y=z(3, 64, dt=f))
    with pytest.raises(moe.MoeError):
        moe.grouped_linear_i8(**{**ok, "xq": z(4, 32), "w": z(2, 64, 32)})
    x = z(4, 64, dt=torch.bfloat16)
    good = [offs, 2, 0, 1, z(2, 128, 64), z(2, 128, dt=f), z(2, 128, 64), z(2, 128, dt=f), z(2, 64, 128), z(2, 64, dt=f)]
    for i, v in ((4, z(2, 128, 32)), (5, z(2, 127, dt=f)), (6, z(2, 64, 64)), (8, z(2, 128, 64)), (9, z(2, 128, dt=f)), (1, 3)):
        with pytest.raises((TypeError, ValueError)):
            moe.grouped_ffn_i8(x, *[v if j == i else t for j, t in enumerate(good)])
    with pytest.raises(moe.MoeError):
        moe.grouped_ffn_i8(x, *good, workspace=z(64, dt=torch.uint8))
    with pytest.raises((TypeError, ValueError)):
        moe.grouped_ffn_i8(x.float(), *good)
    l = z(4, 16, dt=f)
    for kw in (dict(k=0), dict(k=17), dict(k=2, n_groups=3), dict(k=9, n_groups=4, top_groups=2), dict(k=2, scale=float("inf"))):
        with pytest.raises(moe.MoeError):
            moe.route(l, **kw)
    for kw in (dict(score="tanh"), dict(group_rank="mean"), dict(bias=z(15, dt=f)), dict(topk_ids=z(4, 2, dt=f))):
        with pytest.raises((TypeError, ValueError)):
            moe.route(l, 2, **kw)
    with pytest.raises(TypeError):
        moe.route(l.half(), 2)


# ------------------------------------------------------------------ the largest sizes
def test_ffn_most_groups():
    """512 experts in two segments and 256 shared ones, each group of a few tens of rows, on the LDS-tiled kernels."""
    announce("ffn most groups")
    g = _gen(18)
    sizes = lambda: torch.randint(0, 140, (512,), generator=g).tolist()
    d, I = 256, 256
    rows, offs, E, nseg, S, x, ws, ss = _ffn_case(g, dict(sizes=sizes(), prio_sizes=sizes(), T=53, shared=256), d, I)
    h = moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *_ffn_args(ws, ss), x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _ffn_check(f64_of(h), x, rows, offs, E, nseg, ws, ss)


def test_quantize_more_rows_than_one_launch():
    announce("quantize 2^23 + 77 rows")
    x = torch.randn((4096, 8), generator=_gen(19)).bfloat16().to(DEV)
    q0, s0 = moe.quantize_rows_i8(x)
    T = 2 ** 23 + 77
    q, s = moe.quantize_rows_i8(x.repeat(2049, 1)[:T].contiguous())
    assert torch.equal(q, q0.repeat(2049, 1)[:T]) and torch.equal(s, s0.repeat(2049)[:T])


def test_route_more_tokens_than_one_launch():
    announce("route 2^25 + 33 tokens")
    l = torch.randn((4096, 4), generator=_gen(20)).bfloat16().to(DEV)
    i0, w0 = moe.route(l, 2, "sigmoid")
    T = 2 ** 25 + 33
    i, w = moe.route(l.repeat(8193, 1)[:T].contiguous(), 2, "sigmoid")
    assert torch.equal(i, i0.repeat(8193, 1)[:T]) and torch.equal(w, w0.repeat(8193, 1)[:T])


def test_layer_refuses_what_its_raw_calls_would_read_wrongly():
    z = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt, device=DEV)
    f = torch.float32
    E, k, d, I, T = 4, 2, 64, 128, 5
    good = (z(E, I, d), z(E, I, dt=f), z(E, I, d), z(E, I, dt=f), z(E, d, I), z(E, d, dt=f))
    make = lambda **kw: moe.MoeLayer(E, k, d, I, T, torch.bfloat16, None, None, None, device=DEV, **{"int8_weights": good, **kw})
    for i, v in ((0, z(E, I, d + 64)), (1, z(E, I - 1, dt=f)), (4, z(E, I, d)), (5, z(E, d))):
        with pytest.raises((TypeError, ValueError)):
            make(int8_weights=tuple(v if j == i else t for j, t in enumerate(good)))
    for r in (dict(bias=z(E - 1, dt=f)), dict(bias=z(E)), dict(score="tanh"), dict(group_rank="mean"), dict(bias=z(E, dt=f).cpu())):
        with pytest.raises((TypeError, ValueError)):
            make(routing=r)
    layer = make(routing=dict(score="sigmoid"))
    x = z(T, d, dt=torch.bfloat16)
    layer.bound_calls(z(T, E, dt=f), x)
    with pytest.raises(ValueError):
        layer.bound_calls(z(T, E + 1, dt=f), x)
    layer.int8_weights = good[:5] + (z(E, d - 1, dt=f),)
    with pytest.raises(ValueError):
        layer.bound_calls(z(T, E, dt=f), x)


# groups of some 20 and 60 rows, enough of them that every CU has work at 32 rows a tile
STREAM = {
    "rows_32": dict(sizes=[14 + (5 * i) % 13 for i in range(64)], T=230, shared=1),
    "rows_64": dict(sizes=[45 + (7 * i) % 31 for i in range(64)], T=150),
    "rows_64_priority": dict(sizes=[40 + (7 * i) % 31 for i in range(48)], T=90, prio_sizes=[(11 * i) % 70 + 20 for i in range(48)]),
}


@pytest.mark.parametrize("name", STREAM)
@pytest.mark.parametrize("K,O,dtype", [(192, 448, "f32"), (576, 384, "bf16")])
def test_linear_many_small_groups(name, K, O, dtype):
    announce(f"linear small groups {name} {K} {O} {dtype}")
    g = _gen(K + O + len(name))
    b = STREAM[name]
    rows, offs, E, nseg = _batch(g, **b)
    S = b.get("shared", 0)
    xq, xs = _codes(g, b["T"], K), torch.rand(b["T"], generator=g) + 0.1
    w, ws = _codes(g, E + S, O, K), torch.rand((E + S, O), generator=g) + 0.1
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    y = moe.grouped_linear_i8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, S, nseg, moe.pack_i8_codes(w).to(DEV), ws.to(DEV),
                              x_rows=rows.to(DEV), out_dtype=dt)
    torch.cuda.synchronize()
    ref = Q.grouped_linear(xq.numpy(), xs.numpy(), rows.numpy(), offs.tolist(), E, nseg, w.numpy(), ws.numpy())
    tol = (3 * 2.0 ** -24 + torch.finfo(dt).eps / 2) * (1 + 1e-6)
    assert np.all(np.abs(f64_of(y) - ref) <= tol * np.abs(ref))


@pytest.mark.parametrize("name", STREAM)
def test_ffn_many_small_groups(name):
    announce(f"ffn small groups {name}")
    g = _gen(30 + len(name))
    rows, offs, E, nseg, S, x, ws, ss = _ffn_case(g, STREAM[name], 448, 576)
    h = moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *_ffn_args(ws, ss), x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _ffn_check(f64_of(h), x, rows, offs, E, nseg, ws, ss)


@pytest.mark.parametrize("rows,K,O", [(9, 8192, 64), (16, 2240, 192), (100, 64, 1024), (33, 1984, 512)])
def test_linear_few_rows_long_and_short_sums(rows, K, O):
    """K of one step, of fewer blocks than a block has waves, and of several batches per wave."""
    announce(f"linear few rows {rows} {K} {O}")
    g = _gen(rows + K)
    xq, xs = _codes(g, rows, K), torch.rand(rows, generator=g) + 0.1
    w, ws = _codes(g, 1, O, K), torch.rand((1, O), generator=g) + 0.1
    offs = torch.tensor([0, rows], dtype=torch.int32)
    y = moe.grouped_linear_i8(xq.to(DEV), xs.to(DEV), offs.to(DEV), 1, 0, 1, moe.pack_i8_codes(w).to(DEV), ws.to(DEV),
                              out_dtype=torch.float32)
    ref = Q.grouped_linear(xq.numpy(), xs.numpy(), np.arange(rows), offs.tolist(), 1, 1, w.numpy(), ws.numpy())
    assert np.all(np.abs(f64_of(y) - ref) <= 4 * 2.0 ** -24 * (1 + 1e-6) * np.abs(ref))


@pytest.mark.parametrize("d,I", [(64, 64), (4160, 192), (192, 2624), (1088, 1088)])
def test_ffn_few_rows_long_and_short_sums(d, I):
    announce(f"ffn few rows {d} {I}")
    g = _gen(d + I)
    rows, offs, E, nseg, S, x, ws, ss = _ffn_case(g, dict(sizes=[1, 0, 2, 0, 1], T=3), d, I)
    h = moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *_ffn_args(ws, ss), x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _ffn_check(f64_of(h), x, rows, offs, E, nseg, ws, ss)
