"""Routing with scores and the int8 calls at the ends of their documented ranges, against the float64 definitions."""
import numpy as np
import pytest
import torch

from oracle import int8_oracle as Q
import i8_plan
from helpers import announce, f64_of, np_of, require_gpu

import top_expert_routing_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ route
def _tiny_scores(g, k, score):
    """Rows whose k best logits give scores near and below the smallest normal double.  Softmax: one expert that the
    bias keeps out has all the mass."""
    tops = [-700.0, -706.0, -708.0, -709.0, -709.3, -709.7, -709.9, -720.0, -740.0, -744.0, -745.0, -745.25, -760.0, -250.0, -490.0]
    E = 32
    l = torch.full((2 * len(tops), E), -790.0)
    for i, top in enumerate(tops):
        l[2 * i, 1:1 + k] = top                                            # equal scores
        l[2 * i + 1, 1:1 + k] = top - 3 * torch.rand(k, generator=g)       # unequal ones
    if score == "softmax":
        l[:, 0] = 0.0
    bias = torch.zeros(E)
    bias[0] = -10.0
    bias[1:1 + k] = 1.0
    return l, bias


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 8])
@pytest.mark.parametrize("scale", [1.0, 2.5, 16.0, -3.0e38])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_tiny_scores(score, k, scale, renorm):
    """The weights of chosen experts whose scores sum to next to nothing are still their shares of the scale."""
    announce(f"route tiny scores {score} {k} {scale} {renorm}")
    l, bias = _tiny_scores(_gen(21), k, score)
    for dtype in (torch.float32, torch.bfloat16):
        lt = l.to(dtype)
        ids, w = moe.route(lt.to(DEV), k, score, bias.to(DEV), renormalize=renorm, scale=scale)
        ref_ids, ref_w = Q.route(f64_of(lt), k, score, f64_of(bias), renormalize=renorm, scale=scale)
        np.testing.assert_array_equal(np_of(ids), ref_ids)
        got = f64_of(w)
        assert np.isfinite(got).all()
        # the call's promise: 1e-6 of the value, or 2^-149
        assert np.all(np.abs(got - ref_w) <= np.maximum(1e-6 * np.abs(ref_w), 2.0 ** -149))
        if renorm:
            assert (np.abs(ref_w).sum(1) > 0).sum() > len(lt) // 2


def test_route_tiny_scores_order_groups():
    """Sums of sigmoids below e^-709.8 still tell the groups apart."""
    l = torch.full((2, 16), -800.0)
    l[0, 0:2], l[0, 12:14] = -740.0, -712.0
    l[1, 4:6], l[1, 8:10] = -712.0, -710.0
    ids, w = moe.route(l.to(DEV), 2, "sigmoid", n_groups=4, top_groups=1, group_rank="top2")
    assert ids.tolist() == [[12, 13], [8, 9]] and w.tolist() == [[0.5, 0.5]] * 2


# ------------------------------------------------------------------ quantize
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [2 ** 31 - 8, 2 ** 31 - 2048, 2 ** 30 + 8])
def test_quantize_longest_rows(d, dtype):
    """One row of nearly 2^31 values: the loop's last step passes int32 for some of the lanes."""
    announce(f"quantize longest row {d} {dtype}")
    x = torch.zeros((1, d), dtype=dtype, device=DEV)
    where = torch.cat([torch.arange(0, d, 16777259), torch.arange(d - 4096, d)]).to(DEV)
    x[0, where] = (torch.arange(len(where), device=DEV) % 255 - 127).to(dtype)        # scale 1: codes are the values
    q, s = moe.quantize_rows_i8(x)
    assert s.tolist() == [1.0]
    assert torch.equal(q, x.to(torch.int8))


# ------------------------------------------------------------------ the widest matrices
def test_linear_more_blocks_than_one_row_of_a_launch():
    """33 experts of one row each and 32.5 million output channels: 2^23 + 256 blocks of 512 threads."""
    E, K, O = 33, 64, 32537728
    announce(f"linear {E} x {K} -> {O}")
    kernel, _, blocks, x, y = i8_plan.launches([("linear", E, E, 0, 1, K, O)])[0]
    assert kernel == "stream" and blocks * 512 >= 2 ** 32 and y > 1
    if torch.cuda.mem_get_info()[0] < 100 * 2 ** 30:
        pytest.skip("needs 69 GB of weights")
    g = _gen(22)
    xq = torch.randint(-127, 128, (E, K), generator=g, dtype=torch.int8).to(DEV)
    xs = (torch.rand(E, generator=g) + 0.5).to(DEV)
    w = torch.ones((E, O, K), dtype=torch.int8, device=DEV)          # the same in any order of codes
    ws = torch.rand((E, O), device=DEV) + 0.5
    y = torch.zeros((E, O), dtype=torch.bfloat16, device=DEV)
    offs = torch.arange(E + 1, dtype=torch.int32, device=DEV)
    moe.grouped_linear_i8(xq, xs, offs, E, 0, 1, w, ws, y)
    sums = xq.double().sum(1)
    tol = (3 * 2.0 ** -24 + torch.finfo(torch.bfloat16).eps / 2) * (1 + 1e-6)
    for e in range(E):
        ref = sums[e] * xs[e].double() * ws[e].double()
        assert bool(((y[e].double() - ref).abs() <= tol * ref.abs()).all()), e
    del w, ws, y
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ the layer
def test_layer_refuses_tokens_its_raw_calls_would_read_wrongly():
    """bound_calls hands out addresses: fp32 tokens, too few of them, or of another width would be read out of range."""
    z = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt, device=DEV)
    f, b = torch.float32, torch.bfloat16
    E, k, d, I, T = 4, 2, 64, 128, 5
    q = (z(E, I, d), z(E, I, dt=f), z(E, I, d), z(E, I, dt=f), z(E, d, I), z(E, d, dt=f))
    for fused in (True, False):
        layer = moe.MoeLayer(E, k, d, I, T, b, None, None, None, device=DEV, int8_weights=q, fused_gather=fused)
        l = z(T, E, dt=f)
        layer.bound_calls(l, z(T, d, dt=b))
        for x in (z(T, d, dt=f), z(T - 1, d, dt=b), z(T, d - 8, dt=b), z(T, 2 * d, dt=b)[:, ::2], z(T, d, dt=b).cpu()):
            with pytest.raises((TypeError, ValueError)):
                layer.bound_calls(l, x)


# ------------------------------------------------------------------ empty calls and the largest ones
def _i8(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)


def test_empty_calls():
    """No tokens, no sorted rows, or no rows in any group: nothing is read or written, with and without a row list."""
    e = moe.route(torch.empty((0, 16), device=DEV), 2, "sigmoid", n_groups=4, top_groups=2)
    assert e[0].shape == (0, 2) and e[1].shape == (0, 2)
    g = _gen(23)
    E, d, I = 3, 256, 256
    w = [moe.pack_i8_codes(_i8(g, E, *s)).to(DEV) for s in ((I, d), (I, d), (d, I))]
    s = [torch.ones((E, n), device=DEV) for n in (I, I, d)]
    args = [t for pair in zip(w, s) for t in pair]
    none = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    x, empty = torch.ones((7, d), dtype=torch.bfloat16, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
    xq, xs = moe.quantize_rows_i8(x)
    assert moe.grouped_linear_i8(xq, xs, none, E, 0, 1, w[0], s[0], x_rows=empty).shape == (0, I)
    assert moe.grouped_linear_i8(xq[:0], xs[:0], none, E, 0, 1, w[0], s[0]).shape == (0, I)
    assert moe.grouped_ffn_i8(x, none, E, 0, 1, *args, x_rows=empty).shape == (0, d)
    assert moe.grouped_ffn_i8(x[:0], none, E, 0, 1, *args).shape == (0, d)
    for rows, kernel in ((5, "few"), (400, "stream"), (40000, "tile_wide")):
        assert i8_plan.ffn(rows, E, 0, 1, d, I)[0][0] == kernel
        list_ = torch.zeros(rows, dtype=torch.int32, device=DEV)
        for at in (0, rows):
            offs = torch.full((E + 1,), at, dtype=torch.int32, device=DEV)
            h = torch.full((rows, d), 3.0, dtype=torch.bfloat16, device=DEV)
            moe.grouped_ffn_i8(x, offs, E, 0, 1, *args, h, x_rows=list_)
            y = torch.full((rows, I), 3.0, device=DEV)
            moe.grouped_linear_i8(xq, xs, offs, E, 0, 1, w[0], s[0], y, x_rows=list_)
            assert bool((h == 3).all()) and bool((y == 3).all())


def _linear_rows(xq, xs, w, ws, rows):
    """y of some rows of a plain linear map, from exact integer sums (64-bit)."""
    return (xq[rows].double().cpu() @ w[0].double().T) * xs[rows].double().cpu()[:, None] * ws[0].double()


@pytest.mark.parametrize("rows,K,kernel", [(2 ** 24, 64, "stream"), (2 ** 23 - 64, 192, "stream"), (2 ** 23 - 64, 256, "tile_wide")])
def test_linear_largest_row_counts(rows, K, kernel):
    """As many sorted rows as a call takes; codes whose offsets come next to 2^31."""
    announce(f"linear {rows} rows x {K}")
    O = 64
    assert rows * K < 2 ** 31 and i8_plan.linear(rows, 1, 0, 1, K, O)[0] == kernel
    g = _gen(24)
    some = _i8(g, 65537, K).to(DEV)
    xq = some.repeat(rows // 65537 + 1, 1)[:rows].contiguous()
    xs = (torch.arange(rows, device=DEV) % 251 + 1).float()
    w, ws = _i8(g, 1, O, K), torch.rand((1, O), generator=g) + 0.5
    offs = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    y = moe.grouped_linear_i8(xq, xs, offs, 1, 0, 1, moe.pack_i8_codes(w).to(DEV), ws.to(DEV))
    pick = torch.cat([torch.arange(300), torch.arange(rows - 700, rows), torch.randint(0, rows, (4000,), generator=g)])
    ref = _linear_rows(xq, xs, w, ws, pick.to(DEV))
    tol = (3 * 2.0 ** -24 + torch.finfo(torch.bfloat16).eps / 2) * (1 + 1e-6)
    assert bool(((y[pick.to(DEV)].double().cpu() - ref).abs() <= tol * ref.abs()).all())
    # every other row: the same codes, so the same sums; scales are whole numbers
    unit = moe.grouped_linear_i8(xq, torch.ones_like(xs), offs, 1, 0, 1, moe.pack_i8_codes(w).to(DEV), ws.to(DEV), out_dtype=torch.float32)
    whole = rows // 65537 * 65537
    assert torch.equal(unit[:whole].view(-1, 65537, O), unit[:65537].expand(rows // 65537, -1, -1))


@pytest.mark.parametrize("rows,kernel", [(60, "few"), (3000, "stream"), (140000, "tile_wide")])
def test_linear_row_lists_into_the_longest_codes(rows, kernel):
    """Tokens whose codes end next to 2^31, read through a row list."""
    n_x, K, O = 2 ** 23 - 1, 256, 128
    announce(f"linear {rows} of {n_x} tokens")
    assert i8_plan.linear(rows, 1, 0, 1, K, O)[0] == kernel
    g = _gen(25)
    xq = _i8(g, 4097, K).to(DEV).repeat(n_x // 4097 + 1, 1)[:n_x].contiguous()
    xs = (torch.arange(n_x, device=DEV) % 13 + 1).float()
    w, ws = _i8(g, 1, O, K), torch.rand((1, O), generator=g) + 0.5
    list_ = torch.cat([n_x - 1 - torch.arange(rows // 2), torch.randint(0, n_x, (rows - rows // 2,), generator=g)])
    y = moe.grouped_linear_i8(xq, xs, torch.tensor([0, rows], dtype=torch.int32, device=DEV), 1, 0, 1, moe.pack_i8_codes(w).to(DEV),
                              ws.to(DEV), x_rows=list_.to(DEV, torch.int32), out_dtype=torch.float32)
    ref = _linear_rows(xq, xs, w, ws, list_.to(DEV))
    assert bool(((y.double().cpu() - ref).abs() <= 3 * 2.0 ** -24 * (1 + 1e-6) * ref.abs()).all())


def test_ffn_largest_row_count():
    """2^23 - 64 sorted rows of 700 tokens: each is what the same token gives in a batch of 70000."""
    rows, d, I = 2 ** 23 - 64, 256, 256
    announce(f"ffn {rows} rows")
    g = _gen(26)
    x = torch.randn((700, d), generator=g).bfloat16().to(DEV)
    args = [t for s in ((I, d), (I, d), (d, I)) for t in (moe.pack_i8_codes(_i8(g, 1, *s)).to(DEV), torch.full((1, s[0]), 2e-3, device=DEV))]
    assert {p[0] for n in (rows, 70000) for p in i8_plan.ffn(n, 1, 0, 1, d, I)} == {"tile_wide"}
    run = lambda n: moe.grouped_ffn_i8(x, torch.tensor([0, n], dtype=torch.int32, device=DEV), 1, 0, 1, *args,
                                       x_rows=torch.arange(n, dtype=torch.int32, device=DEV) % 700)
    small = run(70000)[:700]
    assert bool((small != 0).any(1).all())
    h = run(rows)
    whole = rows // 700 * 700
    assert torch.equal(h[:whole].view(-1, 700, d), small.expand(rows // 700, -1, -1)) and torch.equal(h[whole:], small[:rows - whole])


# ------------------------------------------------------------------ graphs, streams
@pytest.mark.parametrize("rows,kernels", [(40, ["few", "few"]), (1500, ["stream", "stream"]), (20000, ["tile_half", "stream"]),
                                          (90000, ["tile_wide", "tile_wide"])])
def test_ffn_graphs_and_two_streams_on_each_kernel(rows, kernels):
    """Captured and replayed with new tokens, between eager work, and twice at once with workspaces of their own."""
    announce(f"ffn graph {rows} {kernels}")
    E, d, I, T = 2, 256, 256, 500
    assert [p[0] for p in i8_plan.ffn(rows, E, 0, 1, d, I)] == kernels
    g = _gen(27)
    args = [t for s in ((I, d), (I, d), (d, I)) for t in (moe.pack_i8_codes(_i8(g, E, *s)).to(DEV), torch.full((E, s[0]), 2e-3, device=DEV))]
    offs = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device=DEV)
    list_ = torch.randint(0, T, (rows,), generator=g, dtype=torch.int32).to(DEV)
    x = torch.randn((T, d), generator=g).bfloat16().to(DEV)
    h = torch.zeros((rows, d), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(moe.ffn_i8_workspace_bytes(rows, T, d, I, E), dtype=torch.uint8, device=DEV)
    eager = lambda: moe.grouped_ffn_i8(x, offs, E, 0, 1, *args, x_rows=list_)
    step = lambda: moe.grouped_ffn_i8(x, offs, E, 0, 1, *args, h, ws, x_rows=list_)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        x.copy_(torch.randn((T, d), generator=g).bfloat16())
        h.zero_()
        ws.random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, eager())
    outs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s in streams * 2:
        with torch.cuda.stream(s):
            outs.append(eager())
    torch.cuda.synchronize()
    assert all(torch.equal(o, h) for o in outs)
