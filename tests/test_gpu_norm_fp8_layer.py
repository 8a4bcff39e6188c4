"""MoeLayer with a norm in front and with block-scaled FP8 experts: eagerly, through its raw calls and captured, against
the calls that it is made of, and against the plain formulas."""
import pytest
import torch

import workloads
from oracle import fp8_oracle as Q
from helpers import announce, f64_of, require_gpu

import top_expert_routing_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _case(T, prio, S, d=320, I=192, seed=3):
    wl = workloads.custom(T=T, E=16, k=4, d=d, I=I, dtype="bf16", S=S, n_priority=prio, seed=seed, device=DEV)
    g = torch.Generator().manual_seed(seed)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV)
    wr = (torch.randn((16, d), generator=g) * 0.1).bfloat16().to(DEV)
    res = torch.randn((T, d), generator=g).to(DEV)
    return wl, w, wr, res


def _blocks(*ws):
    return tuple(t for w in ws for c, s in [moe.quantize_fp8_blocks(w)] for t in (moe.pack_fp8_codes(c), s))


def _layer(wl, prio, S, **kw):
    s = wl.spec
    return moe.MoeLayer(s.E, s.k, s.d, s.I, s.T, torch.bfloat16, kw.pop("w_gate", None), kw.pop("w_up", None),
                        kw.pop("w_down", None), n_shared=S, n_priority=prio, device=DEV, **kw)


@pytest.mark.parametrize("T,prio,S,router,res_type", [(48, 0, 1, True, "f32"), (300, 16, 0, False, "bf16"), (1, 0, 0, True, None),
                                                      (2500, 64, 0, True, "bf16")])
def test_layer_with_norm_and_fp8_experts(T, prio, S, router, res_type):
    announce(f"layer norm fp8 {T} {prio} {S} {router} {res_type}")
    wl, w, wr, res = _case(T, prio, S)
    q = _blocks(wl.w_gate, wl.w_up, wl.w_down)
    layer = _layer(wl, prio, S, fp8_block_weights=q, norm=(w, EPS), w_router=wr if router else None)
    res0 = None if res_type is None else res.bfloat16() if res_type == "bf16" else res
    r = None if res0 is None else res0.clone()
    y = layer.forward(wl.logits, wl.x, residual=r).clone()

    r2 = None if res0 is None else res0.clone()
    xn, xq, xs = moe.rmsnorm(wl.x, w, EPS, residual=r2, codes="fp8")
    if r is not None:
        assert torch.equal(r, r2)
    logits = moe.router(xn, wr) if router else wl.logits
    ids, tw = moe.gate(logits, 4)
    assert torch.equal(layer.topk_ids, ids) and torch.equal(layer.topk_w, tw)
    p = moe.permute(ids, 16, S, prio)
    nseg = 2 if prio else 1
    h = moe.grouped_ffn_fp8(xq, xs, p["group_offsets"], 16, S, nseg, *q, x_rows=p["sorted_token"])
    assert torch.equal(layer.h_sorted, h)
    assert torch.equal(y, moe.combine(h, p["flat_to_sorted"], tw, S))

    # the plain formulas: norm in 64 bits, experts on the same codes
    v = f64_of(wl.x)
    if res0 is not None:
        v = Q.residual_sum(v, f64_of(res0), res_type == "bf16")
    rows = p["sorted_token"].cpu()
    first = p["group_offsets"].cpu().tolist()
    rstd, prod = Q.rmsnorm(v, f64_of(w), EPS)
    ref = torch.from_numpy(prod.astype("float64") * rstd[:, None])[rows.long()]
    want = torch.zeros_like(ref)
    for e in range(len(first) - 1):
        a, b = first[e], first[e + 1]
        m = e % 16 if e < nseg * 16 else 16 + e - nseg * 16
        if a < b:
            gate, up, down = (t[m].double().cpu() for t in (wl.w_gate, wl.w_up, wl.w_down))
            gt = ref[a:b] @ gate.T
            want[a:b] = (gt * torch.sigmoid(gt) * (ref[a:b] @ up.T)) @ down.T
    # a rounding to E4M3 is off by at most 2^-4 / sqrt(3) of a value in the root mean square; there are six in the path of
    # an output (rows and matrices of gate and of up, the SwiGLU product, the down matrix)
    assert (h.double().cpu() - want).norm() <= 6 * 2.0 ** -4 / 3 ** 0.5 * want.norm()

    # the raw calls, and captured
    if r is not None:
        r.copy_(res0)
    calls = layer.bound_calls(wl.logits, wl.x, residual=r)
    assert calls[0][0] == "moe_rmsnorm"
    layer.y.zero_()
    for name, fn, a in calls:
        assert fn(*a) == 0, name
    torch.cuda.synchronize()
    assert torch.equal(layer.y, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(wl.logits, wl.x, residual=r)
    for _ in range(3):
        layer.y.zero_()
        if r is not None:
            r.copy_(res0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.y, y)
        if r is not None:
            assert torch.equal(r, r2)


@pytest.mark.parametrize("T,prio", [(7, 0), (130, 8)])
def test_layer_with_fp8_experts_alone(T, prio):
    """Without a norm the layer quantises its input itself."""
    announce(f"layer fp8 {T} {prio}")
    wl, _, wr, _ = _case(T, prio, 0)
    q = _blocks(wl.w_gate, wl.w_up, wl.w_down)
    layer = _layer(wl, prio, 0, fp8_block_weights=q, w_router=wr)
    y = layer.forward(wl.logits, wl.x).clone()
    xq, xs = moe.quantize_blocks_fp8(wl.x)
    p = moe.permute(layer.topk_ids, 16, 0, prio)
    h = moe.grouped_ffn_fp8(xq, xs, p["group_offsets"], 16, 0, 2 if prio else 1, *q, x_rows=p["sorted_token"])
    assert torch.equal(layer.h_sorted, h)
    calls = layer.bound_calls(wl.logits, wl.x)
    assert [c[0] for c in calls] == ["moe_router", "moe_gate", "moe_permute", "moe_quantize_blocks_fp8", "moe_grouped_ffn_fp8",
                                     "moe_combine"]
    layer.y.zero_()
    for name, fn, a in calls:
        assert fn(*a) == 0, name
    torch.cuda.synchronize()
    assert torch.equal(layer.y, y)


@pytest.mark.parametrize("kind,fused", [("bf16", True), ("bf16", False), ("packed", True), ("int8", False), ("combine", True)])
def test_norm_in_front_of_the_other_experts(kind, fused):
    """A layer with a norm gives what the norm and then the layer without one give, with fp32 rows going in too."""
    announce(f"layer norm {kind} {fused}")
    wl, w, wr, res = _case(40, 0, 1, d=256)
    ws = (wl.w_gate, wl.w_up, wl.w_down)
    kw = dict(fused_gather=fused, w_router=wr)
    if kind in ("packed", "combine"):
        ws = tuple(moe.pack_weights(t) for t in ws)
        kw.update(packed_weights=True, fused_combine=kind == "combine")
    if kind == "int8":
        kw["int8_weights"] = tuple(t for x in ws for c, s in [moe.quantize_rows_i8(x)] for t in (moe.pack_i8_codes(c), s))
    kw.update(w_gate=ws[0], w_up=ws[1], w_down=ws[2])

    def same(a, b, h):
        """The fused combine adds its 5 terms (4 experts, a shared one) to a token in fp32 in no fixed order (libmoe.h), weights
        at most 1: two orders differ by 2 * 4 * 2^-24 of the terms' magnitudes, at most 5 max|h|, and then each
        is rounded to bf16, off by 2^-8 of itself.  Everything else is the same bits."""
        if kind != "combine":
            return torch.equal(a, b)
        a, b = a.double(), b.double()
        return bool(((a - b).abs() <= 8 * 2.0 ** -24 * 5 * h + 2.0 ** -8 * (a.abs() + b.abs())).all())
    for x in (wl.x, wl.x.float() * 1.01):
        xn, _, _ = moe.rmsnorm(x, w, EPS, residual=res.clone(), y=torch.empty_like(wl.x))
        want = _layer(wl, 0, 1, **dict(kw)).forward(wl.logits, xn).clone()
        layer = _layer(wl, 0, 1, norm=(w, EPS), **dict(kw))
        h = 0.0
        got = layer.forward(wl.logits, x, residual=res.clone()).clone()
        if kind == "combine":
            h = moe.grouped_ffn_packed(xn, layer.perm["group_offsets"], 16, 1, 1, *ws, x_rows=layer.perm["sorted_token"])
            h = h.double().abs().max()
        assert same(got, want, h)
        layer.y.zero_()
        r = res.clone()
        for name, fn, a in layer.bound_calls(wl.logits, x, residual=r):
            assert fn(*a) == 0, name
        torch.cuda.synchronize()
        assert same(layer.y, want, h)


def test_layer_refusals():
    wl, w, wr, res = _case(5, 0, 0)
    q = _blocks(wl.w_gate, wl.w_up, wl.w_down)
    make = lambda **kw: _layer(wl, 0, 0, **{"fp8_block_weights": q, **kw})
    for i, v in ((0, q[4]), (1, q[1][:, :1]), (3, q[3].double()), (4, q[4][:8]), (5, q[5].cpu())):
        with pytest.raises((TypeError, ValueError)):
            make(fp8_block_weights=tuple(v if j == i else t for j, t in enumerate(q)))
    for kw in (dict(fp8_block_weights=q[:4]), dict(fp8_weights=q), dict(int8_weights=q), dict(fused_combine=True),
               dict(fused_gather=False), dict(norm=(w[:64], EPS)), dict(norm=(w.half(), EPS)), dict(norm=(w, 0.0)),
               dict(norm=(w, float("nan"))), dict(norm=(w.cpu(), EPS))):
        with pytest.raises((TypeError, ValueError)):
            make(**kw)
    plain = make()
    for call in (plain.forward, plain.bound_calls):
        with pytest.raises(ValueError):
            call(wl.logits, wl.x, residual=res)
        with pytest.raises((TypeError, ValueError)):
            call(wl.logits, wl.x.float())
        with pytest.raises((TypeError, ValueError)):
            call(wl.logits, wl.x[:4])
    layer = make(norm=(w, EPS))
    for call in (layer.forward, layer.bound_calls):
        for x, r in ((wl.x[:4], res), (wl.x, res[:4]), (wl.x, res.half()), (wl.x.half(), res), (wl.x, res.cpu()),
                     (wl.x[:, :64], res), (wl.x.T.contiguous().T, res)):
            with pytest.raises((TypeError, ValueError)):
                call(wl.logits, x, residual=r)
    layer.norm = (w[:64], EPS)
    with pytest.raises(ValueError):
        layer.bound_calls(wl.logits, wl.x)
    layer.norm = (w, EPS)
    layer.fp8_block_weights = q[:5] + (q[5][:, :1],)
    with pytest.raises(ValueError):
        layer.bound_calls(wl.logits, wl.x)


def test_router_weights_are_of_the_rows_that_it_reads():
    """The norm's rows are bf16, so an fp32 router matrix does not go with them, nor one of another width."""
    wl, w, wr, _ = _case(5, 0, 0)
    q = _blocks(wl.w_gate, wl.w_up, wl.w_down)
    for bad in (wr.float(), wr[:, :64].contiguous(), wr[:8]):
        layer = _layer(wl, 0, 0, fp8_block_weights=q, norm=(w, EPS), w_router=bad)
        for call in (layer.forward, layer.bound_calls):
            with pytest.raises((TypeError, ValueError)):
                call(wl.logits, wl.x)
