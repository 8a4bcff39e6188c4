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
