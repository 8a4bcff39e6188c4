"""The LDS-tiled int8 kernels against their float64 definitions, at sizes whose kernels are asserted: both tile heights,
priority segments on either side of the rules, and as many groups as a call can have.  Tolerances as in
test_gpu_route_int8.py."""
import numpy as np
import pytest
import torch

import i8_plan
from oracle import int8_oracle as Q
from helpers import announce, f64_of, require_gpu
from test_gpu_route_int8 import _batch, _codes, _ffn_args, _ffn_case, _ffn_check, _gen

import top_expert_routing_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _linear_check(g, b, K, O, dt, kernel):
    rows, offs, E, nseg = _batch(g, **b)
    S = b.get("shared", 0)
    assert i8_plan.linear(len(rows), E, S, nseg, K, O)[0] == kernel
    xq, xs = _codes(g, b["T"], K), torch.rand(b["T"], generator=g) + 0.1
    w, ws = _codes(g, E + S, O, K), torch.rand((E + S, O), generator=g) + 0.1
    args = [t.to(DEV) for t in (xq, xs, offs)] + [E, S, nseg, moe.pack_i8_codes(w).to(DEV), ws.to(DEV)]
    y = moe.grouped_linear_i8(*args, x_rows=rows.to(DEV), out_dtype=dt)
    torch.cuda.synchronize()
    ref = Q.grouped_linear(xq.numpy(), xs.numpy(), rows.numpy(), offs.tolist(), E, nseg, w.numpy(), ws.numpy())
    tol = (3 * 2.0 ** -24 + torch.finfo(dt).eps / 2) * (1 + 1e-6)
    assert np.all(np.abs(f64_of(y) - ref) <= tol * np.abs(ref))
    assert torch.equal(y, moe.grouped_linear_i8(*args, x_rows=rows.to(DEV), out_dtype=dt))


def _sizes(g, E, lo, hi):
    return torch.randint(lo, hi, (E,), generator=g).tolist()


def _most_half_groups():
    """The largest number of groups whose lists fit the 128-row tiles."""
    fits = lambda E: i8_plan.linear(80 * E, E, 0, 1, 256, 192)[0] == "tile_half"
    return next(E for E in range(500, 300, -1) if fits(E))


@pytest.mark.parametrize("more,kernel", [(0, "tile_half"), (1, "tile_wide")])
def test_linear_groups_around_the_tiles_lists(more, kernel):
    E = _most_half_groups() + more
    announce(f"linear {E} groups on {kernel}")
    g = _gen(40 + more)
    _linear_check(g, dict(sizes=_sizes(g, E, 60, 101), T=300), 256, 192, torch.float32, kernel)


def test_linear_most_groups():
    """512 experts in two segments and 256 shared ones: 1280 groups."""
    announce("linear 1280 groups")
    g = _gen(42)
    b = dict(sizes=_sizes(g, 512, 40, 101), prio_sizes=_sizes(g, 512, 0, 30), T=80, shared=256)
    _linear_check(g, b, 256, 128, torch.bfloat16, "tile_wide")


@pytest.mark.parametrize("more,kernel", [(0, "tile_half"), (1, "tile_wide")])
def test_ffn_groups_around_the_tiles_lists(more, kernel):
    E = _most_half_groups() + more
    announce(f"ffn {E} groups on {kernel}")
    g = _gen(44 + more)
    rows, offs, E, nseg, S, x, ws, ss = _ffn_case(g, dict(sizes=_sizes(g, E, 60, 101), T=90), 256, 256)
    assert [p[0] for p in i8_plan.ffn(len(rows), E, S, nseg, 256, 256)] == [kernel, "tile_wide"]
    h = moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *_ffn_args(ws, ss), x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _ffn_check(f64_of(h), x, rows, offs, E, nseg, ws, ss)


@pytest.mark.parametrize("per_expert,kernel", [(64, "stream"), (65, "tile_half")])
def test_linear_priority_batch_around_the_tiles(per_expert, kernel):
    """The rows of an expert over both segments decide."""
    announce(f"linear priority {per_expert} rows an expert on {kernel}")
    g = _gen(per_expert)
    prio = _sizes(g, 40, 0, 41)
    _linear_check(g, dict(sizes=[per_expert - p for p in prio], prio_sizes=prio, T=200), 320, 1856, torch.float32, kernel)


# batches of several tiles a block, partial and empty ones: (gate/up kernel, batch)
LARGE = {
    "ragged": ("tile_half", dict(sizes=[1, 0, 255, 256, 257, 129, 700, 40, 2000, 16, 1500, 33], T=900)),
    "many": ("tile_half", dict(sizes=[100 + 7 * (i % 13) for i in range(44)], T=700)),
    "hot": ("tile_wide", dict(sizes=[0, 13100, 0, 300], T=2048)),
    "priority": ("tile_half", dict(sizes=[600, 0, 1, 900, 1300], T=800, prio_sizes=[64, 3, 0, 130, 1000], shared=1)),
    "priority_hot": ("tile_wide", dict(sizes=[0, 6000, 40, 2200], T=600, prio_sizes=[130, 700, 0, 257])),
}


@pytest.mark.parametrize("name", LARGE)
@pytest.mark.parametrize("d,I", [(1280, 960), (1472, 1088)])
def test_ffn_large_on_tiles(name, d, I):
    announce(f"ffn large on tiles {name} {d} {I}")
    kernel, b = LARGE[name]
    g = _gen(d + I + len(name))
    rows, offs, E, nseg, S, x, ws, ss = _ffn_case(g, b, d, I)
    assert [p[0] for p in i8_plan.ffn(len(rows), E, S, nseg, d, I)] == [kernel, "tile_wide"]
    args = _ffn_args(ws, ss)
    h = moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *args, x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    _ffn_check(f64_of(h), x, rows, offs, E, nseg, ws, ss)
    assert torch.equal(h, moe.grouped_ffn_i8(x.to(DEV), offs.to(DEV), E, S, nseg, *args, x_rows=rows.to(DEV)))
