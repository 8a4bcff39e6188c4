"""The large-group kernels of the block-scaled FP8 products (tile_codes, tile_exact) where their lists, tails and rows end."""
import pytest
import torch

import fp8_plan
from helpers import announce, require_gpu
from test_gpu_norm_fp8 import DEV, F8, LARGE, _batch, _dt, _ffn_args, _ffn_case, _ffn_check, _gen, _linear_case, _linear_check

import top_expert_routing_amd as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _linear(case, dtype, x_rows="list", y=None, offs=None):
    rows, o, E, nseg, S, xq, xs, w, ws = case
    at = rows.long()
    if x_rows is None:
        xq, xs = xq.view(torch.uint8)[at].view(F8), xs[at]
    return moe.grouped_linear_fp8(xq.to(DEV), xs.to(DEV), (o if offs is None else offs).to(DEV), E, S, nseg,
                                  moe.pack_fp8_codes(w).to(DEV), ws.to(DEV), y=y, out_dtype=_dt(dtype),
                                  x_rows=rows.to(DEV) if x_rows == "list" else x_rows)


@pytest.mark.parametrize("K,O,dtype", [(320, 1344, "bf16"), (448, 1344, "f32"), (1152, 1280, "bf16")])
def test_rows_are_read_directly_and_through_a_list(K, O, dtype):
    announce(f"fp8 tiles rows {K} {O} {dtype}")
    case = _linear_case(_gen(K), LARGE["ragged"], K, O)
    assert fp8_plan.linear(len(case[0]), case[2], 0, 1, K, O, dtype == "f32").startswith("tile")
    y = _linear(case, dtype)
    _linear_check(y, case)
    assert torch.equal(y, _linear(case, dtype, None))
    # numbers outside [0, n_x) stand for the first and the last row
    rows = case[0].clone()
    T = case[5].shape[0]
    rows[rows == 0], rows[rows == T - 1] = -5, T + 1000
    assert torch.equal(y, _linear(case, dtype, rows.to(DEV)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_before_the_first_group_and_behind_the_last_stay(dtype):
    announce(f"fp8 tiles rows outside {dtype}")
    case = _linear_case(_gen(5), LARGE["many"], 512, 1024)
    n, offs = len(case[0]), case[1].clone()
    cut = 37
    offs[0] += cut
    offs[-1] -= cut
    y = torch.full((n, 1024), float("nan"), dtype=_dt(dtype), device=DEV)
    _linear(case, dtype, y=y, offs=offs)
    full = _linear(case, dtype)
    assert torch.equal(y[cut:n - cut], full[cut:n - cut])
    assert y[:cut].isnan().all() and y[n - cut:].isnan().all()


@pytest.mark.parametrize("E,nseg,S", [(400, 2, 0), (512, 1, 256)])
def test_most_groups_of_a_tile_list(E, nseg, S):
    announce(f"fp8 tiles most groups {E} {nseg} {S}")
    g = _gen(E + nseg)
    sizes = lambda a, b: torch.randint(a, b, (E,), generator=g).tolist()
    b = dict(sizes=sizes(40, 130), T=64, shared=S, **({"prio_sizes": sizes(0, 60)} if nseg == 2 else {}))
    case = rows, offs, E, nseg, S, xq, xs, ws, ss = _ffn_case(g, b, 384, 384)
    assert fp8_plan.ffn(len(rows), E, S, nseg, 384, 384) == ("tile_codes", "tile_codes")
    h = moe.grouped_ffn_fp8(xq.to(DEV), xs.to(DEV), offs.to(DEV), E, S, nseg, *_ffn_args(ws, ss), x_rows=rows.to(DEV))
    _ffn_check(h, case)


@pytest.mark.parametrize("K", [320, 384, 448, 512, 576, 640])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_number_of_stages(K, dtype):
    """Three blocks of K and more, the last one whole or half, with blocks that have no tile, one and several."""
    announce(f"fp8 tiles stages {K} {dtype}")
    case = _linear_case(_gen(K), dict(sizes=[129, 0, 64, 1, 1700, 127], T=300), K, 1088)
    assert fp8_plan.linear(len(case[0]), 6, 0, 1, K, 1088, dtype == "f32").startswith("tile")
    _linear_check(_linear(case, dtype), case)


def test_what_is_not_finite_stays_in_its_rows_and_columns():
    """NaN and infinite scales of a row reach that row of y alone, those of a matrix block its columns alone."""
    announce("fp8 tiles not finite")
    case = rows, offs, E, nseg, S, xq, xs, w, ws = _linear_case(_gen(7), dict(sizes=[700, 900], T=200), 448, 1280)
    for dtype in ("bf16", "f32"):
        want = _linear(case, dtype)
        xs2, ws2, xb, wb = xs.clone(), ws.clone(), xq.view(torch.uint8).clone(), w.view(torch.uint8).clone()
        xs2[3, 3], xs2[5, 0], xb[7, 447] = float("nan"), float("inf"), 0x7f
        ws2[0, 2, 3], wb[1, 1279, 0] = float("nan"), 0xff
        got = _linear((rows, offs, E, nseg, S, xb.view(F8), xs2, wb.view(F8), ws2), dtype)
        bad = torch.zeros(want.shape, dtype=torch.bool, device=DEV)
        at = rows.to(DEV)
        bad |= ((at == 3) | (at == 7))[:, None]
        bad[:700, 256:384] = True
        bad[700:, 1279] = True
        assert got[bad].isnan().all()
        inf = (at == 5)[:, None] & ~bad
        assert not got[inf].isfinite().any()
        assert torch.equal(got[~bad & ~inf], want[~bad & ~inf])


def test_two_calls_at_once_and_replayed():
    """Captured on one stream while another one runs the same products: the tiles keep nothing between calls."""
    announce("fp8 tiles two at once")
    g = _gen(9)
    rows, offs, E, nseg, S, xq, xs, ws, ss = _ffn_case(g, LARGE["priority"], 960, 1088)
    x, sc, od, rd, args = xq.to(DEV), xs.to(DEV), offs.to(DEV), rows.to(DEV), _ffn_args(ws, ss)
    call = lambda h=None, wk=None: moe.grouped_ffn_fp8(x, sc, od, E, S, nseg, *args, h, wk, x_rows=rd)
    want = call()
    hs = [torch.zeros_like(want) for _ in range(2)]
    wk = [torch.empty(moe.ffn_fp8_workspace_bytes(len(rows), 1088), dtype=torch.uint8, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(hs[0], wk[0])
        call(hs[0], wk[0])
    other = torch.cuda.Stream()
    for _ in range(3):
        for h in hs:
            h.zero_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            call(hs[1], wk[1])
        torch.cuda.synchronize()
        assert torch.equal(hs[0], want) and torch.equal(hs[1], want)
