"""The SwiGLU product's codes inside the block-scaled FP8 FFN, read out through a down matrix of ones on the diagonal.

h is then code * scale rounded to bf16, 2^-8 of it at most, and neighbouring codes are 2^-4 of their size or more apart, so
h over the block's scale in 64 bits names the code.

Bound: a gate or up sum takes at most 128 roundings inside its blocks and one for each block, each up to 2^-23 of a partial sum
and independent of the others, so its error is sqrt(128 + blocks) * 2^-23 of its row's typical size in the root mean square;
silu, the products and the quotient add (12 + 5 |gate|) * 2^-24 of a value.  Moving a quotient by a share of a step passes a
border with that probability at most, so the shares' sum, and four of its standard deviations, bound the number of codes
that are neighbours of those of 64 bits; and errors a hundred times under a step move no code by two.  Products cut to a
multiple of 2^(E - 13), as the FP8 matrix instructions cut them, are off by 1.5e-5 to 5e-5 of a sum, ten times this.
"""
import numpy as np
import pytest
import torch

import fp8_plan
from oracle import fp8_oracle as Q
from helpers import announce, f64_of, require_gpu
from test_gpu_norm_fp8 import DEV, F8, _batch, _codes, _ffn_args, _gen, _nb, _scales

import top_expert_routing_amd as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("kernel,d,b", [
    ("few", 1024, dict(sizes=[9, 0, 4, 3], T=20)),
    ("stream", 1024, dict(sizes=[33, 64, 0, 17, 60, 48], T=60)),
    ("tile_codes", 1024, dict(sizes=[300, 1, 257, 700, 0, 64, 65, 800], T=900)),
    ("tile_codes", 2112, dict(sizes=[129, 640, 0, 500], T=700)),
    ("tile_codes", 1984, dict(sizes=[300, 0, 200], T=300, prio_sizes=[20, 64, 130], shared=1)),
    # the shortest K of the tiles, its last block a half, and one stage more than the ring holds
    ("tile_codes", 320, dict(sizes=[5600, 129, 0, 63, 1, 65], T=800)),
    ("tile_codes", 448, dict(sizes=[1, 64, 4200, 127, 0], T=700)),
])
def test_codes_are_those_of_fp32_sums(kernel, d, b):
    announce(f"ffn fp8 codes {kernel} {d}")
    g = _gen(d + len(b["sizes"]))
    rows, offs, E, nseg = _batch(g, **b)
    S, T = b.get("shared", 0), b["T"]
    x = torch.randn((T, d), generator=g)
    xq, xs = Q.quantize_blocks(x.numpy())
    wg, wu = _codes(g, E + S, d, d), _codes(g, E + S, d, d)
    sg, su = (_scales(g, E + S, _nb(d), _nb(d)) * 0.04 for _ in range(2))
    one = torch.eye(d).to(F8).expand(E + S, d, d).contiguous()
    assert set(fp8_plan.ffn(len(rows), E, S, nseg, d, d)) == {kernel}
    h = moe.grouped_ffn_fp8(torch.from_numpy(xq).float().to(F8).to(DEV), torch.from_numpy(xs).to(DEV), offs.to(DEV), E, S, nseg,
                            *_ffn_args((wg, wu, one), (sg, su, torch.ones((E + S, _nb(d), _nb(d))))), x_rows=rows.to(DEV))
    torch.cuda.synchronize()
    got = f64_of(h)
    wide = Q.wide_rows(xq, xs)
    turned, far, shares = 0, 0, 0.0
    first = offs.tolist()
    for k in range(len(first) - 1):
        at = rows[first[k]:first[k + 1]].numpy()
        if not len(at):
            continue
        e = Q.group_expert(k, E, nseg)
        gate = wide[at] @ Q.wide_matrix(f64_of(wg[e]), sg[e].numpy()).T
        up = wide[at] @ Q.wide_matrix(f64_of(wu[e]), su[e].numpy()).T
        sig = 1 / (1 + np.exp(-gate))
        a = gate * sig * up
        q, s = Q.quantize_blocks(a.astype(np.float32))
        s = np.repeat(s.astype(np.float64), 128, axis=1)[:, :d]
        size = lambda v: np.sqrt((v * v).mean(axis=1, keepdims=True))
        off = (128 + _nb(d)) ** 0.5 * 2.0 ** -23 * (np.abs(up * sig * (1 + gate * (1 - sig))) * size(gate) + np.abs(gate * sig) * size(up))
        off += (12 + 5 * np.abs(gate)) * 2.0 ** -24 * np.abs(a)
        shares += float((off / s / Q.e4m3_step(a / s)).sum())
        code = Q.e4m3(np.clip(got[first[k]:first[k + 1]] / s, -448, 448))
        turned += int((code != q).sum())
        far += int((np.abs(code - q) > np.maximum(Q.e4m3_step(code), Q.e4m3_step(q))).sum())
    print(f"codes that are neighbours: {turned}, at most {shares:.1f} expected; further off: {far}; of {got.size}", flush=True)
    assert turned <= shares + 4 * shares ** 0.5 + 3 and far == 0
