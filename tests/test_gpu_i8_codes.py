"""Codes of the SwiGLU product inside moe_grouped_ffn_i8: each is the nearest one to its exact quotient, up to the
promised distance from a border."""
import numpy as np
import pytest
import torch

import i8_plan
from oracle import int8_oracle as Q
from helpers import announce, f64_of, require_gpu

import top_expert_routing_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# how far below zero the gate's values of a row lie, about; a rate of 0 leaves both signs
GATES = [0.0, 1.0, 10.0, 20.0, 40.0, 55.0]


@pytest.mark.parametrize("rows,kernel", [(16, "few"), (400, "stream"), (16640, "tile_half"), (70000, "tile_wide")])
def test_ffn_codes_lie_next_to_their_quotients(rows, kernel):
    """A down matrix of ones on the diagonal hands the codes out: h = block scale * code, rounded to bf16, at most 2^-8 of
    it off, and 127 * 2^-8 = 0.496 of a code still tells it (the scale's own error, below 3e-5, moves it by less than
    0.004).  The promise: a code is at most half a step from
    the exact quotient, or 2^-16 (22 + 2.2 (n + m)) more, n and m how far below zero the gate's value is, its own and
    the lowest of its block."""
    announce(f"ffn codes {rows} {kernel}")
    d = I = 256
    assert i8_plan.ffn(rows, 1, 0, 1, d, I)[0][0] == kernel
    g = torch.Generator().manual_seed(rows)
    x = torch.randn((rows, d), generator=g).abs().bfloat16()
    wg = torch.randint(0, 128, (1, I, d), generator=g, dtype=torch.int8)
    wu = (torch.randn((1, I, d), generator=g) * 40).round().clamp(-127, 127).to(torch.int8)
    wd = torch.eye(d, dtype=torch.int8)[None]
    one = torch.ones((1, d))
    su = torch.rand((1, I), generator=g) * 1e-3 + 1e-3
    xq, sx = Q.quantize(f64_of(x))
    sums = Q._dot(xq, wg[0].numpy()) * sx.astype(np.float64)[:, None]
    up = Q._dot(xq, wu[0].numpy()) * sx.astype(np.float64)[:, None] * su[0].numpy().astype(np.float64)
    worst = 0.0
    for below in GATES if rows < 50000 else GATES[:4:3]:
        w, s = wg, torch.full((1, I), -below / float(sums.mean()))
        dots = sums
        if below == 0.0:
            w, s = wu.flip(1), su
            dots = Q._dot(xq, w[0].numpy()) * sx.astype(np.float64)[:, None]
        gate = dots * s[0].numpy().astype(np.float64)
        assert gate.min() > -86.0                          # the factor of the gate is a normal number
        h = moe.grouped_ffn_i8(x.to(DEV), torch.tensor([0, rows], dtype=torch.int32, device=DEV), 1, 0, 1,
                               moe.pack_i8_codes(w.contiguous()).to(DEV), s.to(DEV), moe.pack_i8_codes(wu).to(DEV), su.to(DEV),
                               moe.pack_i8_codes(wd).to(DEV), one.to(DEV))
        a = (gate / (1.0 + np.exp(-gate)) * up).reshape(rows, 2, 128)
        scale = np.abs(a).max(2, keepdims=True) * np.float64(np.float32(1.0) / np.float32(127.0))
        quotient = a / scale
        code = np.rint(f64_of(h).reshape(rows, 2, 128) / scale)
        n = np.maximum(0.0, -gate).reshape(rows, 2, 128)
        margin = 2.0 ** -16 * (22 + 2.2 * (n + n.max(2, keepdims=True)))
        off = np.abs(code - quotient) - 0.5
        worst = max(worst, float(off.max()))
        print(f"gates near -{below}: {off.max():.2e} past half a step, promised {margin.max():.2e}", flush=True)
        assert np.abs(code).max() == 127 and (off <= margin).all()
