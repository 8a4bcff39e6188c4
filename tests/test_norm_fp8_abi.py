"""The norm and the block-scaled FP8 calls: exports, refusals on the host, workspace sizes (CPU only; no kernel is
launched)."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import top_expert_routing_amd as m
from top_expert_routing_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, WS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
BF16, F32 = _lib.MOE_BF16, _lib.MOE_F32
FAKE = 1 << 20          # a non-NULL, 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    return m.load()


@pytest.mark.parametrize("header,names", [("libmoe_norm.h", _lib.NORM_EXPORTS), ("libmoe_fp8.h", _lib.FP8_EXPORTS)])
def test_headers_declare_what_is_exported(lib, header, names):
    text = open(os.path.join(ROOT, "include", header)).read()
    declared = re.findall(r"^moe_status\s+(moe_\w+)\s*\(", text, re.M)
    assert sorted(declared) == sorted(names)
    for n in names:
        assert hasattr(lib, n)


def test_norm_validation(lib):
    names = ["x", "xt", "res", "rt", "w", "wt", "T", "d", "eps", "out", "y", "yt", "code", "q", "s", "stream"]
    base = [FAKE, BF16, FAKE, F32, FAKE, BF16, 4, 64, 1e-6, FAKE, FAKE, BF16, 2, FAKE, FAKE, None]

    def call(**kw):
        return lib.moe_rmsnorm(*[kw.get(n, v) for n, v in zip(names, base)])
    for bad in (dict(T=-1), dict(d=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(code=3),
                dict(code=-1), dict(x=None), dict(w=None), dict(y=None, code=0), dict(res=None), dict(out=None),
                dict(q=None), dict(s=None), dict(code=1, q=None), dict(code=1, s=None)):
        assert call(**bad) == INV, bad
    for k in ("x", "res", "w", "out", "y"):
        assert call(**{k: FAKE + 8}) == INV, k
    assert call(q=FAKE + 4) == INV and call(s=FAKE + 2) == INV
    for bad in (dict(xt=2), dict(rt=7), dict(wt=-1), dict(yt=2), dict(d=12), dict(T=1 << 30, d=264)):
        assert call(**bad) == UNS, bad
    assert call(T=0) == 0
    assert call(T=0, x=None, w=None) == 0
    # types of tensors that are not given are not looked at
    assert call(T=0, res=None, out=None, rt=9, y=None, yt=9) == 0


def test_quantize_validation(lib):
    names = ["x", "t", "T", "d", "q", "s", "stream"]
    base = [FAKE, BF16, 4, 64, FAKE, FAKE, None]

    def call(**kw):
        return lib.moe_quantize_blocks_fp8(*[kw.get(n, v) for n, v in zip(names, base)])
    for bad in (dict(T=-1), dict(d=0), dict(x=None), dict(q=None), dict(s=None), dict(x=FAKE + 8), dict(q=FAKE + 4),
                dict(s=FAKE + 2)):
        assert call(**bad) == INV, bad
    for bad in (dict(t=2), dict(d=12), dict(T=1 << 30, d=264)):
        assert call(**bad) == UNS, bad
    assert call(T=0, x=None) == 0


def test_linear_validation(lib):
    names = ["xq", "xs", "rows", "n_x", "offs", "n_rows", "E", "S", "nseg", "K", "O", "w", "ws", "dt", "y", "stream"]
    base = [FAKE, FAKE, FAKE, 16, FAKE, 64, 8, 0, 1, 256, 320, FAKE, FAKE, BF16, FAKE, None]

    def call(**kw):
        return lib.moe_grouped_linear_fp8(*[kw.get(n, v) for n, v in zip(names, base)])
    for bad in (dict(n_rows=-1), dict(E=0), dict(S=-1), dict(nseg=0), dict(nseg=3), dict(K=0), dict(O=0), dict(n_x=0)):
        assert call(**bad) == INV, bad
    for bad in (dict(E=513), dict(S=257), dict(K=96), dict(O=96), dict(n_rows=(1 << 24) + 1, K=64, O=64), dict(n_x=1 << 24),
                dict(n_rows=1 << 23, rows=None), dict(K=65536, O=65536), dict(dt=5)):
        assert call(**bad) == UNS, bad
    for k in ("xq", "xs", "offs", "w", "ws", "y"):
        assert call(**{k: None}) == INV, k
        assert call(**{k: FAKE + 2}) == INV, k
    for k in ("xq", "w", "y"):
        assert call(**{k: FAKE + 8}) == INV, k
    assert call(rows=FAKE + 2) == INV
    assert call(n_rows=0, xq=None, y=None, offs=None) == 0


def test_ffn_validation_and_workspace(lib):
    n = ctypes.c_size_t(0)
    names = ["xq", "xs", "rows", "n_x", "offs", "n_rows", "E", "S", "nseg", "d", "I", "wg", "sg", "wu", "su", "wd", "sd", "h",
             "ws", "nb", "stream"]
    base = [FAKE, FAKE, FAKE, 16, FAKE, 64, 8, 0, 1, 256, 320, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
            ctypes.byref(n), None]

    def call(**kw):
        n.value = kw.pop("size", 1 << 30)
        return lib.moe_grouped_ffn_fp8(*[kw.get(a, v) for a, v in zip(names, base)])
    up = lambda v: (v + 255) // 256 * 256
    need = m.ffn_fp8_workspace_bytes(64, 320)
    assert call(ws=None) == 0 and n.value == need >= up(64 * 320) + up(3 * 64 * 4)
    assert call(ws=None, n_x=0, rows=None, E=3, S=2, nseg=2, d=64) == 0 and n.value == need   # n_rows and I alone
    assert call(size=need - 1) == WS
    for bad in (dict(n_rows=-1), dict(E=0), dict(nseg=3), dict(d=0), dict(I=0), dict(nb=None)):
        assert call(**bad) == INV, bad
    for bad in (dict(E=513), dict(S=257), dict(d=264), dict(I=264), dict(n_rows=1 << 24), dict(n_x=1 << 24)):
        assert call(**bad) == UNS, bad
    for k in ("xq", "xs", "offs", "wg", "sg", "wu", "su", "wd", "sd", "h"):
        assert call(**{k: None}) == INV, k
        assert call(**{k: FAKE + 2}) == INV, k
    assert call(ws=FAKE + 8) == INV
    assert call(n_x=0) == INV                          # a row list of no tokens
    assert call(n_rows=0, xq=None, h=None) == 0


def test_weight_blocks():
    """quantize_fp8_blocks: a scale for each 128 x 128 block, the last ones smaller, and blocks of zeros."""
    w = torch.randn((2, 192, 320), generator=torch.Generator().manual_seed(1))
    w[1, 128:, 256:] = 0
    q, s = m.quantize_fp8_blocks(w)
    assert q.dtype == torch.float8_e4m3fn and q.shape == w.shape and s.shape == (2, 2, 3)
    for e, a, b in ((0, 0, 0), (0, 1, 2), (1, 0, 1)):
        part = w[e, 128 * a:128 * a + 128, 128 * b:128 * b + 128]
        assert abs(float(s[e, a, b]) - float(part.abs().max()) / 448) <= 2.0 ** -22 * float(s[e, a, b])
        back = q[e, 128 * a:128 * a + 128, 128 * b:128 * b + 128].float() * s[e, a, b]
        # half a step: 2^-4 of the value, or of the smallest normal one (2^-6 * 2^-4)
        assert torch.all((back - part).abs() <= (2.0 ** -4 * part.abs()).clamp(min=2.0 ** -10 * float(s[e, a, b])) * (1 + 1e-5))
    assert s[1, 1, 2] == 1 and not q[1, 128:, 256:].float().any()
    p = m.pack_fp8_codes(q)
    assert p.dtype == q.dtype and torch.equal(p.view(torch.uint8), m.pack_fp8_codes(q.view(torch.uint8)))
    qn, pn = q.view(torch.uint8).numpy(), p.view(torch.uint8).numpy().reshape(2, -1)
    for e, r, k in [(0, 0, 0), (1, 191, 319), (0, 17, 70), (1, 5, 129), (0, 15, 63), (1, 16, 64)]:
        off = ((r // 16) * (320 // 64) + k // 64) * 1024 + (((k % 64) // 16) * 16 + r % 16) * 16 + k % 16
        assert pn[e, off] == qn[e, r, k]


def test_bindings_refuse_host_tensors_and_names():
    x = torch.zeros((2, 64))
    f8 = torch.float8_e4m3fn
    with pytest.raises(ValueError):
        m.rmsnorm(x, x[0])
    with pytest.raises(ValueError):
        m.quantize_blocks_fp8(x)
    with pytest.raises(ValueError):
        m.grouped_linear_fp8(x.to(f8), x[:, :1], torch.zeros(2, dtype=torch.int32), 1, 0, 1,
                             torch.zeros((1, 64, 64)).to(f8), torch.zeros((1, 1, 1)))
    with pytest.raises(ValueError):
        m.grouped_ffn_fp8(x.to(f8), x[:, :1], torch.zeros(2, dtype=torch.int32), 1, 0, 1, *[None] * 6)
