"""Routing with scores and the int8 calls: exports, refusals on the host, workspace sizes, packing
(CPU only; no kernel is launched)."""
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


@pytest.mark.parametrize("header,names", [("libmoe_route.h", _lib.ROUTE_EXPORTS), ("libmoe_int8.h", _lib.INT8_EXPORTS)])
def test_headers_declare_what_is_exported(lib, header, names):
    text = open(os.path.join(ROOT, "include", header)).read()
    declared = re.findall(r"^moe_status\s+(moe_\w+)\s*\(", text, re.M)
    assert sorted(declared) == sorted(names)
    for n in names:
        assert hasattr(lib, n)


def test_route_validation(lib):
    base = [FAKE, F32, None, 4, 64, 8, 0, 8, 4, 0, 1, 1.0, FAKE, FAKE, None]
    names = ["logits", "dtype", "bias", "T", "E", "k", "score", "n_groups", "top_groups", "rank", "renorm", "scale",
             "ids", "w", "stream"]

    def call(**kw):
        return lib.moe_route(*[kw.get(n, v) for n, v in zip(names, base)])
    assert call(T=-1) == INV
    assert call(E=0) == INV
    assert call(k=0) == INV
    assert call(k=33) == INV                       # 4 groups of 8 experts stay
    assert call(n_groups=0) == INV
    assert call(n_groups=7) == INV                 # 64 % 7 != 0
    assert call(top_groups=0) == INV
    assert call(top_groups=9) == INV
    assert call(score=2) == INV
    assert call(rank=2) == INV
    assert call(renorm=2) == INV
    assert call(scale=math.nan) == INV
    assert call(scale=math.inf) == INV
    assert call(dtype=5) == UNS
    assert call(E=520) == UNS
    assert call(E=512, n_groups=128, top_groups=128) == UNS
    assert call(T=1 << 23, E=512) == UNS           # T * E past int32
    assert call(logits=None) == INV
    assert call(ids=None) == INV
    assert call(w=None) == INV
    assert call(logits=FAKE + 2) == INV
    assert call(logits=FAKE + 1, dtype=BF16) == INV
    assert call(bias=FAKE + 2) == INV
    assert call(T=0, logits=None, ids=None, w=None) == 0


def test_quantize_validation(lib):
    f = lib.moe_quantize_rows_i8
    assert f(FAKE, BF16, -1, 64, FAKE, FAKE, None) == INV
    assert f(FAKE, BF16, 4, 0, FAKE, FAKE, None) == INV
    assert f(FAKE, BF16, 4, 60, FAKE, FAKE, None) == UNS
    assert f(FAKE, 9, 4, 64, FAKE, FAKE, None) == UNS
    assert f(FAKE, BF16, 1 << 20, 1 << 12, FAKE, FAKE, None) == UNS
    assert f(None, BF16, 4, 64, FAKE, FAKE, None) == INV
    assert f(FAKE, BF16, 4, 64, None, FAKE, None) == INV
    assert f(FAKE, BF16, 4, 64, FAKE, None, None) == INV
    assert f(FAKE + 8, BF16, 4, 64, FAKE, FAKE, None) == INV
    assert f(FAKE, BF16, 4, 64, FAKE + 4, FAKE, None) == INV
    assert f(FAKE, BF16, 4, 64, FAKE, FAKE + 2, None) == INV
    assert f(None, BF16, 0, 64, None, None, None) == 0


def test_linear_validation(lib):
    names = ["xq", "xs", "rows", "n_x", "offs", "n_rows", "E", "S", "nseg", "K", "O", "w", "ws", "dt", "y", "stream"]
    base = [FAKE, FAKE, None, 0, FAKE, 64, 8, 0, 1, 256, 512, FAKE, FAKE, BF16, FAKE, None]

    def call(**kw):
        return lib.moe_grouped_linear_i8(*[kw.get(n, v) for n, v in zip(names, base)])
    for bad in (dict(n_rows=-1), dict(E=0), dict(S=-1), dict(nseg=0), dict(nseg=3), dict(K=0), dict(O=0)):
        assert call(**bad) == INV, bad
    for bad in (dict(E=513), dict(S=257), dict(K=288), dict(O=288), dict(K=131072 + 64), dict(dt=3),
                dict(n_rows=1 << 24), dict(K=65536, O=65536), dict(rows=FAKE, n_x=1 << 24),
                dict(n_rows=(1 << 24) + 1, K=64, O=64)):
        assert call(**bad) == UNS, bad
    for bad in (dict(xq=None), dict(xs=None), dict(offs=None), dict(w=None), dict(ws=None), dict(y=None),
                dict(xq=FAKE + 8), dict(w=FAKE + 8), dict(ws=FAKE + 4), dict(y=FAKE + 8), dict(offs=FAKE + 2),
                dict(rows=FAKE + 2, n_x=4), dict(rows=FAKE, n_x=0)):
        assert call(**bad) == INV, bad
    assert call(n_rows=0, xq=None, y=None, offs=None) == 0


def test_ffn_validation_and_workspace(lib):
    n = ctypes.c_size_t(0)
    names = ["x", "rows", "n_x", "offs", "n_rows", "E", "S", "nseg", "d", "I", "wg", "sg", "wu", "su", "wd", "sd", "h",
             "ws", "nb", "stream"]
    base = [FAKE, FAKE, 16, FAKE, 64, 8, 0, 1, 256, 320, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
            ctypes.byref(n), None]

    def call(**kw):
        n.value = kw.pop("size", 1 << 30)
        return lib.moe_grouped_ffn_i8(*[kw.get(a, v) for a, v in zip(names, base)])
    up = lambda v: (v + 255) // 256 * 256
    assert call(ws=None) == 0 and n.value == up(16 * 256) + up(16 * 4) + up(64 * 320) + up(3 * 64 * 4)
    assert call(ws=None, n_x=0) == 0 and n.value == up(64 * 256) + up(64 * 4) + up(64 * 320) + up(3 * 64 * 4)
    assert m.ffn_i8_workspace_bytes(64, 16, 256, 320) == up(16 * 256) + 256 + up(64 * 320) + up(3 * 64 * 4)
    need = m.ffn_i8_workspace_bytes(64, 16, 256, 320)
    assert call(size=need - 1) == WS
    assert call(rows=None, size=need) == WS           # without a row list 64 rows are quantised
    for bad in (dict(n_rows=-1), dict(E=0), dict(nseg=3), dict(d=0), dict(n_x=-1), dict(nb=None)):
        assert call(**bad) == INV, bad
    for bad in (dict(E=513), dict(S=257), dict(d=264), dict(I=264), dict(d=131072 + 64), dict(n_rows=1 << 24),
                dict(n_x=1 << 24)):
        assert call(**bad) == UNS, bad
    for k in ("x", "offs", "wg", "sg", "wu", "su", "wd", "sd", "h"):
        assert call(**{k: None}) == INV, k
        assert call(**{k: FAKE + 2}) == INV, k
    assert call(ws=FAKE + 8) == INV
    assert call(n_x=0) == INV                          # a row list of no tokens
    assert call(n_rows=0, x=None, h=None) == 0


def test_pack_layout():
    g = torch.Generator().manual_seed(1)
    q = torch.randint(-128, 128, (2, 32, 192), generator=g, dtype=torch.int8)
    p = m.pack_i8_codes(q).numpy().reshape(2, -1)
    qn = q.numpy()
    for e, r, k in [(0, 0, 0), (1, 31, 191), (0, 17, 70), (1, 5, 129), (0, 15, 63), (1, 16, 64)]:
        off = ((r // 16) * (192 // 64) + k // 64) * 1024 + (((k % 64) // 16) * 16 + r % 16) * 16 + k % 16
        assert p[e, off] == qn[e, r, k]
    assert np.array_equal(np.sort(p.ravel()), np.sort(qn.ravel()))
    with pytest.raises(TypeError):
        m.pack_i8_codes(q.float())
    with pytest.raises(ValueError):
        m.pack_i8_codes(q[:, :, :96])


def test_bindings_refuse_host_tensors_and_names():
    x = torch.zeros((2, 64))
    with pytest.raises(ValueError):
        m.route(x, 2)
    with pytest.raises(ValueError):
        m.quantize_rows_i8(x)
    with pytest.raises(ValueError):
        m.grouped_linear_i8(x.to(torch.int8), x[:, 0], torch.zeros(2, dtype=torch.int32), 1, 0, 1,
                            torch.zeros((1, 64, 64), dtype=torch.int8), torch.zeros((1, 64)))
    with pytest.raises(ValueError):
        m.grouped_ffn_i8(x.bfloat16(), torch.zeros(2, dtype=torch.int32), 1, 0, 1, *[None] * 6)
