"""E4M3 codes next to the border between two of them, at scales just above 2^-100, below which a block counts as zeros:
equal to the definition's, whose quotient is rounded correctly to fp32, down to the smallest scale."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as Q
from helpers import announce, f64_of, np_of, require_gpu
from test_gpu_norm_fp8 import DEV, F8

import top_expert_routing_amd as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _rows():
    """Rows of 128: a largest value, and every midpoint of two codes times the scale it gives, as the nearest fp32 number
    and the ones beside it."""
    v = torch.arange(128, dtype=torch.uint8).view(F8).double().numpy()
    v = np.sort(v[np.isfinite(v)])
    mid = (v[1:] + v[:-1]) / 2
    rng = np.random.default_rng(4)
    tops = np.exp2(rng.uniform(-91.1, -78, 300)).astype(np.float32)
    tops[0] = np.float32(float.fromhex("0x1.bffffap-91"))          # scale 0x1.fffffap-100
    rows = []
    for top in tops:
        _, s = Q.quantize_blocks(np.array([[top]], np.float32))
        near = (mid * np.float64(s[0, 0])).astype(np.float32)
        for x in (near, np.nextafter(near, np.float32(1)), np.nextafter(near, np.float32(0))):
            r = np.zeros(128, np.float32)
            r[:126], r[127] = x, -top
            rows.append(r)
    rows[0][126] = np.float32(float.fromhex("0x1.fffffcp-110"))    # quotient 0x1.000002p-10: code 1, not 0
    one = np.zeros(128, np.float32)
    one[0] = np.float32(float.fromhex("0x1.fffffcp-100")) * np.float32(448)
    one[1] = np.float32(float.fromhex("0x1.7ffffcp-108"))          # quotient 0x1.7ffffep-9: below the tie
    return np.stack(rows + [one])


def test_quantize_at_the_smallest_scales():
    announce("quantize smallest scales")
    x = _rows()
    q, s = moe.quantize_blocks_fp8(torch.from_numpy(x).to(DEV))
    qr, sr = Q.quantize_blocks(x)
    np.testing.assert_array_equal(np_of(s), sr)
    np.testing.assert_array_equal(f64_of(q), qr)


@pytest.mark.parametrize("wide", [128, 20480])
def test_norm_at_the_smallest_scales(wide):
    """The same rows through the norm, whose codes are those of r * weight; 20480 columns are read twice."""
    announce(f"norm smallest scales {wide}")
    x = _rows()
    if wide > 128:
        x = np.resize(x, (6, wide))
    x = torch.from_numpy(x.copy()).to(DEV)
    _, q, s = moe.rmsnorm(x, torch.ones(wide, device=DEV), codes="fp8", want_y=False)
    qr, base = Q.quantize_blocks(x.cpu().numpy())
    np.testing.assert_array_equal(f64_of(q), qr)
    np.testing.assert_allclose(f64_of(s), base.astype(np.float64) * 1e3, rtol=1e-5)
