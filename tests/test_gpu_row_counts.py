"""Rows and columns past int32: the C calls take both as int32, so the bindings refuse more instead of passing on what is left
of the number in 32 bits."""
import pytest
import torch

from helpers import announce, require_gpu
from test_gpu_norm_fp8 import DEV

import top_expert_routing_amd as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("T,d", [(1, 2 ** 32 + 8), (2 ** 32 + 5, 8)])
def test_sizes_past_int32_are_refused(T, d):
    announce(f"rows past int32 {T} x {d}")
    x = torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
    w = torch.empty(d, dtype=torch.bfloat16, device=DEV)
    for call in (lambda: moe.quantize_blocks_fp8(x), lambda: moe.quantize_rows_i8(x), lambda: moe.rmsnorm(x, w, codes="i8")):
        with pytest.raises((ValueError, moe.MoeError)):
            call()
    del x, w
    torch.cuda.empty_cache()
