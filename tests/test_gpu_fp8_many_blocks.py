"""The block quantiser on more blocks of 128 columns than one of its launches takes (2^27)."""
import pytest
import torch

from helpers import announce, require_gpu
from test_gpu_norm_fp8 import DEV, F8, _gen

import top_expert_routing_amd as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("T,d", [(2 ** 27 + 77, 8), (2 ** 26 + 5, 136)])
def test_more_blocks_than_one_launch(T, d):
    """Every row of a repeated pattern equals the pattern's; 136 columns are a whole block and one of eight in
    each row, and the launches' border lies between rows."""
    announce(f"quantize {T} x {d}")
    n, nb = 4096, -(-d // 128)
    assert T * nb > 2 ** 27
    x = torch.randn((n, d), generator=_gen(d)).bfloat16().to(DEV)
    q0, s0 = moe.quantize_blocks_fp8(x)
    big = torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
    whole = T // n * n
    big[:whole].view(-1, n, d).copy_(x.expand(whole // n, n, d))
    big[whole:] = x[:T - whole]
    q = torch.full((T, d), 0x7f, dtype=torch.uint8, device=DEV).view(F8)
    s = torch.full((T, nb), -1.0, device=DEV)
    moe.quantize_blocks_fp8(big, q, s)
    del big
    for got, want, cols in ((q.view(torch.uint8), q0.view(torch.uint8), d), (s, s0, nb)):
        for a in range(0, whole, n * 2048):
            part = got[a:min(a + n * 2048, whole)].view(-1, n, cols)
            assert bool((part == want).all()), a
        assert torch.equal(got[whole:], want[:T - whole])
