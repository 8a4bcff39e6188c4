"""quantize_fp8_blocks on weights that are not all finite: the rule of the rows' quantiser (CPU only)."""
import pytest
import torch

import top_expert_routing_amd as m


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_blocks_that_are_not_finite(bad, dtype):
    """Scale NaN and codes 0 in the block itself, the others as they are without it."""
    w = torch.randn((2, 192, 320), generator=torch.Generator().manual_seed(3)).to(dtype)
    q0, s0 = m.quantize_fp8_blocks(w)
    assert torch.isfinite(s0).all()
    hit = torch.zeros(w.shape, dtype=torch.bool)
    for e, r, k in ((0, 5, 7), (1, 191, 319)):
        w[e, r, k] = bad
        hit[e, r // 128 * 128:(r // 128 + 1) * 128, k // 128 * 128:(k // 128 + 1) * 128] = True
    q, s = m.quantize_fp8_blocks(w)
    q, q0 = q.view(torch.uint8), q0.view(torch.uint8)
    assert s[0, 0, 0].isnan() and s[1, 1, 2].isnan() and int(s.isnan().sum()) == 2
    assert not q[hit].any()
    assert torch.equal(q[~hit], q0[~hit]) and torch.equal(s[~s.isnan()], s0[~s.isnan()])
