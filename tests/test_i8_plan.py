"""Which kernel an int8 product runs on, and how it is launched (CPU only)."""
import itertools

import pytest

import i8_plan


def test_sizes_of_the_four_kernels():
    """One size well inside each kernel's range."""
    assert i8_plan.linear(5, 1, 0, 1, 2048, 2048)[0] == "few"
    assert i8_plan.linear(1024, 64, 0, 1, 2048, 1024)[0] == "stream"
    assert i8_plan.linear(4096, 1, 0, 1, 2048, 2048)[0] == "tile_half"
    assert i8_plan.linear(16384, 1, 0, 1, 2048, 2048)[0] == "tile_wide"
    assert [p[0] for p in i8_plan.ffn(8, 64, 0, 1, 2048, 1024)] == ["few", "few"]
    assert [p[0] for p in i8_plan.ffn(1024, 64, 0, 1, 2048, 1024)] == ["stream", "stream"]
    assert [p[0] for p in i8_plan.ffn(8192, 64, 0, 1, 2048, 1024)] == ["tile_half", "tile_wide"]
    assert [p[0] for p in i8_plan.ffn(32768, 64, 0, 1, 2048, 1024)] == ["tile_wide", "tile_wide"]


@pytest.mark.parametrize("E,S,nseg", [(1, 0, 1), (8, 0, 1), (8, 2, 2), (64, 0, 2), (512, 256, 1), (512, 256, 2)])
def test_both_products_of_few_rows_agree(E, S, nseg):
    """The SwiGLU product is in fp32 for both products of an FFN or for neither."""
    for n, d, I in itertools.product((1, 2, 9, 33, 80, 81, 160, 161, 999, 20000), (64, 448, 2048), (64, 320, 1088, 2048)):
        up, down = i8_plan.ffn(n, E, S, nseg, d, I)
        assert (up[0] == "few") == (down[0] == "few"), (n, d, I)
        assert up[1] in (0, 1, 2) and down[1] in (0, 1, 2, 4)
