"""Which kernel an int8 product runs on, and how it is launched (CPU only)."""
import itertools
import os
import shutil
import subprocess

import numpy as np
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


# (E, shared, K or d, O or I) of batches with a priority segment, small to large
PRIORITY = [(128, 0, 2880, 2880), (64, 0, 2048, 1024), (16, 1, 1024, 512), (8, 2, 256, 1344), (300, 4, 512, 512)]


@pytest.mark.parametrize("E,S,d,I", PRIORITY)
def test_a_priority_segment_does_not_change_the_kernels(E, S, d, I):
    """Tiles take an expert's rows of both segments as one sequence, so the rows of an expert decide, however many
    groups they lie in (but for the 128-row tiles, whose lists hold fewer groups)."""
    queries = [(n, E, S) for n in range(1, 300 * E, max(1, E // 3))]
    plan = lambda nseg: i8_plan.ask([q for n, E, S in queries for q in
                                     (("linear", n, E, S, nseg, d, I), ("gate_up", n, E, S, nseg, d, I), ("down", n, E, S, nseg, I, d))])
    for one, two, q in zip(plan(1), plan(2), [n for n, _, _ in queries for _ in range(3)]):
        if two[0] == "tile_wide" and one[0] == "tile_half" and 2 * E + S > 380:
            continue
        assert one == two, (q, one, two)


@pytest.mark.parametrize("E,nseg,shared", [(4, 1, 0), (4, 2, 1), (70, 2, 0), (33, 1, 3)])
def test_the_grid_holds_every_tile(E, nseg, shared):
    """No XCD has more (tile, column chunk) items than the launch gives it blocks."""
    rng = np.random.default_rng(E + nseg)
    for O in (64, 448, 1152, 2048):
        for most in (1, 3, 17, 40):
            sizes = rng.integers(0, most + 1, (nseg, E))
            n = int(sizes.sum()) + 5 * shared
            if n == 0:
                continue
            kernel, width, blocks = i8_plan.linear(n, E, shared, nseg, 192, O)
            bm, columns = (16, 16 * width) if kernel == "few" else (16 * width, 128)
            chunks = -(-O // columns)
            up = lambda rows: -(-rows // bm)
            tiles = [up(sizes[0, e]) for e in range(E)]                      # of each group, in group order
            if nseg == 2:
                tiles += [up(sizes[:, e].sum()) - up(sizes[0, e]) for e in range(E)]
            tiles += [up(5)] * shared
            items = np.zeros(8, int)
            for g, t in enumerate(tiles):
                for j in range(chunks):
                    items[(g * chunks + j) % 8] += t
            assert blocks % 8 == 0 and items.max() <= blocks // 8, (O, most, kernel)


def test_launches_stay_below_two_to_the_32_threads():
    """Every launch of 512-thread blocks that the sizes allow (codes, values and matrices below 2^31) has fewer than
    2^32 threads along x, all the plan's blocks, and XCDs dealt as in one row of blocks."""
    queries = []
    for E, S, nseg in ((1, 0, 1), (64, 0, 1), (512, 256, 1), (512, 256, 2)):
        for n in (1, 33, 64, 160, 768, 1280, 2000, 20480, 1 << 17, 1 << 24):
            for K in (64, 192, 1024, 131072):
                most = min((2 ** 31 - 1) // n, (2 ** 31 - 1) // K)
                for O in {64, 448, most // 64 * 64, most // 128 * 64}:
                    if O and n * K < 2 ** 31:
                        queries += [("linear", n, E, S, nseg, K, O), ("gate_up", n, E, S, nseg, K, O), ("down", n, E, S, nseg, O, K)]
    over = 0
    for q, (kernel, width, blocks, x, y) in zip(queries, i8_plan.launches(queries)):
        assert 0 <= blocks <= 2 ** 25 and x * 512 < 2 ** 32 and y <= 65535, q
        assert x * y >= blocks and (y == 1 or x % 8 == 0), q
        over += blocks * 512 >= 2 ** 32
    assert over > 4                       # some need more than one row


@pytest.mark.parametrize("steps,compiles", [(4, True), (3, False)])
def test_tiles_are_longer_than_what_is_requested_ahead(tmp_path, steps, compiles):
    """A K as short as the stages requested ahead would take a tile's last stages from the wrong rows: such a minimum
    does not compile."""
    csrc = tmp_path / "top_expert_routing_amd" / "csrc"
    native = tmp_path / "tests" / "native"
    csrc.mkdir(parents=True)
    native.mkdir(parents=True)
    shutil.copy(os.path.join(i8_plan.CSRC, "item_plan.h"), csrc)
    text = open(os.path.join(i8_plan.CSRC, "i8_plan.h")).read()
    assert "kTileMinK = 4 * kStep;" in text
    (csrc / "i8_plan.h").write_text(text.replace("kTileMinK = 4 * kStep;", f"kTileMinK = {steps} * kStep;"))
    shutil.copy(i8_plan.SRC, native)
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    r = subprocess.run([cxx, "-std=c++17", "-fsyntax-only", str(native / "i8_plan_query.cpp")], capture_output=True, text=True)
    assert (r.returncode == 0) == compiles and (compiles or "requested ahead" in r.stderr)
