"""Which kernel a block-scaled FP8 product runs on, and how it is launched (CPU only)."""
import itertools
import os
import shutil
import subprocess

import numpy as np
import pytest

import fp8_plan

CSRC = os.path.join(fp8_plan.HERE, "..", "top_expert_routing_amd", "csrc")


def test_sizes_of_the_four_kernels():
    """One size well inside each kernel's range."""
    assert fp8_plan.linear(5, 1, 0, 1, 2048, 2048) == "few"
    assert fp8_plan.linear(1024, 64, 0, 1, 2048, 1024) == "stream"
    assert fp8_plan.linear(4096, 1, 0, 1, 2048, 2048) == "tile_codes"
    assert fp8_plan.linear(4096, 1, 0, 1, 2048, 2048, f32=True) == "tile_exact"
    assert fp8_plan.ffn(8, 64, 0, 1, 2048, 1024) == ("few", "few")
    assert fp8_plan.ffn(1024, 64, 0, 1, 2048, 1024) == ("stream", "stream")
    assert fp8_plan.ffn(32768, 64, 0, 1, 2048, 1024) == ("tile_codes", "tile_codes")
    assert fp8_plan.ffn(32 * 128, 128, 0, 1, 2880, 2880) == ("tile_codes", "tile_codes")
    assert fp8_plan.ffn(32 * 64, 64, 0, 1, 2048, 1024) == ("stream", "stream")


def test_tiles_need_a_row_list_and_a_ring_of_stages():
    """No tile with fewer than three blocks of K, nor with more groups than its lists hold."""
    for K, kernel in ((64, "stream"), (256, "stream"), (320, "tile_codes"), (384, "tile_codes")):
        assert fp8_plan.linear(8192, 1, 0, 1, K, 2048) == kernel
    for E, S, nseg, kernel in ((512, 256, 1, "tile_codes"), (400, 0, 2, "tile_codes"), (400, 1, 2, "stream"), (512, 0, 2, "stream")):
        assert fp8_plan.linear(100000, E, S, nseg, 512, 1024) == kernel


@pytest.mark.parametrize("E,S,nseg", [(1, 0, 1), (8, 0, 1), (8, 2, 2), (64, 0, 2), (512, 256, 1), (512, 256, 2)])
def test_both_products_of_few_rows_agree(E, S, nseg):
    """The SwiGLU product is in fp32 for both products of an FFN or for neither."""
    for n, d, I in itertools.product((1, 2, 9, 33, 80, 81, 160, 161, 999, 20000), (64, 448, 2048), (64, 320, 1088, 2048)):
        up, down = fp8_plan.ffn(n, E, S, nseg, d, I)
        assert (up == "few") == (down == "few"), (n, d, I)


@pytest.mark.parametrize("E,S,d,I", [(128, 0, 2880, 2880), (64, 0, 2048, 1024), (16, 1, 1024, 512), (8, 2, 256, 1344)])
def test_a_priority_segment_does_not_change_the_kernels(E, S, d, I):
    """Tiles take an expert's rows of both segments as one sequence, so the rows of an expert decide."""
    for n in range(1, 300 * E, max(1, E // 3)):
        a, b = (fp8_plan_pair(n, E, S, nseg, d, I) for nseg in (1, 2))
        assert a == b, n
        if n > 40 * E:
            break


def fp8_plan_pair(n, E, S, nseg, d, I):
    return [p[0] for p in fp8_plan.launches([("linear", n, E, S, nseg, d, I), ("linear_f32", n, E, S, nseg, d, I),
                                             ("gate_up", n, E, S, nseg, d, I), ("down", n, E, S, nseg, I, d)])]


@pytest.mark.parametrize("E,nseg,shared", [(4, 1, 0), (4, 2, 1), (70, 2, 0), (33, 1, 3)])
def test_the_grid_holds_every_tile(E, nseg, shared):
    """No XCD has more (tile, column chunk) items than the launch gives it blocks."""
    rng = np.random.default_rng(E + nseg)
    cases, queries = [], []
    for O in (64, 448, 1152, 2048):
        for most in (1, 3, 17, 40):
            sizes = rng.integers(0, most + 1, (nseg, E))
            n = int(sizes.sum()) + 5 * shared
            if n:
                cases.append((O, sizes))
                queries.append(("linear", n, E, shared, nseg, 192, O))
    seen = set()
    for (O, sizes), (kernel, width, blocks, x, y) in zip(cases, fp8_plan.launches(queries)):
        seen.add((kernel, width))
        bm, columns = (16, 16 * width) if kernel == "few" else (16 * width, 128)
        chunks, up = -(-O // columns), lambda rows: -(-rows // bm)
        tiles = [up(sizes[0, e]) for e in range(E)]                      # of each group, in group order
        if nseg == 2:
            tiles += [up(sizes[:, e].sum()) - up(sizes[0, e]) for e in range(E)]
        tiles += [up(5)] * shared
        items = np.zeros(8, int)
        for g, t in enumerate(tiles):
            for j in range(chunks):
                items[(g * chunks + j) % 8] += t
        assert blocks % 8 == 0 and items.max() <= blocks // 8, (O, kernel)
    assert len(seen) > 1


def test_launches_stay_below_two_to_the_32_threads():
    """Every launch of 512-thread blocks that the sizes allow (codes and values below 2^31) has fewer than 2^32 threads
    along x, and all the plan's blocks."""
    queries = []
    for E, S, nseg in ((1, 0, 1), (64, 0, 1), (512, 256, 1), (512, 256, 2)):
        for n in (1, 33, 64, 160, 768, 1280, 2000, 20480, 1 << 17, 1 << 24):
            for K in (64, 192, 1024, 131072):
                most = min((2 ** 31 - 1) // n, (2 ** 31 - 1) // K)
                for O in {64, 448, most // 64 * 64, most // 128 * 64}:
                    if O and n * K < 2 ** 31:
                        queries += [(p, n, E, S, nseg, K, O) for p in ("linear", "linear_f32", "gate_up")] + [("down", n, E, S, nseg, O, K)]
    for q, (kernel, width, blocks, x, y) in zip(queries, fp8_plan.launches(queries)):
        assert 0 <= blocks <= 2 ** 25 and x * 512 < 2 ** 32 and y <= 65535, q
        assert x * y >= blocks and (y == 1 or x % 8 == 0), q
        assert kernel.startswith("tile") or width in (1, 2, 4), q


@pytest.mark.parametrize("stages,compiles", [(3, True), (1, False)])
def test_tiles_are_longer_than_what_is_requested_ahead(tmp_path, stages, compiles):
    """A K as short as the stages requested ahead would take a tile's rows from a list that has not arrived: such a minimum
    does not compile."""
    csrc, native = tmp_path / "top_expert_routing_amd" / "csrc", tmp_path / "tests" / "native"
    csrc.mkdir(parents=True)
    native.mkdir(parents=True)
    for f in ("item_plan.h", "i8_plan.h"):
        shutil.copy(os.path.join(CSRC, f), csrc)
    text = open(os.path.join(CSRC, "fp8_plan.h")).read()
    assert "kTileMinStages = 3;" in text
    (csrc / "fp8_plan.h").write_text(text.replace("kTileMinStages = 3;", f"kTileMinStages = {stages};"))
    shutil.copy(fp8_plan.SRC, native)
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    r = subprocess.run([cxx, "-std=c++17", "-fsyntax-only", str(native / "fp8_plan_query.cpp")], capture_output=True, text=True)
    assert (r.returncode == 0) == compiles and (compiles or "row list" in r.stderr), r.stderr
