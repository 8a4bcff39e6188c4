"""The library's choice of int8 kernels (top_expert_routing_amd/csrc/i8_plan.h), asked through a small host program."""
from __future__ import annotations

import functools
import os
import shutil
import subprocess
import tempfile

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "top_expert_routing_amd", "csrc")
SRC = os.path.join(HERE, "native", "i8_plan_query.cpp")


@functools.lru_cache(maxsize=None)
def _program():
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    folder = tempfile.TemporaryDirectory(prefix="i8_plan")
    exe = os.path.join(folder.name, "i8_plan_query")
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", SRC, "-o", exe], check=True)
    return exe, folder


def launches(queries):
    """(kernel, width, blocks, grid x, grid y) of each (product, n_rows, E, n_shared, nseg, K, cols)."""
    text = "".join(" ".join(map(str, q)) + "\n" for q in queries)
    out = subprocess.run([_program()[0]], input=text, capture_output=True, text=True, check=True, timeout=60).stdout
    plans = [(line.split()[0], *map(int, line.split()[1:])) for line in out.splitlines()]
    assert len(plans) == len(queries)
    return plans


def ask(queries):
    """(kernel, width, blocks) of each of them."""
    return [p[:3] for p in launches(queries)]


def linear(n_rows, E, n_shared, nseg, K, O):
    return ask([("linear", n_rows, E, n_shared, nseg, K, O)])[0]


def ffn(n_rows, E, n_shared, nseg, d, I):
    """Plans of the gate/up and the down product."""
    return ask([("gate_up", n_rows, E, n_shared, nseg, d, I), ("down", n_rows, E, n_shared, nseg, I, d)])
