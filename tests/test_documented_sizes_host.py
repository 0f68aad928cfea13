"""Workspace sizes on the CPU against what the header tells a caller to reserve.

The figures are read from the header's text, so that neither changes alone."""
import os
import re

import pytest

import bucketed_gradient_all_amd as ddp
from conftest import ROOT

with open(os.path.join(ROOT, "include", "ddp.h")) as f:
    HEADER = " ".join(line.strip(" *\n") for line in f)


def _figure(pattern, function):
    """The number in the comment before the function's declaration."""
    comment = HEADER[:HEADER.index(f"size_t {function}(")].rsplit("/*", 1)[1]
    found = re.findall(pattern, comment)
    assert len(found) == 1, (pattern, comment)
    return int(found[0])


@pytest.mark.parametrize("numel", [[0], [1], [1023], [1024], [1025], [2048], [1 << 20] * 3, [5] * 1000, [1 << 30],
                                   [3, 0, 70001, 1 << 24]])
@pytest.mark.parametrize("state", [0, 1])
def test_adamw_tables(numel, state):
    """80 bytes a tensor that has elements, 4 bytes a tile, and each tensor's
    ends: two tiles more; alignment and one spare of 16 bytes."""
    tensor = _figure(r"(\d+) bytes a tensor", "ddp_adamw_workspace_bytes")
    tile = _figure(r"4 bytes per (\d+) elements", "ddp_adamw_workspace_bytes")
    none = [0] * len(numel)
    size = ddp.ddp_adamw_workspace_bytes(ddp.AdamWDesc(numel, none, none, none, none, state=state))
    some = [n for n in numel if n]
    most = tensor * len(some) + sum(4 * (n // tile + 2) for n in some) + 3 * 16
    assert 4 * sum(n // tile for n in some) + tensor * len(some) <= size <= most


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("width,x,y", [(1, 0, 0), (64, 1, 1), (752, 1, 1), (1100, 0, 0), (1280, 0, 1), (1280, 0, 0),
                                       (2057, 1, 1), (2560, 2, 2), (2880, 1, 1), (4096, 0, 0), (16384, 1, 1), (16385, 1, 1),
                                       (8193, 0, 0), (1 << 20, 1, 1)])
def test_layer_norm_partial_sums(width, x, y, kind):
    """At most that many times dweight and dbias in fp32, the alignment and a
    spare of 256 bytes; and a call of fewer rows never asks for more."""
    times = _figure(r"at most (\d+) times dweight and dbias", "ddp_layernorm_grad_workspace_bytes")
    desc = ddp.LayerNormDesc(width, kind=kind, x_dtype=x, y_dtype=y)
    switch = (64 << 20) // (width * (2 if x else 4))   # rows from which on they are read past the caches
    counts = sorted({0, 1, 2, 100, 1000, 100000, (1 << 31) - 1}
                    | {max(0, switch + d) for d in (-1, 0, 1, 2, 1000)} | {switch * 3, switch * 10})
    sizes = [ddp.ddp_layernorm_grad_workspace_bytes(desc, n) for n in counts if n < 1 << 31]
    assert sizes == sorted(sizes)
    assert sizes[-1] <= times * 2 * 4 * width + 2 * 256


def test_the_most_partial_sums_are_asked_for():
    times = _figure(r"at most (\d+) times dweight and dbias", "ddp_layernorm_grad_workspace_bytes")
    most = max(ddp.ddp_layernorm_grad_workspace_bytes(ddp.LayerNormDesc(w, x_dtype=1), 1 << 20) // (8 * w)
               for w in range(8, 16384, 8))
    assert most == times
