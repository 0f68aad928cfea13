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
