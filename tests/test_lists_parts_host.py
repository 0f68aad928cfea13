"""Lists of many tiles on the CPU: the launches of clipping into other buffers
and in place, and the scratch's size."""
import os
import re

from conftest import ROOT
from test_lists_alias_host import run_native


def test_launches_and_tables_of_many_tiles(tmp_path):
    run_native(tmp_path, "list_parts_checks", ["reducer.cpp", "grad_list.cpp"])


def test_the_header_names_the_scratch_and_the_launches():
    text = open(os.path.join(ROOT, "include", "ddp.h")).read()
    source = open(os.path.join(ROOT, "bucketed_gradient_all_amd", "csrc", "grad_list.h")).read()
    partials = int(re.search(r"kMaxPartials = (\d+)", source).group(1))
    assert f"(at most {partials * 8 // 1024} KiB, at least 8 bytes)" in text
    assert "one to three launches" in text
