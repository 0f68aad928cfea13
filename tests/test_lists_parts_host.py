"""Lists of many tiles on the CPU: the launches of clipping into other buffers
and in place, and the scratch's size."""
from test_lists_alias_host import run_native


def test_launches_and_tables_of_many_tiles(tmp_path):
    run_native(tmp_path, "list_parts_checks", ["reducer.cpp", "grad_list.cpp"])
