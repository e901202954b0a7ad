"""The kernels of decode over parts of a cache that start beside the kernel before them load nothing by the read-only path."""
from tests.test_chained_loads import code, read_only_loads


def test_blocks_and_prefixes():
    for name in ("block_decode.cu", "shared_prefix.cu"):
        assert read_only_loads(name) == [], name
    # the join waits for both kernels before it loads: the wait comes first in it
    join = code("block_decode.cu").split("block_join_kernel(")[1]
    assert join.index("griddepcontrol.wait") < join.index("parts.pair[")
