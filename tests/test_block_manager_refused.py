"""A prompt that the pool has no room for leaves no prefix behind: its blocks are never written."""
import pytest

from paged_kv_cache_29_gb300.block_manager import BlockManager, OutOfBlocks


def test_a_refused_prompt_is_not_found_as_a_prefix():
    m = BlockManager(4, 4)
    m.admit("a", range(4))
    with pytest.raises(OutOfBlocks):
        m.admit("b", [*range(4), *range(50, 70)])      # one block found, three fresh ones, then none
    m.check()
    assert m.num_free == 3 and m.sequences() == ["a"]
    assert m.admit("c", [*range(4), *range(50, 58)]) == 4   # what "a" wrote, and nothing of "b"
    m.release("a")
    m.release("c")
    assert m.admit("d", [*range(4), *range(50, 58)]) == 12
    m.check()
