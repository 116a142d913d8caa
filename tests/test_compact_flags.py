"""How a chunk of a compaction says that its cells are loaded, from the kernel's source: another CTA then stores over them, and only a
release that is acquired there keeps the loads before those stores.  (On a GPU a missing one shows as rare wrong cells, if at all.)"""
import re

from tests.test_pair_handover import body


def test_the_flag_of_a_loaded_chunk_is_released_and_acquired():
    move = body("cache_runs.cu", "compact_move_kernel(")
    flag = re.search(r'"st\.(\w+)\.gpu\.global\.u32 \[%0\], %1;" ::"l"\(w\.loaded \+ chunk\)', move)
    assert flag and flag.group(1) == "release"
    lead = move[:flag.start()]
    assert lead.rindex("load_cells(") < lead.rindex("__syncthreads()")  # every thread's loads are before it
    after = move[flag.end():]
    assert after.index("wait_loaded(") < after.index("__syncthreads_and(") < after.index("store_cells(")
    assert "ld.acquire.gpu" in body("cache_runs.cu", "bool wait_loaded(")
