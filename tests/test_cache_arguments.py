"""Arguments that a kernel could only fault on are refused on the host."""
import ctypes

import pytest

import ulysses_dit_attention_gb300 as uaa
from test_cache_pages import Host, err


@pytest.mark.parametrize("starts,seqs", [((1 << 20) + 2, 1 << 20), (1 << 20, (1 << 20) + 1)])
def test_append_of_results_that_are_not_aligned(starts, seqs):
    h = Host(4, 16, 2, 2)
    n, a, b = h._two([0], [1])
    pools = uaa._POOLS.pack(1 << 20, 1 << 20, 1 << 20, 1 << 20, 1, 256)
    P = ctypes.c_void_p
    assert uaa.lib().uaa_pages_append(h.h, pools, n, a, b, P(starts), P(seqs), None) == -1 and "aligned" in err()
    assert h.row(0) == (0, []) and h.free() == 4
