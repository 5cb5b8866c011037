"""A launch that fails after the host's side of a cache has changed: the device has not followed, so the cache takes no
further change.  (The launch is left out on the host; nothing fails on the device.)"""
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa

DEV = "cuda"


def test_the_diagnostic_can_be_set_without_a_gpu():
    uaa.debug_fail_launch(2)
    uaa.debug_fail_launch()


def cache():
    c = uaa.PagedCache(2, 12, 16, 2, 64, 4, 3)
    c.append([0, 1], [20, 40])
    c.fork([0], [2])
    c.free([1])
    c.append([3], [33])
    c.free([0])
    c.fork([2], [0])
    return c


CALLS = {
    "append": lambda c: c.append([0, 3], [1, 1]),
    "fork": lambda c: c.fork([2], [1]),
    "truncate": lambda c: c.truncate([3, 0], [1, 2]),
    "compact": lambda c: c.compact(),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name,n", [("append", 0), ("append", 1), ("fork", 0), ("truncate", 0), ("compact", 0), ("compact", 1)])
def test_a_cache_whose_device_did_not_follow(name, n):
    """Launch 0 of a call that copies pages is the copy, 1 the table's changes."""
    c = cache()
    if name == "compact":
        c.free([0, 2])
        assert c.pages_of(3) == [2, 3, 4]
    before = c.table.clone(), c.lens.clone()
    uaa.debug_fail_launch(n)
    try:
        with pytest.raises(uaa.UAAError, match="UAA_ERR_CUDA.*launch failed"):
            CALLS[name](c)
    finally:
        uaa.debug_fail_launch()
    assert torch.equal(c.table, before[0]) and torch.equal(c.lens, before[1])
    for again in (lambda: c.append([0], [1]), lambda: c.append([], []), lambda: c.fork([3], [1]), lambda: c.free([3]), c.compact):
        with pytest.raises(uaa.UAAError, match="UAA_ERR_CUDA.*earlier call"):
            again()
    assert torch.equal(c.table, before[0]) and torch.equal(c.lens, before[1])
    assert isinstance(c.length(3), int) and c.free_pages >= 0
    one = cache()  # another cache is not concerned
    one.append([3], [1])
    assert one.lens.tolist() == [20, 0, 20, 34]
    uaa.check_device_status()
