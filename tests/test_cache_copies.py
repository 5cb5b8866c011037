"""A cache is one object: who holds which page is kept by a handle that its owner frees, so it is not copied or pickled."""
import copy
import pickle

import pytest
import torch

import ulysses_dit_attention_gb300 as uaa


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, pickle.dumps], ids=["copy", "deepcopy", "pickle"])
def test_a_cache_is_not_copied(how):
    cache = uaa.PagedCache(1, 2, 16, 1, 64, 2, 2, device="cpu")
    with pytest.raises(TypeError, match="PagedCache"):
        how(cache)
    assert cache.free_pages == 2 and cache.length(0) == 0


def test_a_model_that_holds_a_cache_is_not_copied():
    model = torch.nn.Linear(2, 2)
    model.cache = uaa.PagedCache(1, 2, 16, 1, 64, 2, 2, device="cpu")
    with pytest.raises(TypeError, match="PagedCache"):
        copy.deepcopy(model)
    assert copy.copy(model).cache is model.cache
