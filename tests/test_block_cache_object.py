"""api.BlockCache without a GPU: its descriptor stands for the tensors it was made of."""
import dataclasses

import pytest
import torch

from mtp_speculative_draft_lm_b200 import api


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale", "desc", "device"])
def test_fields_are_not_replaced(name):
    """Another tensor in a field would leave the descriptor with the address of one that may be gone."""
    cache = api.BlockCache.empty(3, 2, 64, 16, device="cpu")
    with pytest.raises(dataclasses.FrozenInstanceError):
        setattr(cache, name, torch.zeros(1))
    assert [getattr(cache.desc, n) for n in ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale")] == [
        t.data_ptr() for t in cache.tensors()]


def test_caches_are_equal_to_themselves_alone():
    a, b = (api.BlockCache.empty(2, 1, 64, 16, device="cpu") for _ in range(2))
    assert a == a and a != b and len({a, b}) == 2
