"""The free ring's initial order: every block once, as the host block manager asks it."""
import numpy as np
import pytest
import torch

import paged_kv_cache_400_b200 as pk


@pytest.mark.parametrize("order", [None, [3, 0, 2, 1], np.array([1, 3, 0, 2]), torch.tensor([2, 1, 0, 3])])
def test_good_orders(order):
    ring, state = pk.make_free_ring(4, order, "cpu")
    want = [0, 1, 2, 3] if order is None else [int(x) for x in order]
    assert ring.dtype == torch.int32 and ring.tolist() == want and state.tolist() == [0, 4, 0, 0]


@pytest.mark.parametrize("order", [[0, 1, 2], [0, 1, 2, 2], [0, 1, 2, 4], [-1, 1, 2, 3], [[0, 1], [2, 3]], []])
def test_bad_orders(order):
    with pytest.raises(ValueError):
        pk.make_free_ring(4, order, "cpu")
    if len(order) == 4:  # the block manager refuses the same
        with pytest.raises(pk.PagedKVError):
            pk.BlockManager(4, order)
