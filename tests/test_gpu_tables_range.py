"""Chunk tables over the largest pool that a slot number can name."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
CH = 64


@pytest.mark.parametrize("B", [3, 3000])          # one cluster; the launches for larger tables
def test_largest_pool(B):
    from learned_sparse_kv_b200 import lsa as L
    n_slots = 2 ** 31 - 1
    table = torch.full((B, 3), -1, dtype=torch.int32, device="cuda")
    cached, new = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    table[0, 0], table[1, 0], table[B - 1, 0] = n_slots - 1, 0, 2
    cached[0], cached[1], cached[B - 1] = 64, 1, 64
    new[0], new[1], new[B - 1] = 1, 63, 65
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    nxt, slots, pos, off, free = L.build_tables(table, cached, new, n_slots, 130, status=st)
    assert st.item() == 0 and free.item() == n_slots - 6
    want = np.full((B, 3), -1, np.int32)
    want[0], want[1, 0], want[B - 1] = [n_slots - 1, 1, -1], 0, [2, 3, 4]
    np.testing.assert_array_equal(nxt.cpu().numpy(), want)
    np.testing.assert_array_equal(pos.cpu().numpy(), [64, *range(1, 64), *range(64, 129), -1])
    np.testing.assert_array_equal(slots.cpu().numpy(), [CH, *range(1, 64), *range(3 * CH, 4 * CH), 4 * CH, -1])
    assert off[-1].item() == 129
