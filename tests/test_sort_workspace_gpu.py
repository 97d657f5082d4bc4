"""moe_sort_picks with a workspace of exactly the size asked for, and guards around it."""
import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
from oracle import grouped as og
from test_grouped_gpu import I32, built, draw_ids  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E", [(0, 1, 1), (1, 1, 1), (128, 8, 256), (1025, 1, 7), (513, 8, 64), (16381, 4, 128), (32768, 8, 256),
                                   (20000, 1, 2048), (3000, 5, 1025)])
def test_nothing_is_written_around_the_workspace(T, k, E):
    ids = draw_ids(T, k, E, 0.1, 1)
    n, guard = moe.moe_sort_picks_workspace_size(T, k, E), 4096
    room = torch.full((n + 2 * guard,), 170, dtype=torch.uint8, device="cuda")
    offsets, position = torch.empty(E + 1, dtype=I32, device="cuda"), torch.empty((T, k), dtype=I32, device="cuda")
    moe.moe_sort_picks(torch.tensor(ids).cuda(), E, offsets, position, room[guard:guard + n])
    assert (room[:guard] == 170).all() and (room[guard + n:] == 170).all()
    want = og.order(ids, E)
    np.testing.assert_array_equal(offsets.cpu().numpy(), want[0])
    np.testing.assert_array_equal(position.cpu().numpy(), want[1])
