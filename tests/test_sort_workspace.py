"""moe_sort_picks_workspace_size: a count for each expert of every block and a word for each block, to 16 bytes."""
import os

import pytest

import combine_topk_ids_gb300 as moe


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(moe.LIB_PATH):
        moe.build()
    return moe.lib()


def blocks(picks, E):
    """One block up to 1024 picks; above, blocks of 512, at most 152 of them and 152 * 256 counts."""
    return 1 if picks <= 1024 else min(-(-picks // 512), 152, 152 * 256 // E)


@pytest.mark.parametrize("T,k,E", [(0, 1, 1), (1, 8, 256), (512, 2, 64), (1024, 1, 2048), (1025, 1, 7), (513, 8, 64), (16381, 4, 128),
                                   (19456, 4, 256), (19457, 4, 256), (32768, 8, 256), (32768, 8, 257), (32768, 8, 2048),
                                   (9728, 1, 2048), ((1 << 31) // 8 - 128, 8, 2048), ((1 << 31) - 1024, 1, 1)])
def test_size(T, k, E):
    n = blocks(T * k, E)
    assert n >= 1 and moe.moe_sort_picks_workspace_size(T, k, E) == -(-4 * n * (E + 1) // 16) * 16
