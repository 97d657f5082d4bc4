"""moe_product_fp8's choice of tiles, restated from its rule: the sizes that the GPU tests take reach every
kind of tile and every number of blocks that share one, with one weight matrix and with several."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_topk_ids_gb300", "csrc",
                      "product_fp8.cu")
SMS = 152
# rows of a tile (0: the wide tiles), its columns, ns of a k-step, ns before and after them
TILES = ((16, 128, 200, 1000), (32, 128, 230, 1000), (64, 128, 320, 1000), (128, 128, 550, 1000), (0, 256, 500, 1500))

# M, N, K with the rows of a tile and the blocks that share one: odd sizes, the smallest of each kind that
# a search found, and sizes that the product is measured at
ONE = [(533, 3885, 128, 0, 1), (3, 131, 128, 16, 1), (3, 131, 1536, 16, 2), (3, 133, 2048, 16, 4), (3, 133, 4096, 16, 8),
       (1227, 131, 128, 32, 1), (17, 4977, 2176, 32, 2), (321, 133, 2176, 32, 4), (159, 137, 5888, 32, 8),
       (2459, 133, 128, 64, 1), (1277, 155, 2816, 64, 2), (609, 143, 2048, 64, 4), (321, 133, 14080, 64, 8),
       (1933, 519, 128, 128, 1), (2643, 133, 5888, 128, 2), (1299, 149, 3456, 128, 4), (645, 133, 46080, 128, 8),
       (777, 1003, 1408, 64, 1), (61, 4096, 7168, 64, 4), (101, 4096, 7168, 128, 4), (256, 4096, 7168, 128, 2)]
# M, N, K, G likewise
MANY = [(17, 1045, 128, 17, 0, 1), (3, 131, 128, 3, 16, 1), (3, 133, 1024, 3, 16, 2), (3, 133, 2048, 3, 16, 4), (3, 135, 4224, 3, 16, 8),
        (1117, 133, 128, 17, 32, 1), (19, 917, 1024, 9, 32, 2), (51, 137, 2048, 17, 32, 4), (21, 131, 4224, 9, 32, 8),
        (2207, 131, 128, 17, 64, 1), (39, 967, 1280, 9, 64, 2), (99, 137, 2048, 17, 64, 4), (35, 139, 5888, 9, 64, 8),
        (711, 923, 128, 17, 128, 1), (195, 387, 2816, 17, 128, 2), (195, 135, 2560, 17, 128, 4), (65, 145, 22272, 9, 128, 8)]


def most_tiles(M, G, rows):
    return M // rows + min(G, M) if G else -(-M // rows)


def choice(M, N, K, G=0):
    """The tile with the least estimated time: its rows, and the blocks that share it."""
    kb, best, least = K // 128, None, None
    for tile, cols, step, around in TILES:
        rows, blocks = tile or 128, -(-N // cols)
        most = tiles = most_tiles(M, G, rows) * blocks
        if G:
            groups = min(G, M)
            tiles = max(2 * M // rows + groups, 2 * groups) * blocks // 2
            step = max(step, 370 if tile else 800)
        for split in (1, 2, 4, 8) if tile else (1,):
            if split > 1 and (most * split > SMS or kb < 4 * split):
                break
            ns = -(-tiles * split // SMS) * (-(-kb // split) * step + around)
            ns += (1000 + 8 * rows if split > 1 else 0) + (25 * rows if split == 8 else 0)
            if least is None or ns < least:
                least, best = ns, (tile, split)
    return best


def test_the_tiles_are_the_kernels():
    table = re.search(r"kTiles\[\] = \{\n?(.*?)\};", open(SOURCE).read(), re.S).group(1)
    names = {"kTileN": 128, "kWideN": 256}
    got = tuple(tuple(names.get(v.strip()) or int(v) for v in row.split(",")) for row in re.findall(r"\{(.*?)\}", table))
    assert got == TILES


@pytest.mark.parametrize("M,N,K,rows,split", ONE)
def test_choice_of_one_matrix(M, N, K, rows, split):
    assert choice(M, N, K) == (rows, split)


@pytest.mark.parametrize("M,N,K,G,rows,split", MANY)
def test_choice_of_many(M, N, K, G, rows, split):
    assert choice(M, N, K, G) == (rows, split)


def test_every_kind_is_reached():
    every = {(r, s) for r in (16, 32, 64, 128) for s in (1, 2, 4, 8)} | {(0, 1)}
    assert {t[-2:] for t in ONE} == every and {t[-2:] for t in MANY} == every
