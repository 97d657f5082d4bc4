"""The example's block of grouped operators sees a product that gave up."""
import os
import sys

import pytest
import torch

import combine_topk_ids_gb300 as moe
import gen
from test_grouped_gpu import built  # noqa: F401

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import grouped_experts  # noqa: E402

pytestmark = pytest.mark.gpu


def test_every_call_that_can_give_up_has_the_blocks_word(monkeypatch):
    block, x, residual = grouped_experts.make(gen.CONFIGS["tiny_ll_em"], 8)
    words, product, order = [], moe.moe_product_fp8, moe.moe_sort_picks

    def gives_up_once(*args, status=None, **kw):
        product(*args, status=status, **kw)
        words.append(status)
        if len(words) == 2:          # as the kernel does
            status |= moe.STATUS_TIMEOUT

    def sorted_with(*args, status=None, **kw):
        order(*args, status=status, **kw)
        words.append(status)

    block.status.fill_(0x70)         # what an earlier forward may have left
    block.forward(x, residual)
    block.check()
    monkeypatch.setattr(moe, "moe_sort_picks", sorted_with)
    monkeypatch.setattr(moe, "moe_product_fp8", gives_up_once)
    block.forward(x, residual)
    assert len(words) == 5 and all(w is block.status for w in words)
    with pytest.raises(RuntimeError, match="0x4"):
        block.check()
    block.forward(x, residual)       # the next one starts anew
    block.check()


def test_a_bad_expert_id_is_seen():
    block, x, residual = grouped_experts.make(gen.CONFIGS["tiny_ll_em"], 4)
    block.forward(x, residual)
    block.ids[1, 0] = block.E
    moe.moe_sort_picks(block.ids, block.E, block.offsets, block.position, block.workspace, status=block.status)
    assert block.status.dtype == torch.int32
    with pytest.raises(RuntimeError, match="0x%x" % moe.STATUS_BAD_EXPERT_ID):
        block.check()
