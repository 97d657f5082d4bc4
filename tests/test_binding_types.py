"""What is no tensor raises TypeError wherever the bindings of moe_block.h and moe_grouped.h take a tensor."""
import os

import pytest
import torch

import combine_topk_ids_gb300 as moe

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(moe.LIB_PATH):
        moe.build()
    return moe.lib()


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


POSITION, WEIGHTS = z(3, 2, dtype=I32), z(3, 2, dtype=F32)
CALLS = {
    "moe_sort_picks": dict(topk_ids=z(3, 2, dtype=I32), num_experts=4, offsets=z(5, dtype=I32), position=POSITION,
                           workspace=z(64, dtype=U8), source=z(6, dtype=I32), status=z(1, dtype=I32)),
    "moe_sort_rows": dict(x=z(3, 256, dtype=U8), position=POSITION, rows=z(6, 256, dtype=U8), x_scales=z(3, 2, dtype=F32),
                          rows_scales=z(6, 2, dtype=F32)),
    "moe_sort_rows_backward": dict(drows=z(6, 64), position=POSITION, dx=z(3, 64)),
    "moe_unsort_rows": dict(rows=z(6, 64), weights=WEIGHTS, position=POSITION, out=z(3, 64)),
    "moe_unsort_rows_backward": dict(dout=z(3, 64), rows=z(6, 64), weights=WEIGHTS, position=POSITION, drows=z(6, 64),
                                     dweights=z(3, 2, dtype=F32)),
    "moe_quantize_fp8": dict(x=z(3, 256), codes=z(3, 256, dtype=U8), scales=z(3, 2, dtype=F32), live_rows=z(1, dtype=I32)),
    "moe_swiglu_fp8": dict(gate_up=z(3, 512), codes=z(3, 256, dtype=U8), scales=z(3, 2, dtype=F32), live_rows=z(1, dtype=I32)),
    "moe_product_fp8": dict(a=z(3, 128, dtype=U8), a_scales=z(3, 1, dtype=F32), b=z(2, 64, 128, dtype=U8),
                            b_scales=z(2, 1, 1, dtype=F32), out=z(3, 64), offsets=z(3, dtype=I32), status=z(1, dtype=I32)),
    "moe_add_rmsnorm": dict(x=z(3, 256), residual=z(3, 256), weight=z(256), eps=1e-6, sum_out=z(3, 256), out=z(3, 256),
                            out_fp8=z(3, 256, dtype=U8), scales=z(3, 2, dtype=F32), rstd=z(3, dtype=F32)),
    "moe_add_rmsnorm_backward": dict(dout=z(3, 256), h=z(3, 256), weight=z(256), rstd=z(3, dtype=F32), dx=z(3, 256),
                                     dweight=z(256, dtype=F32), workspace=z(64, dtype=U8), dsum=z(3, 256)),
}


@pytest.mark.parametrize("name,argument", [(n, a) for n, kw in CALLS.items() for a, v in kw.items() if torch.is_tensor(v)])
def test_no_tensor(name, argument):
    for other in ([1, 2], 5, "workspace", object()):
        with pytest.raises(TypeError):
            getattr(moe, name)(**{**CALLS[name], argument: other})


@pytest.mark.parametrize("name", list(CALLS))
def test_all_else_is_right(name):
    with pytest.raises(ValueError, match="host memory"):
        getattr(moe, name)(**CALLS[name])
