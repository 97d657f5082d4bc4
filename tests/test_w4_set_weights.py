"""MoELayerW4.set_weights that fails leaves the layer as it was."""
import os

import pytest
import torch

import combine_topk_ids_gb300 as moe
from combine_topk_ids_gb300 import block

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(moe.LIB_PATH):
        moe.build()


def given(device):
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device=device)  # noqa: E731
    return [z(4, 256, 64), z(4, 256, 2, dtype=BF), z(4, 128, 64), z(4, 128, 2, dtype=BF)]


def off_16_bytes(t):
    """The same tensor one element behind a 16-byte boundary."""
    room = torch.zeros(t.numel() + 16, dtype=t.dtype, device=t.device)
    assert room.data_ptr() % 16 == 0
    return room[1:1 + t.numel()].view(t.shape)


@pytest.mark.parametrize("which", range(4))
def test_refused_weights_are_not_there(which, monkeypatch):
    """The library refuses arrays off 16 bytes: a layer without weights then still has none."""
    monkeypatch.setattr(block, "_stream", lambda stream, dev: None)   # host tensors: refused before any launch
    layer = moe.MoELayerW4(2, 128, 4, 2, 128, 64, device="cpu")
    w = given("cpu")
    w[which] = off_16_bytes(w[which])
    with pytest.raises(moe.MoeError):
        layer.set_weights(*w)
    x, ids = torch.zeros(2, 128, dtype=BF), torch.zeros(2, 2, dtype=torch.int64)
    with pytest.raises(RuntimeError, match="set_weights"):
        layer.forward(x, ids, torch.ones(2, 2))


def test_refused_weights_keep_the_old_ones(monkeypatch):
    monkeypatch.setattr(block, "_stream", lambda stream, dev: None)
    layer = moe.MoELayerW4(2, 128, 4, 2, 128, 64, device="cpu")
    layer.weights = old = given("cpu")
    layer._addresses = addresses = [t.data_ptr() for t in old]
    w = given("cpu")
    w[2] = off_16_bytes(w[2])
    with pytest.raises(moe.MoeError):
        layer.set_weights(*w)
    assert layer.weights is old and layer._addresses is addresses


@pytest.mark.gpu
def test_refused_weights_on_the_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    layer = moe.MoELayerW4(2, 128, 4, 2, 128, 64)
    g = torch.Generator().manual_seed(0)
    w = [torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8).cuda() if t.dtype == torch.uint8
         else torch.rand(t.shape, generator=g).to(BF).cuda() for t in given("cpu")]
    layer.set_weights(*w)
    x = torch.randn((2, 128), generator=g).to(BF).cuda()
    ids, rw = torch.tensor([[0, 3], [2, 1]], device="cuda"), torch.ones((2, 2), device="cuda")
    want = layer.forward(x, ids, rw).clone()
    assert want.abs().sum() > 0
    with pytest.raises(moe.MoeError):
        layer.set_weights(off_16_bytes(w[0]), *w[1:])
    assert torch.equal(layer.forward(x, ids, rw), want)
