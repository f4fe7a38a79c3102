"""Layers sized by their largest batch, called with fewer tokens."""
import pytest
import torch

import mixture_experts_layer_group_b200 as moe
from mixture_experts_layer_group_b200.train import TrainLayer

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    from mixture_experts_layer_group_b200 import build
    build.build()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [7168, 6912, 6848, 1])
def test_a_layer_takes_fewer_tokens_than_its_largest_batch(T):
    """9000 tokens of this layer need less router scratch than 7168 do."""
    cfg = moe.make_cfg(d=2048, d_ff=8, n_routed=512, n_shared=0, top_k=1, score="sigmoid", normalize=True)
    gen = torch.Generator().manual_seed(T)

    def new(*shape, std=1.0):
        return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16).cuda()

    w = {"W_r": new(512, 2048, std=2048 ** -0.5), "b": None, "W1": new(512, 8, 2048, std=2048 ** -0.5),
         "W3": new(512, 8, 2048, std=2048 ** -0.5), "W2": new(512, 2048, 8, std=8 ** -0.5)}
    x, dy = new(T, 2048), new(T, 2048)
    got = []
    for most in (9000, T):
        layer = TrainLayer(cfg, w, max_tokens=most)
        got.append([layer.forward(x), layer.backward(dy), *layer.grads.values(),
                    moe.MoELayer(cfg, w, max_tokens=most)(x)])
        assert layer.device_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
