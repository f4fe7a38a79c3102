"""Workspace sizes: a workspace for some number of tokens or rows also holds a
call of fewer, so a layer sized once by its largest batch takes every batch."""
import pytest

import mixture_experts_layer_group_b200 as moe
from mixture_experts_layer_group_b200 import build as moe_build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe_build.build()


# the layers of the benchmark's configurations at token counts just past a step of the router's split count,
# and the widest routers beside the narrowest experts, where the router's scratch weighs most
CASES = [
    (dict(d=1280, d_ff=896, n_routed=63, n_shared=1, top_k=7), 17056),
    (dict(d=7168, d_ff=2048, n_routed=256, n_shared=1, top_k=8, n_groups=8, topk_groups=4), 18656),
    (dict(d=5120, d_ff=1536, n_routed=160, n_shared=2, top_k=6), 20000),
    (dict(d=512, d_ff=8, n_routed=512, n_shared=0, top_k=1), 9000),
    (dict(d=2048, d_ff=8, n_routed=512, n_shared=0, top_k=1), 9000),
    (dict(d=2048, d_ff=8, n_routed=5, n_shared=0, top_k=1, dtype="f32"), 30001),
    (dict(d=8, d_ff=8, n_routed=2, n_shared=0, top_k=2, dtype="f32"), 5000),
]


@pytest.mark.parametrize("kw,most", CASES, ids=[f"{c['d']}x{c['n_routed']}" for c, _ in CASES])
@pytest.mark.parametrize("size", [moe.workspace_size, moe.workspace_size_host, moe.route_backward_workspace_size,
                                  moe.experts_workspace_size, moe.experts_backward_workspace_size],
                         ids=lambda f: f.__name__)
def test_a_workspace_holds_calls_of_fewer_tokens(kw, most, size):
    cfg = moe.make_cfg(**kw)
    before = 0
    for t in sorted({*range(0, most, 64), *range(1, most, 997), *range(max(0, most - 130), most + 1)}):
        need = size(cfg, t)
        assert need >= before, t
        before = need


def test_a_workspace_still_holds_its_own_call_at_the_largest_sizes():
    """A size is at least that of the call's own tokens: what the routed and shared rows alone take."""
    cfg = moe.make_cfg(d=2048, d_ff=1024, n_routed=8, n_shared=1, top_k=2)
    for T in (1, 63, 64, 65, 1 << 20, 1 << 29):
        assert moe.workspace_size(cfg, T) >= T * 2 * ((2 + 2 + 1) * 2048 + (2 + 1) * 1024)
