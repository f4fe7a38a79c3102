"""The row movements of a training step by themselves, in either type: combine's
backward copies rows, the dispatch's backward adds them up; and the router's
backward by permuted row, as a step calls it.

Tolerance of a sum of n terms added in fp32 and rounded once: each addition is off
by at most 2^-24 of a partial sum, which the terms' absolute values S bound, so
n 2^-24 S; the rounding to bf16 adds 2^-8 of what is rounded."""
import pytest
import torch

import mixture_experts_layer_group_b200 as moe

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _lib():
    from mixture_experts_layer_group_b200 import build
    build.build()
    yield
    torch.cuda.synchronize()


def dispatched(T, N, k, d, dtype, seed, drop=0.0, **cfg_kw):
    """A selection, some pairs of which name no expert, and where the dispatch puts its rows."""
    gen = torch.Generator().manual_seed(seed)
    cfg = moe.make_cfg(d, 8, N, 0, k, dtype=dtype, **cfg_kw)
    idx = torch.stack([torch.randperm(N, generator=gen)[:k] for _ in range(T)]).to(torch.int32)
    idx[torch.rand((T, k), generator=gen) < drop] = -1
    idx = idx.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets, pos = torch.empty(N, **i32), torch.empty(N + 1, **i32), torch.empty((T, k), **i32)
    x = torch.randn((T, d), generator=gen).to(DT[dtype]).cuda()
    gates = torch.rand((T, k), generator=gen).cuda()
    rows, gate = torch.empty((T * k, d), dtype=DT[dtype], device="cuda"), torch.empty(T * k, device="cuda")
    ws = torch.empty(moe.workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    moe.dispatch_rows(cfg, T, idx, gates, x, counts, offsets, pos, rows, gate, ws)
    return cfg, gen, idx, pos, x, gates, gate


SIZES = [(1, 4, 1, 8), (7, 5, 3, 8), (50, 6, 2, 136), (33, 40, 16, 264), (257, 64, 8, 1280), (65, 63, 7, 2056)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("T,N,k,d", SIZES)
def test_combine_backward_copies_rows(T, N, k, d, drop, dtype):
    cfg, gen, idx, pos, dy, _, _ = dispatched(T, N, k, d, dtype, T, drop)
    out = torch.full((T * k, d), 3.0, dtype=DT[dtype], device="cuda")
    moe.combine_backward(cfg, T, dy, pos, out)
    want = torch.full_like(out, 3.0)  # rows that no pair names stay as they are
    for t, p in enumerate(pos.tolist()):
        for r in p:
            if r >= 0:
                want[r] = dy[t]
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("T,N,k,d", SIZES)
def test_dispatch_backward_sums_rows(T, N, k, d, drop, dtype):
    cfg, gen, idx, pos, _, _, _ = dispatched(T, N, k, d, dtype, T + 1, drop)
    dx_rows, shared, router = (torch.randn((n, d), generator=gen).to(DT[dtype]).cuda() for n in (T * k, T, T))
    placed = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    placed[pos[pos >= 0].long()] = True
    dx_rows[~placed] = float("nan")  # rows that no pair names are not read
    pad = torch.cat([dx_rows.double().nan_to_num(0.0), torch.zeros((1, d), dtype=torch.float64, device="cuda")])
    terms = pad[torch.where(pos >= 0, pos, T * k).long()]
    for sh, ro in ((None, None), (shared, None), (None, router), (shared, router)):
        out = torch.full((T, d), 3.0, dtype=DT[dtype], device="cuda")
        moe.dispatch_backward(cfg, T, dx_rows, pos, sh, ro, out)
        parts = [terms.transpose(0, 1)] + [t.double()[None] for t in (sh, ro) if t is not None]
        ref, size = sum(p.sum(0) for p in parts), sum(p.abs().sum(0) for p in parts)
        bound = (k + 2) * 2.0 ** -24 * size
        if dtype == "bf16":
            bound = bound + 2.0 ** -8 * (ref.abs() + bound)
        assert bool(((out.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("T,N,k,d", [(1, 4, 1, 8), (50, 6, 2, 136), (300, 40, 16, 264), (517, 63, 7, 1280)])
def test_router_backward_by_permuted_row_is_that_by_slot(T, N, k, d, score, normalize, dtype):
    """The dispatch carries the gates to the rows; carried by it, the gates' gradients give the same bits."""
    cfg, gen, idx, pos, x, dG, dG_rows = dispatched(T, N, k, d, dtype, T + 2, 0.0, score=score, normalize=normalize,
                                                    route_scale=2.5)
    logits = torch.randn((T, N), generator=gen).cuda()
    W_r = torch.randn((N, d), generator=gen).to(DT[dtype]).cuda()
    ws = torch.empty(moe.route_backward_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    got = []
    for slot_pos, g in ((None, dG), (pos, dG_rows)):
        dx, dW = torch.empty_like(x), torch.empty_like(W_r)
        moe.route_backward(cfg, T, x, W_r, logits, idx, g, slot_pos, dx, dW, ws)
        assert moe.device_status(cfg, T, ws) == 0
        got.append((dx, dW))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
