"""TrainLayer's device status: what each call of a step finds reaches the caller."""
import pytest
import torch

import mixture_experts_layer_group_b200 as moe
from mixture_experts_layer_group_b200.train import TrainLayer

pytestmark = pytest.mark.gpu
T, D, F, N, K = 40, 64, 64, 8, 2


@pytest.fixture(autouse=True)
def _lib():
    from mixture_experts_layer_group_b200 import build
    build.build()
    yield
    torch.cuda.synchronize()


def case(dtype):
    gen = torch.Generator().manual_seed(1)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]

    def new(*shape):
        return (torch.randn(shape, generator=gen) * shape[-1] ** -0.5).to(dt).cuda()

    cfg = moe.make_cfg(d=D, d_ff=F, n_routed=N, n_shared=1, top_k=K, score="sigmoid", normalize=True, dtype=dtype)
    w = {"W_r": new(N, D), "W1": new(N, F, D), "W3": new(N, F, D), "W2": new(N, D, F), "Ws1": new(F, D),
         "Ws3": new(F, D), "Ws2": new(D, F)}
    return TrainLayer(cfg, w, max_tokens=T), new(T, D), new(T, D)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("spoil", ["idx", "counts", "shared_counts"])
def test_status_of_the_backwards_calls(dtype, spoil):
    """The router's backward, the routed block's and the shared one's each report what they were given."""
    layer, x, dy = case(dtype)
    layer.forward(x), layer.backward(dy)
    assert layer.device_status() == 0
    layer.forward(x)
    if spoil == "idx":
        layer.saved["idx"][7, 1] = -1  # no expert: this slot has no gradient
    else:
        layer.saved[spoil][0] += 1     # counts that do not add up: no row is computed
    layer.backward(dy)
    layer.forward(x), layer.backward(dy)  # a clean step afterwards does not hide it
    assert layer.device_status() == moe.MOE_DEV_BAD_EXPERT
    assert layer.device_status() == 0


def test_status_in_a_graph():
    layer, x, dy = case("bf16")
    side = torch.cuda.Stream()
    layer.forward(x), layer.backward(dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer.forward(x)
        layer.backward(dy)
    graph.replay()
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    good = x.clone()
    x[3, 5] = float("nan")
    graph.replay()
    x.copy_(good)
    graph.replay()
    torch.cuda.synchronize()
    assert layer.device_status() == moe.MOE_DEV_NONFINITE
    graph.replay()
    torch.cuda.synchronize()
    assert layer.device_status() == 0


def mark_of(norm):
    return int(norm.view(torch.int32)) == moe.MOE_NORM_INCOMPLETE


@pytest.mark.parametrize("sizes", [[], [5], [40000, 16385, 2], [513] * 700], ids=len)
@pytest.mark.parametrize("inplace,limit", [(True, 0.5), (True, 2.0), (False, 0.5)])
def test_a_norm_buffer_keeps_the_mark_of_an_incomplete_clip(sizes, inplace, limit):
    """The kernel writes the norm over anything but the mark, which it leaves, whatever else the call does."""
    srcs = [torch.full((n,), 2.0 ** -5, device="cuda") for n in sizes]
    dsts = srcs if inplace else [torch.empty_like(t) for t in srcs]
    grads = moe.GradList(srcs, None if inplace else dsts)
    want = 2.0 ** -5 * sum(sizes) ** 0.5
    ws = torch.empty(moe.grad_norm_workspace_size(grads), dtype=torch.uint8, device="cuda")
    sumsq = torch.empty(1, dtype=torch.float64, device="cuda")
    norm = torch.full((1,), float("nan"), device="cuda")

    def clip():
        moe.grad_norm(grads, sumsq, ws)
        moe.grad_clip(grads, sumsq, limit * want, norm)

    clip()
    assert abs(float(norm) - want) <= 2.0 ** -20 * want and not mark_of(norm)
    for t in srcs:
        t.fill_(2.0 ** -5)
    norm.view(torch.int32).fill_(moe.MOE_NORM_INCOMPLETE)
    for _ in range(2):
        clip()
        assert mark_of(norm)
    for t in dsts:  # the gradients are clipped all the same (a second time in place: within the limit)
        assert bool(((t - 2.0 ** -5 * min(1.0, limit)).abs() <= 2.0 ** -24).all())
    norm.zero_()
    clip()
    assert not mark_of(norm) and float(norm) <= want * (1 + 2.0 ** -20)


def test_a_layer_reports_an_incomplete_clip_once():
    layer, x, dy = case("bf16")
    layer.forward(x), layer.backward(dy)
    before = float(layer.clip(1e9))
    assert layer.device_status() == 0
    layer.norm.view(torch.int32).fill_(moe.MOE_NORM_INCOMPLETE)  # as a wait that ran out leaves it
    assert torch.isnan(layer.clip(1e9)).all()
    assert layer.device_status() == moe.MOE_DEV_WAIT_TIMEOUT and layer.device_status() == 0
    assert float(layer.clip(1e9)) == before


def test_the_norms_of_two_clips_keep_their_values():
    layer, x, dy = case("bf16")
    layer.forward(x), layer.backward(dy)
    first = layer.clip(1e9)
    for g in layer.grads.values():
        g.mul_(4.0)
    second = layer.clip(1e9, stream=torch.cuda.current_stream())
    assert float(second) == 4.0 * float(first) > 0.0


# Calls that follow one another without a wait of the host, on one workspace, with other row counts, selections
# and values each time: a kernel that read what the call before left there would give that call's results.


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,f", [(72, 136), (520, 264)])
def test_block_backwards_in_a_row_read_what_is_their_own(dtype, d, f):
    gen = torch.Generator().manual_seed(d)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]

    def new(*shape):
        return torch.randn(shape, generator=gen).to(dt).cuda()

    counts = [[17, 0, 40, 3], [0, 58, 1, 1], [15, 15, 15, 15], [60, 0, 0, 0]]
    R, E = 60, 4
    cfg = moe.make_cfg(d, f, E, 0, 1, dtype=dtype)
    ws = torch.empty(moe.experts_backward_workspace_size(cfg, R), dtype=torch.uint8, device="cuda")
    calls = []
    for c in counts:
        ins = [torch.tensor(c, dtype=torch.int32, device="cuda"), new(R, d), torch.rand(R, generator=gen).cuda(),
               new(E, f, d), new(E, f, d), new(E, d, f), new(R, 2 * f), new(R, d)]
        outs = [torch.empty(R, d, dtype=dt, device="cuda"), torch.empty(R, device="cuda")]
        outs += [torch.empty_like(w) for w in ins[3:6]]
        calls.append((ins, outs))

    def run(ins, outs):
        moe.experts_backward(cfg, R, *ins, *outs, ws)

    want = []
    for ins, outs in calls:
        ws.fill_(255)
        run(ins, outs)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.fill_(7.0)
    for turn in range(30):
        for i in range(len(calls)):
            run(*calls[(i * (turn % 3 + 1)) % len(calls)])
    for ins, outs in calls:
        run(ins, outs)
    torch.cuda.synchronize()
    for (_, outs), ref in zip(calls, want):
        for got, t in zip(outs, ref):
            assert torch.equal(got, t)
    assert moe.device_status(cfg, R, ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [40, 700])
def test_router_backwards_in_a_row_read_what_is_their_own(dtype, T):
    gen = torch.Generator().manual_seed(T)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    d, n, k = 264, 24, 3
    cfg = moe.make_cfg(d, 8, n, 0, k, score="sigmoid", normalize=True, dtype=dtype)
    ws = torch.empty(moe.route_backward_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    calls = []
    for _ in range(3):
        logits = torch.randn(T, n, generator=gen).cuda()
        ins = [torch.randn(T, d, generator=gen).to(dt).cuda(), torch.randn(n, d, generator=gen).to(dt).cuda(), logits,
               torch.topk(logits, k).indices.to(torch.int32), torch.randn(T, k, generator=gen).cuda()]
        calls.append((ins, [torch.empty_like(ins[0]), torch.empty_like(ins[1])]))

    def run(ins, outs):
        moe.route_backward(cfg, T, *ins, None, *outs, ws)

    want = []
    for ins, outs in calls:
        ws.fill_(255)
        run(ins, outs)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    for turn in range(30):
        for i in range(len(calls)):
            run(*calls[(i * (turn % 2 + 1)) % len(calls)])
    for ins, outs in calls:
        run(ins, outs)
    torch.cuda.synchronize()
    for (_, outs), ref in zip(calls, want):
        for got, t in zip(outs, ref):
            assert torch.equal(got, t)
    assert moe.device_status(cfg, T, ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("train", [False, True])
def test_block_forwards_in_a_row_read_what_is_their_own(dtype, train):
    gen = torch.Generator().manual_seed(5)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]

    def new(*shape):
        return torch.randn(shape, generator=gen).to(dt).cuda()

    R, E, d, f = 60, 4, 520, 264
    cfg = moe.make_cfg(d, f, E, 0, 1, dtype=dtype)
    ws = torch.empty(moe.experts_workspace_size(cfg, R), dtype=torch.uint8, device="cuda")
    calls = []
    for c in ([17, 0, 40, 3], [0, 58, 1, 1], [60, 0, 0, 0]):
        ins = [torch.tensor(c, dtype=torch.int32, device="cuda"), new(R, d), torch.rand(R, generator=gen).cuda(),
               new(E, f, d), new(E, f, d), new(E, d, f)]
        calls.append((ins, [torch.empty_like(ins[1])] + ([new(R, 2 * f)] if train else [])))

    def run(ins, outs):
        (moe.experts_train if train else moe.experts)(cfg, R, *ins, *outs, ws)

    want = []
    for ins, outs in calls:
        ws.fill_(255)
        run(ins, outs)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    for turn in range(40):
        for i in range(len(calls)):
            run(*calls[(i * (turn % 2 + 1)) % len(calls)])
    for ins, outs in calls:
        run(ins, outs)
    torch.cuda.synchronize()
    for (_, outs), ref in zip(calls, want):
        for got, t in zip(outs, ref):
            assert torch.equal(got, t)
    assert moe.device_status(cfg, R, ws) == 0
