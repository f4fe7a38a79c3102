"""The training entry points against the formulas in 64 bits (plain torch on
fp64 copies of the inputs), at the sizes and layouts where they can go wrong.

Tolerances. A rounding to bf16 moves a value by at most 2^-8 of itself, to
fp32 by 2^-24. A bf16 result here is a sum of products one of whose factors
was rounded to bf16 once (dg, du or gate h; the forward's h), rounded once at
the end: where the sum has one term the two roundings add up to at most 2 *
2^-8 + 2^-16 of the element; where it has many, their signs are independent
and the root mean square is below that. So ||y - ref|| <= (2^-7 + 2^-14)
||ref|| (BF16_TWO); a result with one rounding gets 2^-8 + 2^-14 (BF16_ONE;
the rest covers the fp32 sums). Where a sum cancels, each factor's rounding
counts by its term: elementwise |y - ref| <= 2^-8 |ref| + (2^-8 + 2^-16) S,
with S the sum of the terms' absolute values. fp32 results are sums of up to
n terms of fp32 products: |y - ref| <= (n + 16) 2^-23 S elementwise (16 for
the score functions, whose exp and division are good to a few units)."""
import math

import pytest
import torch

import mixture_experts_layer_group_b200 as moe
from mixture_experts_layer_group_b200.train import TrainLayer

pytestmark = pytest.mark.gpu

BF16_ONE, BF16_TWO = 2.0 ** -8 + 2.0 ** -14, 2.0 ** -7 + 2.0 ** -14
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F64 = torch.float64


@pytest.fixture(autouse=True)
def _lib():
    from mixture_experts_layer_group_b200 import build
    build.build()
    build.build(debug=True)
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def randn(gen, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * std).to(dtype).cuda()


def rel(y, ref):
    y, ref = y.double(), ref.double()
    n = torch.linalg.vector_norm(ref)
    off = torch.linalg.vector_norm(y - ref)
    return float(off / n) if n > 0 else float(off)


def guarded(shape, dtype, fill=None):
    """A tensor in the middle of a larger buffer, and a check that the rest stays as it was."""
    n = math.prod(shape)
    buf = torch.full((n + 512,), 7.0, dtype=dtype, device="cuda")
    t = buf[256:256 + n].view(shape)
    if fill is not None:
        t.fill_(fill)

    def check():
        assert bool((buf[:256] == 7.0).all()) and bool((buf[256 + n:] == 7.0).all()), "written outside the output"
    return t, check


# --------------------------------------------------------------- experts --


class Block:
    """Inputs of one grouped expert block."""

    def __init__(self, counts, d, F, dtype="bf16", gate=True, seed=0):
        gen = torch.Generator().manual_seed(seed)
        E, R, dt = len(counts), sum(counts), DT[dtype]
        self.E, self.R, self.d, self.F, self.dtype, self.counts = E, R, d, F, dtype, counts
        self.cfg = moe.make_cfg(d, F, E, 0, 1, dtype=dtype)
        self.dcounts = torch.tensor(counts, dtype=torch.int32, device="cuda")
        self.x = randn(gen, (R, d), 1.0, dt)
        self.W1, self.W3 = randn(gen, (E, F, d), d ** -0.5, dt), randn(gen, (E, F, d), d ** -0.5, dt)
        self.W2 = randn(gen, (E, d, F), F ** -0.5, dt)
        self.gate = (torch.rand(R, generator=gen) * 0.9 + 0.05).cuda() if gate else None
        self.gu = randn(gen, (R, 2 * F), 1.0, dt)
        self.dy = randn(gen, (R, d), 1.0, dt)

    def weights(self):
        return self.W1, self.W3, self.W2

    def groups(self):
        lo = 0
        for e, n in enumerate(self.counts):
            if n:
                yield e, slice(lo, lo + n)
            lo += n

    def ws(self, backward=True):
        n = (moe.experts_backward_workspace_size if backward else moe.experts_workspace_size)(self.cfg, self.R)
        return torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")

    def forward(self, x=None):
        dt = DT[self.dtype]
        y, c0 = guarded((self.R, self.d), dt, 0.0)
        gu, c1 = guarded((self.R, 2 * self.F), dt, 0.0)
        ws = self.ws(False)
        moe.experts_train(self.cfg, self.R, self.dcounts, self.x if x is None else x, self.gate, *self.weights(), y,
                          gu, ws)
        torch.cuda.synchronize()
        c0(), c1()
        assert moe.device_status(self.cfg, self.R, ws) == 0
        return y, gu

    def backward(self, grad_dtype=None, accumulate=False, start=None, ws=None, expect=0, stream=None):
        dt, gdt = DT[self.dtype], DT[grad_dtype or self.dtype]
        E, R, d, F = self.E, self.R, self.d, self.F
        out, checks = {}, []
        for name, shape, t in (("dx", (R, d), dt), ("dgate", (R,), torch.float32), ("dW1", (E, F, d), gdt),
                               ("dW3", (E, F, d), gdt), ("dW2", (E, d, F), gdt)):
            out[name], check = guarded(shape, t, 3.0 if start is None else start)
            checks.append(check)
        ws = self.ws() if ws is None else ws
        torch.cuda.synchronize()
        moe.experts_backward(self.cfg, R, self.dcounts, self.x, self.gate, *self.weights(), self.gu, self.dy,
                             *out.values(), ws, grad_dtype=grad_dtype, accumulate=accumulate, stream=stream)
        torch.cuda.synchronize()
        for check in checks:
            check()
        if R:
            assert moe.device_status(self.cfg, R, ws) == expect
        return out

    def exact(self):
        """The gradients in 64 bits, and the sums of the terms' absolute values."""
        E, R, d, F = self.E, self.R, self.d, self.F
        z = lambda *s: torch.zeros(s, dtype=F64, device="cuda")  # noqa: E731
        ref = dict(dx=z(R, d), dgate=z(R), dW1=z(E, F, d), dW3=z(E, F, d), dW2=z(E, d, F))
        mag = {k: v.clone() for k, v in ref.items()}
        for e, r in self.groups():
            W1, W3, W2 = (w[e].double() for w in self.weights())
            x, dy = self.x[r].double(), self.dy[r].double()
            g, u = self.gu[r, :F].double(), self.gu[r, F:].double()
            gate = self.gate[r].double()[:, None] if self.gate is not None else 1.0
            s = torch.sigmoid(g)
            h, q = g * s * u, dy @ W2
            du, dg = gate * q * g * s, gate * q * u * s * (1 + g * (1 - s))
            for out, f in ((ref, lambda t: t), (mag, torch.abs)):
                out["dgate"][r] = (f(q) * f(h)).sum(1) if out is ref else ((f(dy) @ f(W2)) * f(h)).sum(1)
                out["dx"][r] = f(dg) @ f(W1) + f(du) @ f(W3)
                out["dW1"][e], out["dW3"][e] = f(dg).T @ f(x), f(du).T @ f(x)
                out["dW2"][e] = f(dy).T @ f(gate * h)
        return ref, mag


def check_block(b, out, ref, mag, grad_dtype=None):
    for name, y in out.items():
        r, m, t = ref[name], mag[name], y.dtype
        assert torch.isfinite(y).all(), name
        off = (y.double() - r).abs()
        if name == "dgate":
            # q summed over d, times h, summed over F: fp32 throughout
            bound = (b.d + b.F + 16) * 2.0 ** -23 * m
        elif b.dtype == "f32":
            # the factor is itself such a sum over d (dg, du); then the rows or 2 F
            bound = None
            assert rel(y, r) <= (max(2 * b.F, max(b.counts)) + b.d + 16) * 2.0 ** -23, (name, rel(y, r))
        else:
            # a factor rounded to bf16; dg and du carry the relative error of
            # q's fp32 sum, which cancellation in q can raise: 2^-16 of the
            # product of the sums' magnitudes covers (d + 16) 2^-23 at d <= 2048
            bound = (2.0 ** -8 if t == torch.bfloat16 else 0.0) * r.abs() + (2.0 ** -8 + 2.0 ** -13) * m
            assert rel(y, r) <= BF16_TWO, (name, rel(y, r))
        if bound is not None:
            assert bool((off <= bound + 1e-30).all()), (name, float((off - bound).max()))


SHAPES = [
    # groups without rows, of one row, around the 16-row step and the 64-row block
    ([0, 1, 15, 16, 17, 0], 64, 64),
    ([63, 64, 65, 0, 2], 128, 256),
    # around the 256-row unit, several units, columns that are no multiple of any tile
    ([255, 256, 257, 1], 136, 72),
    ([600, 0, 513], 264, 520),
    # the smallest matrices
    ([3, 5], 8, 8),
    ([1], 16, 8),
    # the layer of the 2B configuration, uneven
    ([40, 0, 129, 300, 7], 1280, 896),
    # one dense block
    ([517], 512, 1024),
    # a long reduction over d, with enough rows and features for its larger units
    ([30] * 17 + [0, 300, 257, 1], 2056, 1032),
]
IDS = [("-".join(map(str, c)) if len(c) < 9 else f"{len(c)}groups") + f"_{d}x{F}" for c, d, F in SHAPES]


@pytest.mark.parametrize("counts,d,F", SHAPES, ids=IDS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_train_forward(counts, d, F, dtype):
    b = Block(counts, d, F, dtype, seed=1)
    y, gu = b.forward()
    ws = b.ws(False)
    plain = torch.empty_like(y)
    moe.experts(b.cfg, b.R, b.dcounts, b.x, b.gate, *b.weights(), plain, ws)
    for e, r in b.groups():
        x = b.x[r].double()
        g, u = x @ b.W1[e].double().T, x @ b.W3[e].double().T
        ref = b.gate[r].double()[:, None] * ((g * torch.sigmoid(g) * u) @ b.W2[e].double().T)
        if dtype == "f32":
            assert rel(gu[r], torch.cat([g, u], 1)) <= (d + 16) * 2.0 ** -23
            assert rel(y[r], ref) <= (d + F + 16) * 2.0 ** -23
        else:
            assert rel(gu[r], torch.cat([g, u], 1)) <= BF16_ONE
            assert rel(y[r], ref) <= BF16_TWO
    if dtype == "f32":
        # the same sums in another order, each within the bound above of the exact ones
        assert rel(y, plain.double()) <= 2 * (d + F + 16) * 2.0 ** -23
    else:
        assert rel(y, plain) <= 2 * BF16_TWO


@pytest.mark.parametrize("counts,d,F", SHAPES, ids=IDS)
@pytest.mark.parametrize("dtype,grad_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_experts_backward(counts, d, F, dtype, grad_dtype):
    b = Block(counts, d, F, dtype, seed=2)
    out = b.backward(grad_dtype)
    ref, mag = b.exact()
    check_block(b, out, ref, mag)
    for e, n in enumerate(counts):
        if n == 0:
            for name in ("dW1", "dW3", "dW2"):
                assert not out[name][e].any(), name


def test_experts_backward_in_tiles_that_fill_the_gpu():
    # fp32: 25 x 6 and more tiles of 128 x 128, ragged in every direction
    b = Block([2100, 0, 1, 900, 130], 776, 1000, "f32", seed=21)
    b.forward()
    check_block(b, b.backward(), *b.exact())
    # a workspace for these rows also holds a call of fewer
    small = Block([40, 7], 776, 1000, "f32", seed=22)
    assert (moe.experts_backward_workspace_size(small.cfg, 3000) <=
            moe.experts_backward_workspace_size(small.cfg, 3131))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_beyond_2_31_elements(dtype):
    """The last rows of a block whose gu and scratch rows lie past 2^31 elements; the first group's rows are zero."""
    R, tail, d, F = 530_000, 500, 64, 4104
    b = Block([1, tail], d, F, dtype, seed=31)
    b.forward()
    dt = DT[dtype]
    x, dy, y, dx = (torch.zeros((R, d), dtype=dt, device="cuda") for _ in range(4))
    gate, dgate = torch.ones(R, device="cuda"), torch.empty(R, device="cuda")
    x[-tail:], dy[-tail:], gate[-tail:] = b.x[1:], b.dy[1:], b.gate[1:]
    gu = torch.empty((R, 2 * F), dtype=dt, device="cuda")
    counts = torch.tensor([R - tail, tail], dtype=torch.int32, device="cuda")
    ws = torch.empty(max(moe.experts_workspace_size(b.cfg, R), moe.experts_backward_workspace_size(b.cfg, R)),
                     dtype=torch.uint8, device="cuda")
    moe.experts_train(b.cfg, R, counts, x, gate, *b.weights(), y, gu, ws)
    assert gu.numel() > 2 ** 32 and not gu[:R - tail].any() and not y[:R - tail].any()
    small_y, small_gu = b.forward()
    tol = BF16_TWO if dtype == "bf16" else 2 * (d + F + 16) * 2.0 ** -23  # two sums of the same terms, or a rounding
    assert rel(gu[-tail:], small_gu[1:].double()) <= tol and rel(y[-tail:], small_y[1:].double()) <= tol
    dW = [torch.empty_like(w) for w in b.weights()]
    moe.experts_backward(b.cfg, R, counts, x, gate, *b.weights(), gu, dy, dx, dgate, *dW, ws)
    assert moe.device_status(b.cfg, R, ws) == 0
    b.gu = torch.cat([small_gu[:1], gu[-tail:]])
    ref, mag = b.exact()
    out = dict(dx=dx[-tail:], dgate=dgate[-tail:], dW1=dW[0][1], dW3=dW[1][1], dW2=dW[2][1])
    part = lambda t: {n: v[1:] if v.shape[0] == tail + 1 else v[1] for n, v in t.items()}  # noqa: E731
    check_block(b, out, part(ref), part(mag))
    assert not dx[:R - tail].any() and not any(w[0].any() for w in dW)


def test_experts_backward_without_gates():
    b = Block([33, 0, 70], 136, 264, gate=False, seed=3)
    check_block(b, b.backward(), *b.exact())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_backward_accumulates(dtype):
    b = Block([33, 0, 300], 136, 264, dtype, seed=4)
    once = b.backward("f32")
    more = b.backward("f32", accumulate=True, start=0.75)
    for name in ("dW1", "dW3", "dW2"):
        assert torch.equal(more[name], once[name] + 0.75), name
    assert torch.equal(more["dx"], once["dx"]) and torch.equal(more["dgate"], once["dgate"])


@pytest.mark.parametrize("counts,d,F", [([20, 0, 33, 7, 1, 64], 1032, 776), ([400, 0, 17], 1032, 1288)],
                         ids=["kept", "streamed"])
def test_experts_backward_accumulates_over_runs_of_tiles(counts, d, F):
    b = Block(counts, d, F, "bf16", seed=23)
    b.forward()
    once = b.backward("f32")
    twice = b.backward("f32", accumulate=True, start=0.5)
    for n in ("dW1", "dW3", "dW2"):  # the old value is added to the sum, rounded once
        assert torch.equal(twice[n], once[n] + 0.5), n


def test_experts_backward_skips_what_is_not_asked_for():
    b = Block([33, 0, 70], 136, 264, seed=5)
    full = b.backward()
    ws = b.ws()
    args = (b.cfg, b.R, b.dcounts, b.x, b.gate, *b.weights(), b.gu, b.dy)
    dx = torch.empty_like(b.x)
    moe.experts_backward(*args, dx, None, None, None, None, ws)
    assert torch.equal(dx, full["dx"])
    dgate = torch.empty_like(b.gate)
    moe.experts_backward(*args, None, dgate, None, None, None, ws)
    assert torch.equal(dgate, full["dgate"])
    dW = [torch.empty_like(w) for w in b.weights()]
    moe.experts_backward(*args, None, None, *dW, ws)
    for t, name in zip(dW, ("dW1", "dW3", "dW2")):
        assert torch.equal(t, full[name]), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_backward_without_rows(dtype):
    b = Block([0, 0], 64, 32, dtype)
    for name, t in b.backward().items():
        if name.startswith("dW"):
            assert not t.any(), name
    for t in b.backward("f32", accumulate=True).values():
        assert bool((t == 3.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_backward_reports_counts_that_do_not_add_up(dtype):
    b = Block([10, 20], 64, 32, dtype)
    b.dcounts[1] = 21
    out = b.backward(expect=moe.MOE_DEV_BAD_EXPERT)
    for name in ("dW1", "dW3", "dW2"):
        assert not out[name].any(), name
    assert bool((out["dx"] == 3.0).all()) and bool((out["dgate"] == 3.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 15, 17, 63, 64, 100, 257])
def test_a_groups_rows_do_not_reach_its_neighbours(dtype, n):
    """NaN and infinite rows, gates and weights of one group leave every other group's results as they were."""
    counts = [n, 40, n]
    b = Block(counts, 136, 72, dtype, seed=6)
    clean = b.backward()
    r = slice(n, n + 40)
    for t in (b.x, b.dy, b.gu):
        t[r] = float("nan")
    b.dy[n + 3] = float("inf")
    b.gate[r] = float("nan")
    for w in b.weights():
        w[1] = float("inf")
    out = b.backward()
    for name in ("dW1", "dW3", "dW2"):
        assert torch.equal(out[name][0], clean[name][0]) and torch.equal(out[name][2], clean[name][2]), name
        assert not torch.isfinite(out[name][1]).all()
    for name in ("dx", "dgate"):
        assert torch.equal(out[name][:n], clean[name][:n]) and torch.equal(out[name][n + 40:], clean[name][n + 40:])


def test_extreme_pre_activations():
    """Saturated gates: sigmoid 0 and 1, and a zero gate, give finite gradients."""
    b = Block([40], 64, 64, seed=7)
    b.gu[:, :16] = 90.0
    b.gu[:, 16:32] = -90.0
    b.gu[:, 32:40] = -300.0
    b.gate[:5] = 0.0
    out = b.backward()
    check_block(b, out, *b.exact())
    assert not out["dx"][:5].any() and out["dgate"][:5].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_experts_backward_is_deterministic_and_takes_any_stream(dtype):
    b = Block([300, 0, 17, 130], 264, 520, dtype, seed=8)
    first = b.backward()
    side = torch.cuda.Stream()
    ws = b.ws()
    ws.fill_(255)  # whatever an earlier user left there
    second = b.backward(ws=ws, stream=side)
    for name in first:
        assert torch.equal(first[name], second[name]), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,d,F", [SHAPES[1], SHAPES[6], SHAPES[-1]], ids=[IDS[1], IDS[6], IDS[-1]])
def test_experts_do_not_read_what_the_workspace_held(counts, d, F, dtype):
    b = Block(counts, d, F, dtype, seed=41)
    clean, full = (torch.full((max(b.ws().numel(), b.ws(False).numel()),), fill, dtype=torch.uint8, device="cuda")
                   for fill in (0, 255))
    got = []
    for ws in (clean, full, full):
        y, gu = torch.empty_like(b.x), torch.empty_like(b.gu)
        moe.experts_train(b.cfg, b.R, b.dcounts, b.x, b.gate, *b.weights(), y, gu, ws)
        got.append(dict(b.backward(ws=ws), y=y, gu=gu))
        ws.fill_(255)
    for other in got[1:]:
        for name, t in got[0].items():
            assert torch.equal(t, other[name]), name


def test_experts_backward_in_a_graph():
    b = Block([300, 0, 17, 130], 264, 520, seed=9)
    want = b.backward()
    out = {k: torch.zeros_like(v) for k, v in want.items()}
    ws = b.ws()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.experts_backward(b.cfg, b.R, b.dcounts, b.x, b.gate, *b.weights(), b.gu, b.dy, *out.values(), ws)
    graph.replay()
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(out[name], want[name]), name
    # other values and other counts of the same total
    b.dy.mul_(0.5)
    b.counts = [17, 130, 300, 0]
    b.dcounts.copy_(torch.tensor(b.counts, dtype=torch.int32))
    want = b.backward()
    graph.replay()
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(out[name], want[name]), name


def test_experts_backward_against_differences():
    """fp32: the derivative of <dy, y> along a random direction of every
    input, from central differences of the 64-bit forward's formula at the
    gradient's own inputs. The difference quotient is off by O(eps^2) of the
    third derivative: at eps = 1e-5 about 1e-10 of these O(1) functions, far
    below the gradient's own fp32 error of (2 F + d) 2^-23 of its terms."""
    b = Block([9, 0, 20], 24, 16, "f32", seed=10)
    _, gu = b.forward()
    b.gu = gu
    out = b.backward()
    gen = torch.Generator().manual_seed(3)

    def loss(x, gate, W1, W3, W2):
        total = 0.0
        for e, r in b.groups():
            g, u = x[r] @ W1[e].T, x[r] @ W3[e].T
            total = total + (b.dy[r].double() * (gate[r][:, None] * ((g * torch.sigmoid(g) * u) @ W2[e].T))).sum()
        return float(total)

    inputs = [t.double() for t in (b.x, b.gate, *b.weights())]
    for i, name in enumerate(("dx", "dgate", "dW1", "dW3", "dW2")):
        v = torch.randn(inputs[i].shape, generator=gen, dtype=F64).cuda()
        eps = 1e-5
        up, down = list(inputs), list(inputs)
        up[i], down[i] = inputs[i] + eps * v, inputs[i] - eps * v
        want = (loss(*up) - loss(*down)) / (2 * eps)
        terms = out[name].double() * v
        assert abs(float(terms.sum()) - want) <= 1e-4 * float(terms.abs().sum()), name


# ---------------------------------------------------------------- router --


def route_case(T, N, k, d, score, normalize, dtype, seed=0, scale=2.5):
    gen = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    cfg = moe.make_cfg(d, 8, N, 0, k, score=score, normalize=normalize, route_scale=scale, dtype=dtype)
    logits = randn(gen, (T, N), 1.5)
    return dict(cfg=cfg, T=T, N=N, k=k, d=d, x=randn(gen, (T, d), 1.0, dt), W_r=randn(gen, (N, d), d ** -0.5, dt),
                logits=logits, idx=torch.topk(logits + 0.3 * randn(gen, (T, N)), k, dim=1).indices.to(torch.int32),
                dG=randn(gen, (T, k), 0.1), score=score, normalize=normalize, scale=scale, dtype=dtype)


def route_run(c, grad_dtype=None, accumulate=False, slot_pos=None, dG=None, start=3.0, expect=0):
    dx, c0 = guarded((c["T"], c["d"]), DT[c["dtype"]], start)
    dW, c1 = guarded((c["N"], c["d"]), DT[grad_dtype or c["dtype"]], start)
    ws = torch.full((moe.route_backward_workspace_size(c["cfg"], c["T"]),), 255, dtype=torch.uint8, device="cuda")
    moe.route_backward(c["cfg"], c["T"], c["x"], c["W_r"], c["logits"], c["idx"], c["dG"] if dG is None else dG,
                       slot_pos, dx, dW, ws, grad_dtype=grad_dtype, accumulate=accumulate)
    torch.cuda.synchronize()
    c0(), c1()
    assert moe.device_status(c["cfg"], c["T"], ws) == expect
    return dx, dW


def route_exact(c, dG=None):
    """By automatic differentiation of the gates in 64 bits."""
    z = c["logits"].double().requires_grad_()
    s = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
    sel = s.gather(1, c["idx"].long())
    gates = c["scale"] * (sel / sel.sum(1, keepdim=True) if c["normalize"] else sel)
    dz, = torch.autograd.grad(gates, z, (c["dG"] if dG is None else dG).double())
    return dz, dz @ c["W_r"].double(), dz.T @ c["x"].double()


def route_check(c, dx, dW, exact, dG=None):
    """Proof of the bounds: dz_j is s_j (1 - s_j) ds_j or s_j (ds_j - sum_i
    ds_i s_i), and a normalised ds_j is (c / Z) (dG_j - sum_i dG_i s_i / Z).
    Both differences cancel, so the fp32 error goes by the magnitude A_j of
    their terms and not by dz_j: each factor is good to a few units of 2^-24,
    a sum over the N scores (the softmax) or k slots to N + k, together
    (N + k + 16) 2^-23 A_j. The products then add (terms + 16) 2^-23 of the
    sum of the absolute terms. In bf16 layers dz is rounded to bf16 as an
    operand of the products: 2^-8 of itself (and the norm's bound applies)."""
    dz, rx, rW = exact
    z, idx, g = c["logits"].double(), c["idx"].long(), (c["dG"] if dG is None else dG).double().abs()
    s = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
    sel = s.gather(1, idx)
    Z = sel.sum(1, keepdim=True)
    ds = c["scale"] * (g / Z + (g * sel).sum(1, keepdim=True) / Z ** 2 if c["normalize"] else g)
    A = torch.zeros_like(s).scatter_(1, idx, ds) * s
    if c["score"] == "softmax":
        A = A + s * (ds * sel).sum(1, keepdim=True)
    err = (c["N"] + c["k"] + 16) * 2.0 ** -23 * A + (2.0 ** -8 if c["dtype"] == "bf16" else 0.0) * dz.abs()
    W, x = c["W_r"].double().abs(), c["x"].double().abs()
    ex = err @ W + (c["N"] + 16) * 2.0 ** -23 * (dz.abs() @ W)
    eW = err.T @ x + (c["T"] + 16) * 2.0 ** -23 * (dz.abs().T @ x)
    for y, r, e in ((dx, rx, ex), (dW, rW, eW)):
        bound = e + (2.0 ** -8 * (r.abs() + e) if y.dtype == torch.bfloat16 else 0.0)
        off = (y.double() - r).abs()
        assert bool((off <= bound + 1e-30).all()), float((off / (bound + 1e-30)).max())
        assert c["dtype"] == "f32" or float(torch.linalg.vector_norm(off)) <= (
            BF16_TWO * float(torch.linalg.vector_norm(r)) + float(torch.linalg.vector_norm(e)) * 2.0 ** -8)


ROUTES = [(1, 4, 2, 64), (7, 63, 7, 136), (300, 64, 16, 512), (1000, 100, 6, 264), (517, 256, 8, 1280),
          (64, 512, 16, 72), (2100, 16, 2, 256), (5, 2, 2, 8)]


@pytest.mark.parametrize("T,N,k,d", ROUTES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype,grad_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_route_backward(T, N, k, d, score, normalize, dtype, grad_dtype):
    c = route_case(T, N, k, d, score, normalize, dtype, seed=T + N)
    route_check(c, *route_run(c, grad_dtype), route_exact(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [40, 2100])
def test_route_backward_accumulates(dtype, T):
    c = route_case(T, 64, 4, 256, "sigmoid", True, dtype, seed=1)
    _, once = route_run(c, "f32")
    _, more = route_run(c, "f32", accumulate=True, start=0.5)
    assert torch.equal(more, once + 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_route_backward_takes_gradients_by_permuted_row(dtype):
    c = route_case(300, 20, 3, 136, "softmax", False, dtype, seed=2)
    cfg, T, k, dt = c["cfg"], c["T"], c["k"], DT[dtype]
    ws = torch.empty(moe.workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets, slot_pos = torch.empty(20, **i32), torch.empty(21, **i32), torch.empty((T, k), **i32)
    # the dispatch carries the gates to the rows: use it to carry the gradients
    rows, dG_rows = torch.empty((T * k, c["d"]), dtype=dt, device="cuda"), torch.empty(T * k, device="cuda")
    moe.dispatch_rows(cfg, T, c["idx"], c["dG"], c["x"], counts, offsets, slot_pos, rows, dG_rows, ws)
    want, got = route_run(c), route_run(c, slot_pos=slot_pos, dG=dG_rows)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_route_backward_ignores_and_reports_invalid_experts():
    c = route_case(50, 16, 4, 64, "softmax", False, "f32", seed=3)
    good = route_run(c)
    # drop one slot of token 7: the same as a zero gradient there
    dG = c["dG"].clone()
    dG[7, 2] = 0.0
    want = route_run(c, dG=dG)
    for bad in (-1, 16):
        c["idx"][7, 2] = bad
        got = route_run(c, expect=moe.MOE_DEV_BAD_EXPERT)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not torch.equal(good[0], want[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_route_backward_without_tokens(dtype):
    c = route_case(0, 16, 4, 64, "softmax", False, dtype)
    dW = torch.full((16, 64), 3.0, dtype=DT[dtype], device="cuda")
    moe.route_backward(c["cfg"], 0, None, None, None, None, None, None, None, dW, None, ws_bytes=0)
    assert not dW.any()


def test_route_backward_skips_what_is_not_asked_for():
    c = route_case(300, 64, 4, 136, "sigmoid", True, "bf16", seed=5)
    dx, dW = route_run(c)
    ws = torch.empty(moe.route_backward_workspace_size(c["cfg"], 300), dtype=torch.uint8, device="cuda")
    for which in (0, 1):
        got = torch.empty_like((dx, dW)[which])
        outs = [None, None]
        outs[which] = got
        moe.route_backward(c["cfg"], 300, c["x"], c["W_r"], c["logits"], c["idx"], c["dG"], None, *outs, ws)
        assert torch.equal(got, (dx, dW)[which])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 130, 1030])
def test_route_train_keeps_the_logits(dtype, T):
    gen = torch.Generator().manual_seed(4)
    dt, d, N, k = DT[dtype], 1280, 63, 7
    cfg = moe.make_cfg(d, 8, N, 0, k, score="softmax", dtype=dtype)
    x, W_r = randn(gen, (T, d), 1.0, dt), randn(gen, (N, d), d ** -0.5, dt)
    ws = torch.empty(moe.workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    res = []
    for train in (False, True):
        idx, gates = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
        logits, check = guarded((T, N), torch.float32)
        if train:
            moe.route_train(cfg, T, x, W_r, None, idx, gates, logits, ws)
        else:
            moe.route(cfg, T, x, W_r, None, idx, gates, ws)
        torch.cuda.synchronize()
        check()
        res.append((idx, gates))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    z = x.double() @ W_r.double().T
    bound = (d + 16) * 2.0 ** -23 * (x.double().abs() @ W_r.double().abs().T)
    assert bool(((logits.double() - z).abs() <= bound).all())


# --------------------------------------------------------------- clipping --


def clip(srcs, max_norm, dsts=None, stream=None):
    g = moe.GradList(srcs, dsts)
    ws = torch.full((moe.grad_norm_workspace_size(g),), 255, dtype=torch.uint8, device="cuda")
    sumsq = torch.full((1,), -1.0, dtype=F64, device="cuda")
    norm = torch.full((1,), -1.0, device="cuda")
    torch.cuda.synchronize()
    moe.grad_norm(g, sumsq, ws, stream=stream)
    moe.grad_clip(g, sumsq, max_norm, norm, stream=stream)
    torch.cuda.synchronize()
    return float(sumsq), float(norm)


def exact_norm(srcs):
    return math.sqrt(sum(float(t.double().square().sum()) for t in srcs))


def check_clip(srcs, dsts, before, norm, max_norm):
    want = exact_norm(before)
    # up to 32 squares are summed in fp32: up to 32 * 2^-24 = 2^-19 relative, halved by the root
    assert abs(norm - want) <= 2.0 ** -20 * want
    c = min(1.0, max_norm / want) if want > 0 and math.isfinite(want) else 1.0
    for s, d, b in zip(srcs, dsts, before):
        eps = 2.0 ** -8 if b.dtype == torch.bfloat16 else 2.0 ** -23
        assert bool(((d.double() - b.double() * c).abs() <= (eps + 2.0 ** -20) * (b.double() * c).abs() + 1e-44).all())
        if s is not d:
            assert torch.equal(s, b)


@pytest.mark.parametrize("sizes", [[1], [7, 0, 9], [1000, 1, 33], [40000, 16384, 16385, 2], [1 << 20, 12345],
                                   list(range(1, 80)), [513] * 700], ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ratio", [0.3, 2.0])
@pytest.mark.parametrize("inplace", [False, True])
def test_clip(sizes, dtype, ratio, inplace):
    gen = torch.Generator().manual_seed(len(sizes))
    srcs = [randn(gen, (n,), 0.01, DT[dtype]) for n in sizes]
    before = [t.clone() for t in srcs]
    dsts = srcs if inplace else [torch.full_like(t, 5.0) for t in srcs]
    max_norm = ratio * exact_norm(before)
    _, norm = clip(srcs, max_norm, None if inplace else dsts)
    check_clip(srcs, dsts, before, norm, max_norm)
    if ratio > 1:
        for d, b in zip(dsts, before):
            assert torch.equal(d, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_clip_at_odd_offsets(dtype, shift):
    """Views of one bucket at every alignment, and destinations aligned otherwise; nothing around them changes."""
    gen = torch.Generator().manual_seed(5)
    sizes = [1, 2, 3, 5, 17, 1001, 33000, 7]
    src = randn(gen, (sum(sizes) + 2 * len(sizes),), 0.01, DT[dtype])
    dst = torch.full((src.numel() + shift,), 5.0, dtype=DT[dtype], device="cuda")
    srcs, dsts, at, used = [], [], 0, torch.zeros(dst.numel(), dtype=torch.bool, device="cuda")
    for n in sizes:
        srcs.append(src[at:at + n])
        dsts.append(dst[at + shift:at + shift + n])
        used[at + shift:at + shift + n] = True
        at += n + 2
    before = [t.clone() for t in srcs]
    max_norm = 0.5 * exact_norm(before)
    _, norm = clip(srcs, max_norm, dsts)
    check_clip(srcs, dsts, before, norm, max_norm)
    assert bool((dst[~used] == 5.0).all())


@pytest.mark.parametrize("n", [1000, 1 << 20, 1 << 26])
def test_clip_reads_the_sum_of_its_own_norm(n):
    """The clip's launch overlaps the norm's end: it must not read what the sum's buffer held before."""
    t = torch.full((n,), 2.0 ** -10, device="cuda")
    grads = moe.GradList([t], [torch.empty_like(t)])
    ws = torch.empty(moe.grad_norm_workspace_size(grads), dtype=torch.uint8, device="cuda")
    want = 2.0 ** -10 * n ** 0.5
    for old in (float("nan"), 0.0, 1e30):
        sumsq = torch.full((1,), old, dtype=torch.float64, device="cuda")
        norm = torch.empty(1, device="cuda")
        ws.fill_(255)
        torch.cuda.synchronize()
        moe.grad_norm(grads, sumsq, ws)
        moe.grad_clip(grads, sumsq, want / 4, norm)
        assert abs(float(norm) - want) <= 2.0 ** -20 * want, old
        assert bool(((grads.dsts[0] - 2.0 ** -12).abs() <= 2.0 ** -30).all()), old


def test_clip_mixes_types_and_is_deterministic():
    gen = torch.Generator().manual_seed(6)
    srcs = [randn(gen, (n,), 0.01, dt) for n in (70001, 5, 300000) for dt in (torch.float32, torch.bfloat16)]
    a = clip(srcs, 1e9)
    b = clip(srcs, 1e9, stream=torch.cuda.Stream())
    assert a == b
    assert abs(a[1] - exact_norm(srcs)) <= 2.0 ** -20 * a[1]


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e18, 1e25])
def test_norm_over_the_whole_range(scale):
    gen = torch.Generator().manual_seed(7)
    t = randn(gen, (5003,), 1.0) * scale
    before = t.clone()
    want = exact_norm([t])
    sumsq, norm = clip([t], 0.5 * want)
    assert abs(math.sqrt(sumsq) - want) <= 2.0 ** -20 * want
    assert bool(((t.double() - 0.5 * before.double()).abs() <= 2.0 ** -19 * before.double().abs()).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(bad):
    for dtype in DT.values():
        t = torch.ones(1000, dtype=dtype, device="cuda")
        t[777] = bad
        out = torch.zeros_like(t)
        _, norm = clip([t], 0.1, [out])
        assert not math.isfinite(norm)
        assert torch.equal(torch.nan_to_num(out, 9.0, 9.0, 9.0), torch.nan_to_num(t, 9.0, 9.0, 9.0))


def test_clip_at_its_limits():
    t = torch.full((100,), 2.0, device="cuda")
    assert clip([t], 20.0)[1] == 20.0 and bool((t == 2.0).all())  # at the limit: as it is
    assert clip([t], math.inf)[1] == 20.0 and bool((t == 2.0).all())
    assert clip([t], 0.0)[1] == 20.0 and not t.any()
    assert clip([t], 0.0)[1] == 0.0 and not t.any()               # a zero norm is within a zero limit
    assert clip([], 1.0) == (0.0, 0.0)
    assert clip([torch.empty(0, device="cuda")], 1.0) == (0.0, 0.0)


def test_clip_of_more_than_2_31_elements():
    n = (1 << 31) + 37
    t = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    want = 2.0 ** -10 * math.sqrt(n)
    _, norm = clip([t], want / 4)
    assert abs(norm - want) <= 2.0 ** -20 * want
    lo, hi = torch.aminmax(t)
    assert float(lo) == float(hi) == 2.0 ** -12


def test_clip_in_a_graph():
    gen = torch.Generator().manual_seed(8)
    srcs = [randn(gen, (n,), 0.01) for n in (5000, 3, 70000)]
    dsts = [torch.zeros_like(t) for t in srcs]
    g = moe.GradList(srcs, dsts)
    ws = torch.empty(moe.grad_norm_workspace_size(g), dtype=torch.uint8, device="cuda")
    sumsq, norm = torch.zeros(1, dtype=F64, device="cuda"), torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.grad_norm(g, sumsq, ws)
        moe.grad_clip(g, sumsq, 0.1, norm)
    del g  # the graph keeps its own table
    for scale in (1.0, 3.0):
        for t in srcs:
            t.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        check_clip(srcs, dsts, [t.clone() for t in srcs], float(norm), 0.1)


# ------------------------------------------------------------- a whole step --


def layer_case(T, d, F, N, ns, k, score, normalize, dtype, seed=0, bias=True):
    gen = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    cfg = moe.make_cfg(d, F, N, ns, k, score=score, normalize=normalize, route_scale=2.5, dtype=dtype)
    w = {"W_r": randn(gen, (N, d), d ** -0.5, dt), "b": randn(gen, (N,), 0.01) if bias else None,
         "W1": randn(gen, (N, F, d), d ** -0.5, dt), "W3": randn(gen, (N, F, d), d ** -0.5, dt),
         "W2": randn(gen, (N, d, F), F ** -0.5, dt)}
    if ns:
        w |= {"Ws1": randn(gen, (ns * F, d), d ** -0.5, dt), "Ws3": randn(gen, (ns * F, d), d ** -0.5, dt),
              "Ws2": randn(gen, (d, ns * F), (ns * F) ** -0.5, dt)}
    return cfg, w, randn(gen, (T, d), 1.0, dt), randn(gen, (T, d), 1.0, dt)


def layer_exact(cfg, w, x, dy, idx, score, normalize):
    """y and the gradients by automatic differentiation in 64 bits, with the given selection."""
    p = {n: t.double().requires_grad_() for n, t in w.items() if n != "b" and t is not None}
    x = x.double().requires_grad_()
    z = x @ p["W_r"].T
    s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
    sel = s.gather(1, idx.long())
    gates = 2.5 * (sel / sel.sum(1, keepdim=True) if normalize else sel)
    y = torch.zeros_like(x)
    for e in range(cfg.n_routed):
        t, slot = torch.nonzero(idx == e, as_tuple=True)
        if t.numel():
            g, u = x[t] @ p["W1"][e].T, x[t] @ p["W3"][e].T
            y = y.index_add(0, t, gates[t, slot][:, None] * ((torch.nn.functional.silu(g) * u) @ p["W2"][e].T))
    if "Ws1" in p:
        g, u = x @ p["Ws1"].T, x @ p["Ws3"].T
        y = y + (torch.nn.functional.silu(g) * u) @ p["Ws2"].T
    names = list(p)
    grads = torch.autograd.grad(y, [x] + [p[n] for n in names], dy.double())
    return y, grads[0], dict(zip(names, grads[1:]))


# The whole step rounds g, u, h, the gated rows and y in the forward (bf16);
# backward dg, du, gate h, the rows of dx and the sums. A gradient is reached
# by at most six roundings in a chain (g or u, dg or du, a row, the result,
# and through the gate h and y_row), each at most 2^-8 relative, of
# independent signs across terms: 6 * 2^-8.
LAYER_TOL = {"bf16": 6 * 2.0 ** -8, "f32": 2e-5}


@pytest.mark.parametrize("T,d,F,N,ns,k,score,normalize,dtype", [
    (300, 256, 128, 16, 1, 4, "sigmoid", True, "bf16"),
    (517, 136, 264, 10, 2, 3, "softmax", False, "bf16"),
    (1, 64, 64, 8, 1, 2, "sigmoid", True, "bf16"),
    (77, 136, 200, 12, 1, 3, "sigmoid", True, "f32"),
    (256, 256, 512, 16, 0, 2, "softmax", False, "f32"),
])
def test_training_step(T, d, F, N, ns, k, score, normalize, dtype):
    cfg, w, x, dy = layer_case(T, d, F, N, ns, k, score, normalize, dtype, seed=T)
    layer = TrainLayer(cfg, w, max_tokens=T, grad_dtype="f32")
    y = layer.forward(x)
    dx = layer.backward(dy)
    ry, rx, rg = layer_exact(cfg, w, x, dy, layer.saved["idx"], score, normalize)
    tol = LAYER_TOL[dtype]
    assert rel(y, ry) <= tol and rel(dx, rx) <= tol, (rel(y, ry), rel(dx, rx))
    for n, t in layer.grads.items():
        assert rel(t, rg[n]) <= tol, (n, rel(t, rg[n]))
    # a second micro-batch on top: twice the gradients, to the last bit
    once = {n: t.clone() for n, t in layer.grads.items()}
    layer.forward(x)
    layer.backward(dy, accumulate=True)
    for n, t in layer.grads.items():
        assert torch.equal(t, 2 * once[n]), n
    want = exact_norm(layer.grads.values())
    before = {n: t.clone() for n, t in layer.grads.items()}
    norm = layer.clip(0.25 * want)
    assert abs(float(norm) - want) <= 2.0 ** -20 * want
    for n, t in layer.grads.items():
        assert bool(((t - 0.25 * before[n]).abs() <= 2.0 ** -19 * before[n].abs()).all()), n
    if w["b"] is not None:
        b = w["b"].clone()
        layer.balance(1e-3)
        mean = T * k / N
        want_b = torch.where(layer.saved["counts"] > mean, b - 1e-3, torch.where(layer.saved["counts"] < mean, b + 1e-3, b))
        assert torch.equal(w["b"], want_b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_step_without_tokens(dtype):
    cfg, w, x, dy = layer_case(6, 64, 64, 8, 1, 2, "sigmoid", True, dtype)
    layer = TrainLayer(cfg, w, max_tokens=6)
    b = w["b"].clone()
    y, dx = layer.forward(x[:0]), layer.backward(dy[:0])
    assert y.shape == dx.shape == (0, 64)
    for n, t in layer.grads.items():
        assert not t.any(), n
    assert float(layer.clip(1.0)) == 0.0
    layer.balance(1e-3)
    assert torch.equal(b, w["b"]) and layer.device_status() == 0


def test_training_steps_on_two_streams_at_once():
    """Two layers, each on a stream of its own, a dozen steps in flight: each step's results are those it has alone."""
    cases = [layer_case(300, 256, 384, 16, 1, 4, "sigmoid", True, dt, seed=i) for i, dt in enumerate(("bf16", "f32"))]
    layers = [TrainLayer(c, w, max_tokens=300) for c, w, _, _ in cases]
    alone = []
    for layer, (_, _, x, dy) in zip(layers, cases):
        alone.append([layer.forward(x), layer.backward(dy), {n: t.clone() for n, t in layer.grads.items()}])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [None, None]
    for _ in range(6):
        for i, (layer, (_, _, x, dy)) in enumerate(zip(layers, cases)):
            with torch.cuda.stream(streams[i]):
                got[i] = [layer.forward(x), layer.backward(dy)]
    torch.cuda.synchronize()
    for i, layer in enumerate(layers):
        assert torch.equal(got[i][0], alone[i][0]) and torch.equal(got[i][1], alone[i][1])
        for n, t in layer.grads.items():
            assert torch.equal(t, alone[i][2][n]), n
        assert layer.device_status() == 0


@pytest.mark.parametrize("handle", [False, True])
def test_training_step_on_a_stream_that_is_not_current(handle):
    """Buffers of a step on another stream are not handed to the current stream's work while it runs."""
    cfg, w, x, dy = layer_case(400, 256, 384, 16, 1, 4, "sigmoid", True, "bf16", seed=3)
    alone = TrainLayer(cfg, w, max_tokens=400)
    want = alone.forward(x), alone.backward(dy)
    layer, side = TrainLayer(cfg, w, max_tokens=400), torch.cuda.Stream()
    arg = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    for _ in range(8):
        y = layer.forward(x, stream=arg)
        dx = layer.backward(dy, stream=arg)
        norm = layer.clip(1e9, stream=arg)
        for _ in range(40):  # the current stream overwrites whatever the allocator gives it
            torch.full((400 * 4, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
    assert torch.equal(norm, alone.clip(1e9))
    for n, t in layer.grads.items():
        assert torch.equal(t, alone.grads[n]), n


def test_training_step_on_the_default_streams_handle():
    cfg, w, x, dy = layer_case(40, 64, 64, 8, 1, 2, "sigmoid", True, "bf16", seed=4)
    layer, other = TrainLayer(cfg, w, max_tokens=40), TrainLayer(cfg, w, max_tokens=40)
    want = other.forward(x), other.backward(dy)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = layer.forward(x, stream=0), layer.backward(dy, stream=0)
        bits = layer.device_status(stream=0)
    torch.cuda.synchronize()
    assert bits == 0 and all(torch.equal(a, b) for a, b in zip(want, got))


def test_training_step_keeps_the_status_of_its_calls():
    cfg, w, x, dy = layer_case(40, 64, 64, 8, 0, 2, "sigmoid", True, "bf16")
    layer = TrainLayer(cfg, w, max_tokens=40)
    layer.forward(x), layer.backward(dy)
    assert layer.device_status() == 0
    x[3, 5] = float("nan")
    layer.forward(x)
    assert layer.device_status() & 16  # a token's logits were not finite
    assert layer.device_status() == 0


def test_training_step_in_a_graph():
    """A step captured once and replayed on new tokens gives an eager step's results."""
    cfg, w, x, dy = layer_case(200, 256, 128, 16, 1, 4, "sigmoid", True, "bf16", seed=1)
    layer = TrainLayer(cfg, w, max_tokens=200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x), layer.backward(dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = layer.forward(x)
        dx = layer.backward(dy)
        norm = layer.clip(1e-3)
    eager = TrainLayer(cfg, w, max_tokens=200)
    for seed in (2, 3):
        _, _, x2, dy2 = layer_case(200, 256, 128, 16, 1, 4, "sigmoid", True, "bf16", seed=seed)
        x.copy_(x2), dy.copy_(dy2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager.forward(x2)) and torch.equal(dx, eager.backward(dy2))
        assert torch.equal(norm, eager.clip(1e-3))
        for n in layer.grads:
            assert torch.equal(layer.grads[n], eager.grads[n]), n


def test_two_graphs_of_fp32_steps_share_a_layer():
    """Two captures of one layer's step, of different token counts, replayed in turn on one workspace."""
    cfg, w, x, dy = layer_case(600, 136, 264, 12, 1, 3, "softmax", False, "f32", seed=5)
    layer, eager = (TrainLayer(cfg, w, max_tokens=600) for _ in range(2))
    side = torch.cuda.Stream()
    layer.forward(x), layer.backward(dy)
    torch.cuda.synchronize()
    graphs = []
    for T in (600, 37):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = layer.forward(x[:T])
            dx = layer.backward(dy[:T], accumulate=True)
        graphs.append((T, graph, y, dx))
    for g in (*layer.grads.values(), *eager.grads.values()):
        g.zero_()
    for T, graph, y, dx in graphs + graphs[::-1]:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager.forward(x[:T])) and torch.equal(dx, eager.backward(dy[:T], accumulate=True))
    for n in layer.grads:
        assert torch.equal(layer.grads[n], eager.grads[n]), n
    assert layer.device_status() == 0


def test_combine_and_dispatch_backward_are_each_others_transpose():
    """<dispatch_backward(rows), v> = <rows, combine_backward(v)> exactly on small whole numbers, with
    dropped pairs (an invalid expert) left out of both."""
    T, N, k, d = 50, 6, 2, 64
    gen = torch.Generator().manual_seed(2)
    cfg = moe.make_cfg(d, 8, N, 0, k, dtype="f32")
    idx = torch.stack([torch.randperm(N, generator=gen)[:k] for _ in range(T)]).to(torch.int32).cuda()
    idx[3, 1] = -1
    ws = torch.empty(moe.workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets, pos = torch.empty(N, **i32), torch.empty(N + 1, **i32), torch.empty((T, k), **i32)
    x = torch.randint(-8, 9, (T, d), generator=gen).float().cuda()
    rows, gate = torch.zeros((T * k, d), device="cuda"), torch.zeros(T * k, device="cuda")
    moe.dispatch_rows(cfg, T, idx, torch.ones((T, k), device="cuda"), x, counts, offsets, pos, rows, gate, ws)
    v_rows = torch.full((T * k, d), 0.0, device="cuda")
    moe.combine_backward(cfg, T, x, pos, v_rows)
    assert torch.equal(v_rows, rows)
    r = torch.randint(-8, 9, (T * k, d), generator=gen).float().cuda()
    a, b2 = (torch.randint(-8, 9, (T, d), generator=gen).float().cuda() for _ in range(2))
    out = torch.empty_like(x)
    moe.dispatch_backward(cfg, T, r, pos, None, None, out)
    assert float((out * x).sum()) == float((r * v_rows).sum())
    for sh, ro in ((a, None), (None, b2), (a, b2)):
        more = torch.empty_like(x)
        moe.dispatch_backward(cfg, T, r, pos, sh, ro, more)
        assert torch.equal(more, out + (0 if sh is None else sh) + (0 if ro is None else ro))


@pytest.mark.parametrize("counts,d,F", SHAPES[:5] + SHAPES[-1:], ids=IDS[:5] + IDS[-1:])
def test_debug_build_finds_no_index_out_of_bounds(counts, d, F):
    b = Block(counts, d, F, seed=11)
    y, gu = b.forward()
    want = b.backward()
    with moe.using_library(moe.DEBUG_LIB_PATH):
        y2, gu2 = b.forward()
        got = b.backward()
    assert torch.equal(y, y2) and torch.equal(gu, gu2)
    for name in want:
        assert torch.equal(want[name], got[name]), name
