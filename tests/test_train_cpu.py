"""Host-side checks of the training entry points that need no GPU: sizes,
refusals (every one before any device work) and the binding's tables."""
import ctypes
import math

import pytest
import torch

import mixture_experts_layer_group_b200 as moe
from mixture_experts_layer_group_b200 import build as moe_build
from mixture_experts_layer_group_b200.train import TrainLayer

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
A = 1 << 20  # an aligned address that is never touched: every call below is refused first


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe_build.build()


def cfg(**kw):
    base = dict(d=64, d_ff=32, n_routed=8, n_shared=0, top_k=2)
    base.update(kw)
    return moe.make_cfg(**base)


def status(call, *args, **kw):
    with pytest.raises(moe.MoeError) as e:
        call(*args, **kw)
    return e.value.status


def backward(c=None, rows=4, stream=0, ws_bytes=1 << 30, **kw):
    a = dict(counts=A, x=A, gate=A, W1=A, W3=A, W2=A, gu=A, dy=A, dx=A, dgate=A, dW1=A, dW3=A, dW2=A, ws=A)
    opt = {k: kw.pop(k) for k in ("grad_dtype", "accumulate") if k in kw}
    a.update(kw)
    return status(moe.experts_backward, c or cfg(), rows, *a.values(), ws_bytes=ws_bytes, stream=stream, **opt)


@pytest.mark.parametrize("name", ["counts", "x", "W1", "W3", "W2", "gu", "dy"])
def test_experts_backward_needs_its_inputs(name):
    assert backward(**{name: None}) == INVALID
    assert backward(**{name: A + 2}) == INVALID


@pytest.mark.parametrize("name", ["dx", "dW1", "dW3", "dW2"])
def test_experts_backward_refuses_misaligned_outputs(name):
    assert backward(**{name: A + 8}) == INVALID


@pytest.mark.parametrize("name", ["dW1", "dW3", "dW2"])
def test_weight_gradients_come_together(name):
    assert backward(**{name: None}) == INVALID


def test_experts_backward_refuses_types_sizes_and_workspaces():
    assert backward(gate=A + 2) == INVALID
    assert backward(dgate=A + 1) == INVALID
    assert backward(accumulate=True) == UNSUPPORTED            # bf16 gradients
    assert backward(cfg(dtype="f32"), grad_dtype="bf16") == INVALID
    assert backward(rows=-1) == INVALID
    assert backward(cfg(d=60)) == INVALID
    assert backward(cfg(n_routed=513)) == UNSUPPORTED
    assert backward(ws=None) == WORKSPACE
    assert backward(ws=A + 128) == WORKSPACE
    assert backward(ws_bytes=moe.experts_backward_workspace_size(cfg(), 4) - 1) == WORKSPACE
    with pytest.raises(ValueError):
        backward(grad_dtype="fp16")


def test_experts_backward_without_rows_or_gradients_is_a_no_op():
    moe.experts_backward(cfg(), 0, None, None, None, None, None, None, None, None, None, None, None, None, None, None,
                         ws_bytes=0, stream=0)
    moe.experts_backward(cfg(), 0, None, None, None, None, None, None, None, None, None, None, A, A, A, None,
                         grad_dtype="f32", accumulate=True, ws_bytes=0, stream=0)


def test_experts_train_needs_a_buffer_for_the_pre_activations():
    for gu in (None, A + 8):
        assert status(moe.experts_train, cfg(), 4, A, A, A, A, A, A, A, gu, A, ws_bytes=1 << 30, stream=0) == INVALID


def test_workspaces_cover_the_scratch():
    c = cfg(d=512, d_ff=256, n_routed=4)
    rows = 1000
    assert moe.experts_backward_workspace_size(c, rows) >= 3 * rows * 256 * 2 + rows * 8 * 4
    assert moe.experts_backward_workspace_size(c, 2 * rows) > moe.experts_backward_workspace_size(c, rows)
    r = cfg(d=512, n_routed=63)
    assert moe.route_backward_workspace_size(r, rows) >= 2 * rows * 64 * 2
    assert moe.grad_norm_workspace_size(0) > 0
    assert moe.grad_norm_workspace_size(2000) > moe.grad_norm_workspace_size(500)
    n = ctypes.c_size_t()
    assert moe.lib().moe_grad_norm_workspace_size(-1, ctypes.byref(n)) == INVALID
    assert moe.lib().moe_grad_norm_workspace_size(1, None) == INVALID


def route_bwd(c=None, T=4, ws_bytes=1 << 30, **kw):
    a = dict(x=A, W_r=A, logits=A, idx=A, dgates=A, slot_pos=A, dx=A, dW_r=A, ws=A)
    opt = {k: kw.pop(k) for k in ("grad_dtype", "accumulate") if k in kw}
    a.update(kw)
    return status(moe.route_backward, c or cfg(), T, *a.values(), ws_bytes=ws_bytes, stream=0, **opt)


def test_route_backward_refusals():
    for name in ("x", "W_r", "logits", "idx", "dgates"):
        assert route_bwd(**{name: None}) == INVALID, name
        assert route_bwd(**{name: A + 2}) == INVALID, name
    assert route_bwd(slot_pos=A + 2) == INVALID
    assert route_bwd(dx=A + 8) == INVALID
    assert route_bwd(dW_r=A + 8) == INVALID
    assert route_bwd(ws=None) == WORKSPACE
    assert route_bwd(ws_bytes=moe.route_backward_workspace_size(cfg(), 4) - 1) == WORKSPACE
    assert route_bwd(T=-1) == INVALID
    assert route_bwd(accumulate=True) == UNSUPPORTED
    assert route_bwd(cfg(dtype="f32"), grad_dtype="bf16") == INVALID
    for logits in (None, A + 2):
        assert status(moe.route_train, cfg(), 4, A, A, None, A, A, logits, A, ws_bytes=1 << 30, stream=0) == INVALID


def test_combine_and_dispatch_backward_refusals():
    c = cfg()
    for i in range(3):
        args = [A, A, A]
        args[i] = None
        assert status(moe.combine_backward, c, 4, *args, stream=0) == INVALID
        args[i] = A + 2
        assert status(moe.combine_backward, c, 4, *args, stream=0) == INVALID
    for i in (0, 1, 4):
        args = [A, A, None, None, A]
        args[i] = None
        assert status(moe.dispatch_backward, c, 4, *args, stream=0) == INVALID
    for i in range(5):
        args = [A] * 5
        args[i] = A + 2
        assert status(moe.dispatch_backward, c, 4, *args, stream=0) == INVALID
    moe.combine_backward(c, 0, None, None, None, stream=0)
    moe.dispatch_backward(c, 0, None, None, None, None, None, stream=0)


def test_grad_list_checks_its_tensors():
    x = torch.zeros(4, 6)
    g = moe.GradList([x, x.bfloat16()])
    assert len(g) == 2 and g.table[0].numel == 24 and g.table[0].src == g.table[0].dst == x.data_ptr()
    assert (g.table[0].dtype, g.table[1].dtype) == (moe.MOE_F32, moe.MOE_BF16)
    for bad in (dict(srcs=[x.double()]), dict(srcs=[x.half()]), dict(srcs=[x.t()]), dict(srcs=[x], dsts=[x.bfloat16()]),
                dict(srcs=[x], dsts=[]), dict(srcs=[x], dsts=[torch.zeros(23)]), dict(srcs=[x], dsts=[x.t()])):
        with pytest.raises(ValueError):
            moe.GradList(**bad)


def test_grad_calls_refuse_bad_tables_and_limits():
    L = moe.lib()

    def entry(src=A, dst=A, numel=4, dtype=moe.MOE_F32):
        return (moe.GradTensor * 1)(moe.GradTensor(src, dst, numel, dtype, 0))

    for bad in (entry(src=None), entry(src=A + 2), entry(dst=A + 2), entry(numel=-1), entry(dtype=7),
                entry(src=A + 1, dtype=moe.MOE_BF16)):
        assert L.moe_grad_norm(bad, 1, A, A, 1 << 30, None) == INVALID
        assert L.moe_grad_clip(bad, 1, A, 1.0, None, None) == INVALID
    assert L.moe_grad_norm(None, 1, A, A, 1 << 30, None) == INVALID
    assert L.moe_grad_norm(entry(), -1, A, A, 1 << 30, None) == INVALID
    assert L.moe_grad_norm(entry(), 1, None, A, 1 << 30, None) == INVALID
    assert L.moe_grad_norm(entry(), 1, A + 4, A, 1 << 30, None) == INVALID
    assert L.moe_grad_norm(entry(), 1, A, None, 1 << 30, None) == WORKSPACE
    assert L.moe_grad_norm(entry(), 1, A, A, moe.grad_norm_workspace_size(1) - 1, None) == WORKSPACE
    for limit in (-1.0, math.nan, -math.inf):
        assert L.moe_grad_clip(entry(), 1, A, limit, None, None) == INVALID
    assert L.moe_grad_clip(entry(), 1, None, 1.0, None, None) == INVALID
    assert L.moe_grad_clip(entry(), 1, A, 1.0, A + 2, None) == INVALID


def test_grad_tensor_matches_header():
    assert ctypes.sizeof(moe.GradTensor) == 32
    assert [n for n, _ in moe.GradTensor._fields_] == ["src", "dst", "numel", "dtype", "reserved"]


def train_layer(**kw):
    c = cfg(n_shared=1)
    w = dict(W_r=torch.zeros(8, 64), W1=torch.zeros(8, 32, 64), W3=torch.zeros(8, 32, 64), W2=torch.zeros(8, 64, 32),
             Ws1=torch.zeros(32, 64), Ws3=torch.zeros(32, 64), Ws2=torch.zeros(64, 32))
    w = {n: t.to(torch.bfloat16) for n, t in w.items()}
    w.update(kw.pop("weights", {}))
    return TrainLayer(c, w, max_tokens=4, device="cpu", **kw)


def test_train_layer_refuses_weights_it_cannot_take():
    train_layer()
    for name, bad in (("W1", torch.zeros(8, 64, 32, dtype=torch.bfloat16)), ("W2", torch.zeros(8, 64, 32)),
                      ("Ws1", torch.zeros(64, 32, dtype=torch.bfloat16).T)):
        with pytest.raises(ValueError, match=name):
            train_layer(weights={name: bad})
    with pytest.raises(ValueError, match="gradients"):
        train_layer(grad_dtype="f16")


@pytest.mark.parametrize("bad", [
    torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(4, 64), torch.zeros(64, 4, dtype=torch.bfloat16).T,
    torch.zeros(1, 64, dtype=torch.bfloat16).expand(4, 64), torch.zeros(2, 2, 64, dtype=torch.bfloat16)])
def test_train_layer_refuses_rows_it_cannot_read(bad):
    layer = train_layer()
    with pytest.raises(ValueError, match="x is"):
        layer.forward(bad)
    layer.saved = dict(x=torch.zeros(tuple(bad.shape), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dy is"):
        layer.backward(bad)


def test_train_layer_steps_come_in_order():
    layer = train_layer()
    with pytest.raises(ValueError, match="max_tokens"):
        layer.forward(torch.zeros(5, 64, dtype=torch.bfloat16))
    for call in (lambda: layer.backward(torch.zeros(4, 64, dtype=torch.bfloat16)), lambda: layer.balance(1e-3)):
        with pytest.raises(RuntimeError):
            call()
    layer.saved = dict(x=torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="bias"):
        layer.balance(1e-3)


def test_grad_lists_refuse_overlapping_destinations():
    t, u = torch.zeros(64), torch.zeros(64)
    moe.GradList([t[:32], t[32:], u])
    moe.GradList([t, t], [u, torch.zeros(64)])                 # read twice, written apart
    moe.GradList([t[:0], t[:0], t])
    for srcs, dsts in (([t, u, t], None), ([t[:33], t[32:]], None), ([t, u], [u, torch.zeros(64)]),
                       ([t[:32]], [t[16:48]]), ([t[:32], t[32:]], [u[:32], u[16:48]])):
        with pytest.raises(ValueError, match="overlap"):
            moe.GradList(srcs, dsts)
