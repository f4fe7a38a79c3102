"""TrainLayer's device status on the host: the library's calls are replaced by
ones that do what the real ones do to a workspace, each leaving a bit of its own
in the status word."""
import pytest
import torch

import mixture_experts_layer_group_b200 as moe
from mixture_experts_layer_group_b200 import build as moe_build
from mixture_experts_layer_group_b200 import train

WITH_STATUS = ["route_train", "dispatch_rows", "experts_train", "experts_backward", "route_backward"]
WITHOUT = ["combine", "combine_backward", "dispatch_backward"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe_build.build()


class Calls:
    """Stands in for the library: call number n in order of issue leaves bits[n] (0: none)."""

    def __init__(self, monkeypatch):
        self.bits, self.n, self.names = {}, 0, []
        for name in WITH_STATUS:
            monkeypatch.setattr(train, name, lambda *args, _name=name, **kw: self.call(_name, args))
        for name in WITHOUT:
            monkeypatch.setattr(train, name, lambda *args, **kw: None)

    def call(self, name, args):
        ws, = [a for a in args if isinstance(a, torch.Tensor) and a.dtype == torch.uint8]
        assert (ws.data_ptr() - ws.untyped_storage().data_ptr()) % 256 == 0
        T = args[1]
        if T == 0:
            return
        ws.fill_(0xA5)  # scratch, in which an earlier step's words may lie
        ws[:4].view(torch.int32)[0] = self.bits.get(self.n, 0)
        self.names.append(name)
        self.n += 1


def layer_of(n_shared):
    cfg = moe.make_cfg(d=64, d_ff=32, n_routed=8, n_shared=n_shared, top_k=2)
    w = dict(W_r=(8, 64), W1=(8, 32, 64), W3=(8, 32, 64), W2=(8, 64, 32))
    if n_shared:
        w.update(Ws1=(32, 64), Ws3=(32, 64), Ws2=(64, 32))
    return train.TrainLayer(cfg, {n: torch.zeros(s, dtype=torch.bfloat16) for n, s in w.items()}, max_tokens=4,
                            device="cpu")


@pytest.mark.parametrize("n_shared", [0, 1])
def test_device_status_holds_every_calls_bits(monkeypatch, n_shared):
    calls, layer = Calls(monkeypatch), layer_of(n_shared)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)

    def step():
        calls.n, calls.names = 0, []
        layer.forward(x)
        layer.backward(x)
        return calls.n

    total = step()
    assert layer.device_status() == 0
    assert total == 5 + 2 * n_shared and set(calls.names) == set(WITH_STATUS)
    for n in range(total):
        calls.bits = {n: 1 << n}
        step()
        calls.bits = {}
        step()  # a clean step on the same workspace does not clear it
        assert layer.device_status() == 1 << n, calls.names[n]
        assert layer.device_status() == 0
    calls.bits = {n: 1 << n for n in range(total)}
    step()
    assert layer.device_status() == (1 << total) - 1


@pytest.mark.parametrize("n_shared", [0, 1])
def test_device_status_after_a_forward_alone_and_a_step_without_tokens(monkeypatch, n_shared):
    calls, layer = Calls(monkeypatch), layer_of(n_shared)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    calls.bits = {n: 1 << n for n in range(3 + n_shared)}
    layer.forward(x)
    assert layer.device_status() == (1 << 3 + n_shared) - 1
    layer.forward(x[:0]), layer.backward(x[:0])  # nothing runs: the words of the step before do not count again
    assert layer.device_status() == 0


def test_the_calls_workspaces_hold_what_the_calls_need():
    for n_shared in (0, 1):
        layer = layer_of(n_shared)
        need = [moe.workspace_size(layer.cfg, 4)] * 2 + [moe.experts_workspace_size(layer.routed, 8)]
        need += [moe.experts_workspace_size(layer.shared, 4)] if n_shared else []
        need += [moe.experts_backward_workspace_size(layer.routed, 8), moe.route_backward_workspace_size(layer.cfg, 4)]
        need += [moe.experts_backward_workspace_size(layer.shared, 4)] if n_shared else []
        assert len(layer.call_ws) == len(need)
        for ws, n in zip(layer.call_ws, need):
            assert ws.numel() >= n


def test_device_status_reports_a_clip_that_gave_up(monkeypatch):
    """The norm's buffer keeps the mark over later clips until device_status() has reported it."""
    layer, gave_up, norms = layer_of(0), [False, True, False], iter((1.0, 2.0, 3.0, 4.0))

    def grad_clip(grads, sumsq, max_norm, norm_out):
        bits = norm_out.view(torch.int32)
        held = int(bits) == moe.MOE_NORM_INCOMPLETE
        norm_out.fill_(next(norms))
        if held or (gave_up and gave_up.pop(0)):
            bits.fill_(moe.MOE_NORM_INCOMPLETE)

    monkeypatch.setattr(train, "grad_norm", lambda *args: None)
    monkeypatch.setattr(train, "grad_clip", grad_clip)
    assert float(layer.clip(1.0)) == 1.0 and layer.device_status() == 0
    assert torch.isnan(layer.clip(1.0)).all()
    assert torch.isnan(layer.clip(1.0)).all()
    assert layer.device_status() == moe.MOE_DEV_WAIT_TIMEOUT
    assert layer.device_status() == 0
    assert float(layer.clip(1.0)) == 4.0 and layer.device_status() == 0


def test_the_norms_of_two_clips_keep_their_values(monkeypatch):
    layer, values = layer_of(0), iter((1.0, 2.0))
    monkeypatch.setattr(train, "grad_norm", lambda *args: None)
    monkeypatch.setattr(train, "grad_clip", lambda grads, sumsq, max_norm, norm_out: norm_out.fill_(next(values)))
    a, b = layer.clip(1.0), layer.clip(1.0)
    assert (float(a), float(b)) == (1.0, 2.0)


def test_the_mark_of_an_incomplete_clip_is_a_quiet_nan():
    mark = torch.tensor([moe.MOE_NORM_INCOMPLETE], dtype=torch.int32).view(torch.float32)
    assert torch.isnan(mark).all() and moe.MOE_NORM_INCOMPLETE & 0x7fc00000 == 0x7fc00000
    with open("include/moe_b200.h") as f:
        assert f"#define MOE_NORM_INCOMPLETE {moe.MOE_NORM_INCOMPLETE:#010x}u" in f.read()
