"""One training step of the DeepSeekMoE layer on one GPU.

TrainLayer orders the C ABI's training calls around buffers it keeps: the
forward that saves what the backward reads, the backward into weight-gradient
buffers, clipping by the global norm and the loss-free balancing of the
selection bias. Every compute step runs in the library's CUDA kernels; this
module only sizes the buffers and orders the calls. It holds no autograd
graph: forward() and backward() are called in turn, and a step can be captured
into a CUDA graph.
"""
from __future__ import annotations

import contextlib

import torch

from . import (MOE_BF16, MOE_DEV_WAIT_TIMEOUT, MOE_F32, MOE_NORM_INCOMPLETE, GradList, MoeCfg, bias_update, combine,
               combine_backward, dispatch_backward, dispatch_rows, experts_backward, experts_backward_workspace_size,
               experts_train, experts_workspace_size, grad_clip, grad_norm, grad_norm_workspace_size, route_backward,
               route_backward_workspace_size, route_train, workspace_size)

_STATUS_BYTES = 256  # of the status word at the head of a workspace, which is aligned to as many
_DTYPE = {MOE_BF16: torch.bfloat16, MOE_F32: torch.float32}


def _group_cfg(cfg: MoeCfg, groups: int, d_ff: int) -> MoeCfg:
    """The grouped-expert problem of `groups` experts of width d_ff."""
    return MoeCfg(d=cfg.d, d_ff=d_ff, n_routed=groups, n_shared=0, top_k=1, n_groups=1, topk_groups=1, route_scale=1.0,
                  dtype=cfg.dtype)


@contextlib.contextmanager
def _on(stream, *tensors):
    """Makes `stream` (None: leaves the current one) the stream that buffers belong to and calls run on; the
    caller's tensors are kept until what it has queued has read them."""
    if stream is None:
        yield
        return
    if isinstance(stream, torch.cuda.Stream):
        on = stream
    else:  # a handle; 0 is the default stream
        on = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    with torch.cuda.stream(on):
        yield
    for t in tensors:
        t.record_stream(on)


class TrainLayer:
    """The layer with its gradients.

    weights: as for MoELayer (bf16 or fp32 tensors in the layouts of the C
    ABI; FP8 weights are not trained). grads: the weights' gradients by name,
    of grad_dtype ("f32" or "bf16"; None: the layer's type), written by each
    backward(), or added to by backward(accumulate=True) (fp32). max_tokens
    bounds a call's tokens. All calls of one TrainLayer belong on one stream
    of the current device: the current one, or `stream`, which the results
    then belong to (the caller orders it after what wrote the arguments)."""

    def __init__(self, cfg: MoeCfg, weights: dict, max_tokens: int, grad_dtype=None, device="cuda"):
        self.cfg, self.w, self.max_tokens = cfg, weights, max_tokens
        self.grad_dtype = grad_dtype or {MOE_BF16: "bf16", MOE_F32: "f32"}[cfg.dtype]
        if self.grad_dtype not in ("f32", "bf16") or (self.grad_dtype == "bf16" and cfg.dtype == MOE_F32):
            raise ValueError(f"weight gradients are fp32, or bf16 in a bf16 layer: got {grad_dtype!r}")
        self.device = device
        self.dtype = _DTYPE[cfg.dtype]
        self.routed = _group_cfg(cfg, cfg.n_routed, cfg.d_ff)
        self.shared = _group_cfg(cfg, 1, cfg.n_shared * cfg.d_ff) if cfg.n_shared else None
        T, R = max_tokens, max_tokens * cfg.top_k
        forward = [workspace_size(cfg, T), workspace_size(cfg, T), experts_workspace_size(self.routed, R)]
        backward = [experts_backward_workspace_size(self.routed, R), route_backward_workspace_size(cfg, T)]
        if self.shared is not None:
            forward.append(experts_workspace_size(self.shared, T))
            backward.append(experts_backward_workspace_size(self.shared, T))
        # The calls of a step follow one another, so one buffer serves them all. Each call's workspace starts
        # behind the status word of the call before, which therefore keeps what its call found.
        sizes = forward + backward
        self.ws = torch.empty(max(_STATUS_BYTES * i + n for i, n in enumerate(sizes)), dtype=torch.uint8, device=device)
        self.call_ws = [self.ws[_STATUS_BYTES * i:] for i in range(len(sizes))]
        self.forward_calls = len(forward)
        for n, shape in self._weight_shapes().items():
            t = weights[n]
            if tuple(t.shape) != shape or t.dtype != self.dtype or not t.is_contiguous():
                raise ValueError(f"{n} is a contiguous {self.dtype} tensor {shape}: got {t.dtype} {tuple(t.shape)}")
        gdt = {"bf16": torch.bfloat16, "f32": torch.float32}[self.grad_dtype]
        self.grads = {n: torch.zeros(s, dtype=gdt, device=device) for n, s in self._weight_shapes().items()}
        self.grad_list = GradList(self.grads.values())
        self.clip_ws = torch.empty(grad_norm_workspace_size(self.grad_list), dtype=torch.uint8, device=device)
        self.sumsq = torch.zeros(1, dtype=torch.float64, device=device)
        self.norm = torch.zeros(1, dtype=torch.float32, device=device)
        self.status = torch.zeros(len(sizes), dtype=torch.int32, device=device)  # bits seen so far, by call
        self.saved = None

    def _weight_shapes(self):
        c = self.cfg
        shapes = {"W_r": (c.n_routed, c.d), "W1": (c.n_routed, c.d_ff, c.d), "W3": (c.n_routed, c.d_ff, c.d),
                  "W2": (c.n_routed, c.d, c.d_ff)}
        if c.n_shared:
            ff = c.n_shared * c.d_ff
            shapes.update(Ws1=(ff, c.d), Ws3=(ff, c.d), Ws2=(c.d, ff))
        return shapes

    def _check_rows(self, name, t):
        if t.dim() != 2 or t.shape[1] != self.cfg.d or t.dtype != self.dtype or not t.is_contiguous():
            raise ValueError(f"{name} is a contiguous {self.dtype} tensor [T, {self.cfg.d}]: got {t.dtype} "
                             f"{tuple(t.shape)}, strides {t.stride()}")

    def _new(self, shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device=self.device)

    def _note_status(self, T, first, last):
        """Keeps the device-status bits of calls first .. last - 1, which the next step's calls overwrite."""
        if T == 0:  # nothing ran
            return
        words = self.ws[:_STATUS_BYTES * last].view(torch.int32)[_STATUS_BYTES // 4 * first::_STATUS_BYTES // 4]
        self.status[first:last].bitwise_or_(words)

    def device_status(self, stream=None) -> int:
        """The MOE_DEV_* bits of the calls since the last device_status(), which are then cleared (synchronises)."""
        with _on(stream):
            words = self.status.tolist()
            self.status.zero_()
            norm = self.norm.view(torch.int32)
            if int(norm) == MOE_NORM_INCOMPLETE:  # a clip that gave up since: the mark stays until it is cleared
                words.append(MOE_DEV_WAIT_TIMEOUT)
                norm.zero_()
        bits = 0
        for w in words:
            bits |= w
        return bits

    def forward(self, x, stream=None):
        """y of the tokens x [T, d]; keeps what backward() needs. x itself is kept, not a copy (the routed
        experts' rows are one): it and the weights stay as they are until backward() has run, or the gradients
        of the router and the shared block mix two inputs."""
        self._check_rows("x", x)
        if x.shape[0] > self.max_tokens:
            raise ValueError(f"{x.shape[0]} tokens exceed max_tokens {self.max_tokens}")
        with _on(stream, x):
            return self._forward(x)

    def _forward(self, x):
        cfg, w, T, k = self.cfg, self.w, x.shape[0], self.cfg.top_k
        R, i32, f32 = T * k, torch.int32, torch.float32
        s = dict(x=x, idx=self._new((T, k), i32), gates=self._new((T, k), f32), logits=self._new((T, cfg.n_routed), f32),
                 counts=self._new(cfg.n_routed, i32), slot_pos=self._new((T, k), i32), x_rows=self._new((R, cfg.d)),
                 gate_rows=self._new(R, f32), gu=self._new((R, 2 * cfg.d_ff)))
        y = torch.empty_like(x)
        y_rows = self._new((R, cfg.d))
        offsets = self._new(cfg.n_routed + 1, i32)
        ws = self.call_ws[:self.forward_calls]
        route_train(cfg, T, x, w["W_r"], w.get("b"), s["idx"], s["gates"], s["logits"], ws[0])
        dispatch_rows(cfg, T, s["idx"], s["gates"], x, s["counts"], offsets, s["slot_pos"], s["x_rows"],
                      s["gate_rows"], ws[1])
        experts_train(self.routed, R, s["counts"], s["x_rows"], s["gate_rows"], w["W1"], w["W3"], w["W2"], y_rows,
                      s["gu"], ws[2])
        y_shared = None
        if self.shared is not None:
            s["shared_counts"] = torch.full((1,), T, dtype=i32, device=self.device)
            s["shared_gu"] = self._new((T, 2 * self.shared.d_ff))
            y_shared = self._new((T, cfg.d))
            experts_train(self.shared, T, s["shared_counts"], x, None, w["Ws1"], w["Ws3"], w["Ws2"], y_shared,
                          s["shared_gu"], ws[3])
        self._note_status(T, 0, len(ws))
        combine(cfg, T, y_rows, s["slot_pos"], y_shared, y)
        self.saved = s
        return y

    def backward(self, dy, accumulate=False, stream=None):
        """dx of the last forward's tokens from dy [T, d]; the weights' gradients go to `grads`."""
        if self.saved is None:
            raise RuntimeError("backward() without a forward()")
        x = self.saved["x"]
        if dy.shape != x.shape:
            raise ValueError(f"dy has shape {tuple(dy.shape)}, the forward's tokens {tuple(x.shape)}")
        self._check_rows("dy", dy)
        with _on(stream, dy, x):
            return self._backward(dy, accumulate)

    def _backward(self, dy, accumulate):
        cfg, w, g, s = self.cfg, self.w, self.grads, self.saved
        T, k = dy.shape[0], cfg.top_k
        R = T * k
        opt = dict(grad_dtype=self.grad_dtype, accumulate=accumulate)
        dy_rows, dx_rows = self._new((R, cfg.d)), self._new((R, cfg.d))
        dgate_rows = self._new(R, torch.float32)
        dx, dx_router, dx_shared = torch.empty_like(dy), torch.empty_like(dy), None
        ws = self.call_ws[self.forward_calls:]
        combine_backward(cfg, T, dy, s["slot_pos"], dy_rows)
        experts_backward(self.routed, R, s["counts"], s["x_rows"], s["gate_rows"], w["W1"], w["W3"], w["W2"], s["gu"],
                         dy_rows, dx_rows, dgate_rows, g["W1"], g["W3"], g["W2"], ws[0], **opt)
        route_backward(cfg, T, s["x"], w["W_r"], s["logits"], s["idx"], dgate_rows, s["slot_pos"], dx_router, g["W_r"],
                       ws[1], **opt)
        if self.shared is not None:
            dx_shared = torch.empty_like(dy)
            experts_backward(self.shared, T, s["shared_counts"], s["x"], None, w["Ws1"], w["Ws3"], w["Ws2"],
                             s["shared_gu"], dy, dx_shared, None, g["Ws1"], g["Ws3"], g["Ws2"], ws[2], **opt)
        self._note_status(T, self.forward_calls, len(self.call_ws))
        dispatch_backward(cfg, T, dx_rows, s["slot_pos"], dx_shared, dx_router, dx)
        return dx

    def clip(self, max_norm, group=None, stream=None):
        """Scales the gradients in place to a global norm of at most max_norm;
        returns the norm before (a new fp32 tensor of one element; NaN where the
        gradients may be unscaled because a wait ran out, which device_status()
        then reports). group: a torch.distributed group over whose ranks the
        gradients are spread."""
        with _on(stream):
            grad_norm(self.grad_list, self.sumsq, self.clip_ws)
            if group is not None:
                import torch.distributed as dist
                dist.all_reduce(self.sumsq, group=group)
            grad_clip(self.grad_list, self.sumsq, max_norm, self.norm)
            return self.norm.clone()  # (the buffer is the next clip's)

    def balance(self, gamma, stream=None):
        """The loss-free balancing step of the selection bias from the last forward's expert loads."""
        if self.saved is None:
            raise RuntimeError("balance() without a forward()")
        if self.w.get("b") is None:
            raise ValueError("the layer has no selection bias b")
        s = self.saved
        if s["x"].shape[0] == 0:  # no loads to balance
            return
        with _on(stream):
            bias_update(self.cfg, s["x"].shape[0], s["counts"], gamma, self.w["b"])
