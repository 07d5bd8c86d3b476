"""A packed MoE layer held in device memory: weights packed once with ``moe_pack``, then
``moe_layer_forward`` (or the four stage entry points) per call. Allocation and marshalling
only; the computation is in the library's kernels.
"""
from __future__ import annotations

import contextlib

import torch

from . import native as N


def pack(fmt: str, codes: torch.Tensor, scales, K: int, N_: int):
    """Pack `codes.shape[0]` stored K x N matrices; returns (packed, packed_scales or None)."""
    count = codes.shape[0] if codes.dim() == 3 else 1
    b, sb = N.moe_pack_size(fmt, count, K, N_)
    packed = torch.empty(b, dtype=torch.uint8, device=codes.device)
    pscale = torch.empty(sb, dtype=torch.uint8, device=codes.device) if sb else None
    N.moe_pack(fmt, count, K, N_, codes, scales, packed, pscale)
    return packed, pscale


def pack_expert_set(stored: dict, fmt: str, H: int, I: int) -> dict:
    out = {}
    for name, (K, Nn) in (("gate", (H, I)), ("up", (H, I)), ("down", (I, H))):
        out[name], out[name + "_scale"] = pack(fmt, stored[name], stored[name + "_scale"], K, Nn)
    return out


class PackedLayer:
    """Device-resident packed weights of one layer and a workspace sized for T tokens."""

    def __init__(self, spec, Wr: torch.Tensor, routed: dict, shared: dict | None, T: int | None = None,
                 path: str = "auto"):
        self.spec = spec
        self.shape = N.shape_from_spec(spec, T, path)
        H, I, E = spec.H, spec.I, spec.E
        self.Wr, _ = pack(spec.act, Wr.reshape(1, H, E), None, H, E)
        self.routed = pack_expert_set(routed, spec.w_routed, H, I)
        self.shared = pack_expert_set(shared, spec.w_shared, H, I) if spec.shared else None
        self.ws = torch.empty(N.moe_workspace_size(self.shape), dtype=torch.uint8, device=Wr.device)

    def set_tokens(self, T: int, path: str | None = None):
        p = {0: "auto", 1: "decode", 2: "prefill"}[self.shape.path] if path is None else path
        self.shape = N.shape_from_spec(self.spec, T, p)
        need = N.moe_workspace_size(self.shape)
        if need > self.ws.numel():
            self.ws = torch.empty(need, dtype=torch.uint8, device=self.ws.device)

    def forward_hash(self, x, bias, token_ids, hash_table, y, topk_idx=None, topk_w=None, stream=None):
        N.moe_layer_forward_hash(self.shape, x, self.Wr, bias, token_ids, hash_table, self.routed, self.shared, y,
                                 topk_idx, topk_w, self.ws, stream)
        return y

    def forward(self, x, bias, y, topk_idx=None, topk_w=None, stream=None):
        N.moe_layer_forward(self.shape, x, self.Wr, bias, self.routed, self.shared, y, topk_idx, topk_w,
                            self.ws, stream)
        return y


def _need(name: str, t: torch.Tensor, dtype, *shapes, device=None):
    if tuple(t.shape) not in shapes or t.dtype != dtype or not t.is_contiguous():
        raise ValueError("%s: a contiguous %s tensor of %s is needed" % (name, dtype, " or ".join(map(str, shapes))))
    if device is not None and not (t.is_cuda and t.device == device):
        raise ValueError("%s: a tensor on the layer's GPU is needed" % name)


def _result(like: torch.Tensor, stream):
    """A tensor that `stream` writes and the current stream may go on with: memory of the one, kept until work of the
    other on it has ended too."""
    if stream is None:
        return torch.empty_like(like)
    with torch.cuda.stream(stream):
        t = torch.empty_like(like)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


class TrainableLayer:
    """One layer's experts in training: forward, backward and AdamW step over row-major weights of the
    activations' type (gate, up [E, H, I], down [E, I, H]; the shared expert's without the first axis or
    with one of 1). The router is read only; its scores' gradient follows from backward's routing-weight
    gradient. Allocation and marshalling only, like PackedLayer.

    forward keeps what backward reads (x itself, not a copy), for the last batch alone. Calls, set_tokens and the
    constructor on one stream follow each other; a call on another stream has to wait for the former ones. No memory that a
    call works on (arguments, the layer's own and results) is handed on before that work has ended, whatever its stream.
    state: "f32", or "e4m3" for 8-bit optimizer states; master: fp32 master copies of bf16 weights."""

    NAMES = ("gate", "up", "down")

    def __init__(self, spec, Wr: torch.Tensor, routed: dict, shared: dict | None = None, T: int | None = None,
                 state: str = "f32", master: bool = False):
        self.H, self.I, self.E, self.k, self.act = spec.H, spec.I, spec.E, spec.k, spec.act
        self.dtype = torch.float32 if spec.act == "f32" else torch.bfloat16
        H, E, dev = spec.H, spec.E, Wr.device
        _need("Wr", Wr, self.dtype, (H, E), (1, H, E), device=dev)
        for d, lead in ((routed, [(spec.E,)]), (shared, [(), (1,)])):
            for n in self.NAMES if d is not None else ():
                size = (spec.I, spec.H) if n == "down" else (spec.H, spec.I)
                _need(n, d[n], self.dtype, *[a + size for a in lead], device=dev)
        self.weights = [{n: routed[n] for n in self.NAMES}]
        if shared is not None:
            self.weights.append({n: shared[n] for n in self.NAMES})
        self.grads = [{n: torch.zeros_like(t) for n, t in w.items()} for w in self.weights]
        with torch.cuda.device(dev):
            self.Wr, _ = pack(spec.act, Wr.reshape(1, H, E), None, H, E)
        p = [w[n] for w in self.weights for n in self.NAMES]
        g = [d[n] for d in self.grads for n in self.NAMES]
        if state == "e4m3":
            m, v = ([torch.zeros(t.numel(), dtype=torch.uint8, device=t.device) for t in p] for _ in range(2))
            ms, vs = ([torch.zeros((t.numel() + 255) // 256, device=t.device) for t in p] for _ in range(2))
        elif state == "f32":
            m, v = ([torch.zeros(t.shape, device=t.device) for t in p] for _ in range(2))
            ms = vs = None
        else:
            raise ValueError("state is f32 or e4m3")
        copies = [t.float() for t in p] if master else None
        self.optimizer = N.adamw_tensors(p, g, m, v, copies, ms, vs)
        self.steps = 0
        self.set_tokens(spec.T if T is None else T)

    def _shape(self, T, E, k):
        return N.make_shape(T, self.H, E, k, self.I, act=self.act, w_routed=self.act)

    def set_tokens(self, T: int, stream=None):
        """Buffers for batches of T tokens, made on `stream`."""
        with torch.cuda.stream(stream):
            self._set_tokens(T)

    def _set_tokens(self, T: int):
        dev, P, act = self.Wr.device, T * self.k, dict(dtype=self.dtype, device=self.Wr.device)
        self.T = self.x = None  # no batch fits until all buffers are there
        self.shapes = [self._shape(T, self.E, self.k)] + [self._shape(T, 1, 1)] * (len(self.weights) - 1)
        ws = max(N.moe_workspace_size(self.shapes[0]), *[N.moe_train_workspace_size(s) for s in self.shapes])
        self.ws = torch.empty(ws, dtype=torch.uint8, device=dev)
        self.idx, self.pair_slot = (torch.empty((T, self.k), dtype=torch.int32, device=dev) for _ in range(2))
        self.w = torch.empty((T, self.k), dtype=torch.float32, device=dev)
        self.ones = torch.ones((T, self.k), dtype=torch.float32, device=dev)
        self.off = torch.zeros(self.E + 1, dtype=torch.int32, device=dev)
        self.slot_token = torch.empty(P, dtype=torch.int32, device=dev)
        rows = [P] + [T] * (len(self.weights) - 1)
        self.pre = [[torch.empty((r, self.I), **act) for _ in range(2)] for r in rows]
        self.y, self.dx = ([torch.empty((r, self.H), **act) for r in rows] for _ in range(2))
        self.dy_perm = torch.empty((P, self.H), **act)
        self.T = T
        self.streams = {}  # by handle: those that the allocator knows to work on the layer's memory

    def _gpu(self):
        """The layer's GPU as the current one."""
        return contextlib.nullcontext() if torch._C._cuda_getDevice() == self.Wr.get_device() else torch.cuda.device(self.Wr.device)

    def _work_on(self, stream, *tensors):
        """This call's stream, until whose work so far has ended the allocator keeps tensors and, from the first call on it
        on, everything of the layer."""
        if stream is not None and stream.device != self.Wr.device:
            raise ValueError("stream: one of the layer's GPU is needed")
        handle = torch._C._cuda_getCurrentRawStream(self.Wr.get_device()) if stream is None else stream.cuda_stream
        if handle in self.streams:
            stream = self.streams[handle]
        else:
            stream = self.streams[handle] = torch.cuda.current_stream(self.Wr.device) if stream is None else stream
            tensors += (self.Wr, self.ws, self.idx, self.pair_slot, self.w, self.ones, self.off, self.slot_token, self.dy_perm,
                        *self.y, *self.dx, *[t for pair in self.pre for t in pair],
                        *[t for x in self.optimizer.keep if x is not None for t in x])
        for t in tensors:
            if torch.is_tensor(t) and t.is_cuda:
                t.record_stream(stream)
        return stream

    def forward(self, x, bias=None, stream=None):
        """y [T, H]; routing as moe_route, kept in idx and w."""
        _need("x", x, self.dtype, (self.T, self.H), device=self.Wr.device)
        if bias is not None:
            _need("bias", bias, torch.float32, (self.E,), device=self.Wr.device)
        y = _result(x, stream)
        stream = self._work_on(stream, x, bias)
        self.x = None  # until all that backward reads belongs to this batch
        with self._gpu():
            N.moe_route_permute(self.shapes[0], x, self.Wr, bias, self.idx, self.w, self.off, self.slot_token,
                                self.pair_slot, self.ws, stream)
            groups = [(self.off, self.slot_token), (None, None)]
            for shape, group, w, pre, out in zip(self.shapes, groups, self.weights, self.pre, self.y):
                N.moe_gated_ffn(shape, x, *group, w, *pre, out, self.ws, stream)
            N.moe_combine(self.shapes[0], self.y[0], self.pair_slot, self.w, self.y[1] if len(self.y) > 1 else None, y, stream)
        self.x = x
        return y

    def backward(self, dy, stream=None):
        """(dx through the experts [T, H], gradient of the routing weights [T, k]), both new tensors; fills grads."""
        if self.x is None:
            raise RuntimeError("backward needs a forward pass on this batch size")
        _need("dy", dy, self.dtype, (self.T, self.H), device=self.Wr.device)
        dx, dw = _result(dy, stream), _result(self.w, stream)
        stream = self._work_on(stream, self.x, dy)
        with self._gpu():
            N.moe_combine_backward(self.shapes[0], dy, self.y[0], self.pair_slot, self.w, self.dy_perm, dw, stream)
            groups = [(self.off, self.slot_token, self.dy_perm), (None, None, dy)]
            for shape, (off, slot, d), w, pre, out, grads in zip(self.shapes, groups, self.weights, self.pre, self.dx, self.grads):
                N.moe_gated_ffn_backward(shape, self.x, off, slot, w, *pre, d, out, grads, self.ws, stream)
            N.moe_combine(self.shapes[0], self.dx[0], self.pair_slot, self.ones, self.dx[1] if len(self.dx) > 1 else None, dx,
                          stream)
        return dx, dw

    def step(self, lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, stream=None, **more):
        """One AdamW step of every expert matrix by grads; more: moe_adamw's lr_dev, step_dev, grad_scale, seed."""
        stream = self._work_on(stream, *more.values())
        N.moe_adamw(self.optimizer, lr, beta1, beta2, eps, weight_decay, self.steps + 1, stream=stream, **more)
        self.steps += 1
