"""ctypes binding of ``libmoe.so`` with the C ABI's names (include/moe.h).

Argument marshalling only: torch tensors supply device pointers, the current torch stream is
passed as the HIP stream, and non-OK statuses become ``MoeError``. Every step of the layer
runs in the library's HIP kernels. There is no fallback: if the library is not built, loading
fails loudly.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

DTYPE = {"f32": 0, "bf16": 1, "fp8": 2, "mxfp4": 3, "mxfp4a8": 4, "mxfp8a8": 5, "int8": 6}
SCORE = {"softmax": 0, "sigmoid": 1}
PATH = {"auto": 0, "decode": 1, "prefill": 2}
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_WORKSPACE_TOO_SMALL", 4: "MOE_ERR_HIP"}
EXPORTS = ("moe_status_string", "moe_last_error", "moe_pack_size", "moe_pack", "moe_workspace_size",
           "moe_route", "moe_route_hash", "moe_permute", "moe_route_permute", "moe_grouped_ffn", "moe_combine",
           "moe_layer_forward", "moe_layer_forward_noalloc", "moe_layer_forward_hash", "moe_layer_forward_timed",
           "moe_quantize_mxfp8", "moe_quantize_int8", "moe_logical_workspace_size", "moe_layer_forward_logical",
           "moe_train_workspace_size", "moe_gated_ffn", "moe_gated_ffn_backward", "moe_combine_backward", "moe_adamw",
           "moe_gate", "moe_gate_backward", "moe_route_gated", "moe_layer_forward_gated",
           "moe_orthogonalize_workspace_size", "moe_orthogonalize", "moe_muon_workspace_size", "moe_muon")
# the library's own scratch, the workspace of moe_layer_forward_noalloc
NOALLOC_SCRATCH_BYTES = 64 << 20
TIMED_EVENTS = 7


class MoeError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__("%s: %s" % (STATUS.get(status, status), detail))
        self.status = status


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("I", ctypes.c_int32), ("I_shared", ctypes.c_int32),
                ("act", ctypes.c_int), ("w_routed", ctypes.c_int), ("w_shared", ctypes.c_int),
                ("path", ctypes.c_int)]


class MoeWeights(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("gate_scale", ctypes.c_void_p), ("up_scale", ctypes.c_void_p),
                ("down_scale", ctypes.c_void_p)]


class MoeWeightGrads(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p)]


class MoeAdamwTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "g", "m", "v", "m_scale", "v_scale", "master")] + [("n", ctypes.c_int64)]


class MoeAdamwConfig(ctypes.Structure):
    _fields_ = [("p_type", ctypes.c_int), ("g_type", ctypes.c_int), ("state", ctypes.c_int)] + \
               [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + \
               [("step", ctypes.c_int64), ("seed", ctypes.c_uint32)] + [(n, ctypes.c_void_p) for n in ("lr_dev", "step_dev", "grad_scale")]


class MoeGateRule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int)] + [(n, ctypes.c_int32) for n in ("groups", "top_groups", "group_top", "renormalize")] + \
               [("scale", ctypes.c_double)]


class MoeNewtonSchulz(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32)] + [(n, ctypes.c_double) for n in ("a", "b", "c", "eps")]


class MoeMuonTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "g", "m", "master")] + [(n, ctypes.c_int32) for n in ("count", "rows", "cols")] + \
               [("scale", ctypes.c_double)]


class MoeMuonConfig(ctypes.Structure):
    _fields_ = [("ns", MoeNewtonSchulz), ("p_type", ctypes.c_int), ("g_type", ctypes.c_int)] + \
               [(n, ctypes.c_double) for n in ("lr", "momentum", "weight_decay")] + [("nesterov", ctypes.c_int32)] + \
               [(n, ctypes.c_void_p) for n in ("lr_dev", "grad_scale")]


_lib = None


def load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoe.so is not built: run __graft_entry__.build() "
                               "(expert_ffn_layer_amd/build.py) first")
        lib = ctypes.CDLL(LIB_PATH)
        P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        PS, PW = ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWeights)
        lib.moe_status_string.restype = ctypes.c_char_p
        lib.moe_status_string.argtypes = [ctypes.c_int]
        lib.moe_last_error.restype = ctypes.c_char_p
        lib.moe_last_error.argtypes = []
        lib.moe_pack_size.argtypes = [ctypes.c_int, I32, I32, I32, ctypes.POINTER(SZ), ctypes.POINTER(SZ)]
        lib.moe_pack.argtypes = [ctypes.c_int, I32, I32, I32, P, P, P, P, P]
        lib.moe_workspace_size.argtypes = [PS, ctypes.POINTER(SZ)]
        lib.moe_route.argtypes = [PS, P, P, P, P, P, P, SZ, P]
        lib.moe_route_hash.argtypes = [PS, P, P, P, P, P, I32, P, P, P, SZ, P]
        lib.moe_permute.argtypes = [PS, P, P, P, P, P, SZ, P]
        lib.moe_route_permute.argtypes = [PS, P, P, P, P, P, P, P, P, P, SZ, P]
        lib.moe_grouped_ffn.argtypes = [PS, P, P, P, PW, PW, P, P, P, SZ, P]
        lib.moe_combine.argtypes = [PS, P, P, P, P, P, P]
        lib.moe_layer_forward.argtypes = [PS, P, P, P, PW, PW, P, P, P, P, SZ, P]
        lib.moe_layer_forward_noalloc.argtypes = [PS, P, P, P, PW, PW, P, P, P, P]
        lib.moe_layer_forward_hash.argtypes = [PS, P, P, P, P, P, I32, PW, PW, P, P, P, P, SZ, P]
        lib.moe_layer_forward_timed.argtypes = [PS, P, P, P, PW, PW, P, P, P, P, SZ, P,
                                                ctypes.POINTER(ctypes.c_void_p)]
        lib.moe_quantize_mxfp8.argtypes = [P, I32, I32, P, P, P]
        lib.moe_quantize_int8.argtypes = [P, I32, I32, P, P, P]
        lib.moe_logical_workspace_size.argtypes = [PS, ctypes.POINTER(SZ)]
        lib.moe_layer_forward_logical.argtypes = [PS, P, P, P, PW, PW, P, P, P, P, SZ, P]
        lib.moe_train_workspace_size.argtypes = [PS, ctypes.POINTER(SZ)]
        lib.moe_gated_ffn.argtypes = [PS, P, P, P, PW, P, P, P, P, SZ, P]
        lib.moe_gated_ffn_backward.argtypes = [PS, P, P, P, PW, P, P, P, P, ctypes.POINTER(MoeWeightGrads), P, SZ, P]
        lib.moe_combine_backward.argtypes = [PS, P, P, P, P, P, P, P]
        lib.moe_adamw.argtypes = [ctypes.POINTER(MoeAdamwConfig), ctypes.POINTER(MoeAdamwTensor), I32, P]
        PR = ctypes.POINTER(MoeGateRule)
        lib.moe_gate.argtypes = [PS, PR, P, P, P, P, P]
        lib.moe_gate_backward.argtypes = [PS, PR, P, P, P, P, P]
        lib.moe_route_gated.argtypes = [PS, PR, P, P, P, P, P, P, P, SZ, P]
        lib.moe_layer_forward_gated.argtypes = [PS, PR, P, P, P, PW, PW, P, P, P, P, SZ, P]
        lib.moe_orthogonalize_workspace_size.argtypes = [ctypes.c_int, I32, I32, I32, ctypes.POINTER(SZ)]
        lib.moe_orthogonalize.argtypes = [ctypes.POINTER(MoeNewtonSchulz), ctypes.c_int, I32, I32, I32, P, P, P, SZ, P]
        lib.moe_muon_workspace_size.argtypes = [ctypes.c_int, ctypes.POINTER(MoeMuonTensor), I32, ctypes.POINTER(SZ)]
        lib.moe_muon.argtypes = [ctypes.POINTER(MoeMuonConfig), ctypes.POINTER(MoeMuonTensor), I32, P, SZ, P]
        for name in EXPORTS[2:]:
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


def _check(rc: int):
    if rc != 0:
        raise MoeError(rc, load().moe_last_error().decode())


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _run(tensors, stream, call):
    """call(device pointers of tensors, stream handle) with their GPU as the current one, so that the call and its
    stream belong to it. The first tensor is not None."""
    import torch
    i = tensors[0].get_device()
    if stream is not None and stream.device.index != i:
        raise ValueError("the stream of a call is one of its tensors' GPU")
    at = []
    for t in tensors:
        if t is None:
            at.append(None)
        elif t.get_device() != i or i < 0:
            raise ValueError("the tensors of a call are on one GPU")
        elif not t.is_contiguous():
            raise ValueError("the tensors of a call are contiguous")
        else:
            at.append(t.data_ptr())
    if i != torch._C._cuda_getDevice():  # the current one
        with torch.cuda.device(i):
            rc = call(at, torch._C._cuda_getCurrentRawStream(i) if stream is None else stream.cuda_stream)
    else:
        rc = call(at, torch._C._cuda_getCurrentRawStream(i) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc)


def make_shape(T, H, E, k, I, I_shared=0, act="bf16", w_routed="bf16", w_shared="bf16", path="auto") -> MoeShape:
    return MoeShape(T, H, E, k, I, I_shared, DTYPE[act], DTYPE[w_routed], DTYPE[w_shared], PATH[path])


def shape_from_spec(spec, T=None, path="auto") -> MoeShape:
    return make_shape(spec.T if T is None else T, spec.H, spec.E, spec.k, spec.I,
                      spec.I if spec.shared else 0, spec.act, spec.w_routed, spec.w_shared, path)


def weights(d: dict | None):
    if d is None:
        return None
    return MoeWeights(*[None if d.get(n) is None else d[n].data_ptr()
                        for n in ("gate", "up", "down", "gate_scale", "up_scale", "down_scale")])


def moe_pack_size(fmt: str, count: int, K: int, N: int):
    b, s = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().moe_pack_size(DTYPE[fmt], count, K, N, ctypes.byref(b), ctypes.byref(s)))
    return b.value, s.value


def moe_pack(fmt, count, K, N, w, scale, packed, packed_scale, stream=None):
    _check(load().moe_pack(DTYPE[fmt], count, K, N, _p(w), _p(scale), _p(packed), _p(packed_scale),
                           _stream(stream)))


def moe_workspace_size(shape: MoeShape) -> int:
    b = ctypes.c_size_t()
    _check(load().moe_workspace_size(ctypes.byref(shape), ctypes.byref(b)))
    return b.value


def moe_logical_workspace_size(shape: MoeShape) -> int:
    b = ctypes.c_size_t()
    _check(load().moe_logical_workspace_size(ctypes.byref(shape), ctypes.byref(b)))
    return b.value


def moe_layer_forward_logical(shape, x, Wr, bias, routed: dict, shared: dict | None, y, topk_idx=None,
                              topk_w=None, ws=None, stream=None):
    """Weights in the logical row-major layout (moe_pack's source layout), packed into ws each call."""
    r, s = weights(routed), weights(shared)
    _check(load().moe_layer_forward_logical(ctypes.byref(shape), _p(x), _p(Wr), _p(bias), ctypes.byref(r),
                                            None if s is None else ctypes.byref(s), _p(y), _p(topk_idx),
                                            _p(topk_w), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                            _stream(stream)))


def moe_route(shape, x, Wr_packed, bias, topk_idx, topk_w, ws, stream=None):
    _check(load().moe_route(ctypes.byref(shape), _p(x), _p(Wr_packed), _p(bias), _p(topk_idx), _p(topk_w),
                            _p(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def moe_route_hash(shape, x, Wr_packed, bias, token_ids, hash_table, topk_idx, topk_w, ws, stream=None):
    _check(load().moe_route_hash(ctypes.byref(shape), _p(x), _p(Wr_packed), _p(bias), _p(token_ids),
                                 _p(hash_table), hash_table.shape[0], _p(topk_idx), _p(topk_w), _p(ws),
                                 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def moe_permute(shape, topk_idx, expert_offsets, slot_token, pair_slot, ws, stream=None):
    _check(load().moe_permute(ctypes.byref(shape), _p(topk_idx), _p(expert_offsets), _p(slot_token),
                              _p(pair_slot), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                              _stream(stream)))


def moe_route_permute(shape, x, Wr_packed, bias, topk_idx, topk_w, expert_offsets, slot_token, pair_slot, ws,
                      stream=None):
    _check(load().moe_route_permute(ctypes.byref(shape), _p(x), _p(Wr_packed), _p(bias), _p(topk_idx), _p(topk_w),
                                    _p(expert_offsets), _p(slot_token), _p(pair_slot), _p(ws),
                                    0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def moe_grouped_ffn(shape, x, expert_offsets, slot_token, routed: dict, shared: dict | None, y_perm, y_shared,
                    ws, stream=None):
    r, s = weights(routed), weights(shared)
    _check(load().moe_grouped_ffn(ctypes.byref(shape), _p(x), _p(expert_offsets), _p(slot_token),
                                  ctypes.byref(r), None if s is None else ctypes.byref(s), _p(y_perm),
                                  _p(y_shared), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                  _stream(stream)))


def moe_combine(shape, y_perm, pair_slot, topk_w, y_shared, y, stream=None):
    _check(load().moe_combine(ctypes.byref(shape), _p(y_perm), _p(pair_slot), _p(topk_w), _p(y_shared), _p(y),
                              _stream(stream)))


def moe_layer_forward(shape, x, Wr_packed, bias, routed: dict, shared: dict | None, y, topk_idx=None,
                      topk_w=None, ws=None, stream=None):
    r, s = weights(routed), weights(shared)
    _check(load().moe_layer_forward(ctypes.byref(shape), _p(x), _p(Wr_packed), _p(bias), ctypes.byref(r),
                                    None if s is None else ctypes.byref(s), _p(y), _p(topk_idx), _p(topk_w),
                                    _p(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                    _stream(stream)))


def moe_layer_forward_noalloc(shape, x, Wr_packed, bias, routed: dict, shared: dict | None, y, topk_idx=None,
                              topk_w=None, stream=None):
    r, s = weights(routed), weights(shared)
    _check(load().moe_layer_forward_noalloc(ctypes.byref(shape), _p(x), _p(Wr_packed), _p(bias), ctypes.byref(r),
                                            None if s is None else ctypes.byref(s), _p(y), _p(topk_idx), _p(topk_w),
                                            _stream(stream)))


def moe_layer_forward_hash(shape, x, Wr_packed, bias, token_ids, hash_table, routed: dict, shared: dict | None, y,
                           topk_idx=None, topk_w=None, ws=None, stream=None):
    r, s = weights(routed), weights(shared)
    _check(load().moe_layer_forward_hash(ctypes.byref(shape), _p(x), _p(Wr_packed), _p(bias), _p(token_ids),
                                         _p(hash_table), hash_table.shape[0], ctypes.byref(r),
                                         None if s is None else ctypes.byref(s), _p(y), _p(topk_idx), _p(topk_w),
                                         _p(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                         _stream(stream)))


def moe_layer_forward_timed(shape, x, Wr_packed, bias, routed: dict, shared: dict | None, y, events,
                            topk_idx=None, topk_w=None, ws=None, stream=None):
    """``events``: TIMED_EVENTS torch.cuda.Event(enable_timing=True) objects."""
    r, s = weights(routed), weights(shared)
    arr = (ctypes.c_void_p * TIMED_EVENTS)(*[e.cuda_event for e in events])
    _check(load().moe_layer_forward_timed(ctypes.byref(shape), _p(x), _p(Wr_packed), _p(bias), ctypes.byref(r),
                                          None if s is None else ctypes.byref(s), _p(y), _p(topk_idx),
                                          _p(topk_w), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                          _stream(stream), arr))


def moe_quantize_mxfp8(x, codes, scales, stream=None):
    """x bf16 [rows, K] -> codes uint8 [rows, K], scales uint8 [rows, K / 32] (e8m0)."""
    rows, K = (x.shape[0], x.shape[1]) if x is not None else (0, 32)
    _check(load().moe_quantize_mxfp8(_p(x), rows, K, _p(codes), _p(scales), _stream(stream)))


def moe_quantize_int8(x, codes, scales, stream=None):
    """x bf16 [rows, K] -> codes int8 [rows, K], scales float32 [rows]."""
    rows, K = (x.shape[0], x.shape[1]) if x is not None else (0, 8)
    _check(load().moe_quantize_int8(_p(x), rows, K, _p(codes), _p(scales), _stream(stream)))


def moe_train_workspace_size(shape: MoeShape) -> int:
    b = ctypes.c_size_t()
    _check(load().moe_train_workspace_size(ctypes.byref(shape), ctypes.byref(b)))
    return b.value


def moe_gated_ffn(shape, x, expert_offsets, slot_token, weights_: dict, gate_pre, up_pre, y_perm, ws, stream=None):
    """Weights row-major: gate, up [E, H, I], down [E, I, H]. gate_pre and up_pre may both be None."""
    tensors = (ws, x, expert_offsets, slot_token, gate_pre, up_pre, y_perm, weights_["gate"], weights_["up"], weights_["down"])
    _run(tensors, stream, lambda at, st: load().moe_gated_ffn(shape, *at[1:4], MoeWeights(*at[7:]), *at[4:7], at[0], ws.nbytes, st))


def moe_gated_ffn_backward(shape, x, expert_offsets, slot_token, weights_: dict, gate_pre, up_pre, dy_perm, dx_perm,
                           grads: dict | None, ws, stream=None):
    """grads: gate, up and down tensors that receive the weights' gradients, or None; dx_perm may be None."""
    tensors = (ws, x, expert_offsets, slot_token, gate_pre, up_pre, dy_perm, dx_perm,
               weights_["gate"], weights_["up"], weights_["down"])
    if grads is not None:
        tensors += (grads["gate"], grads["up"], grads["down"])
    _run(tensors, stream, lambda at, st: load().moe_gated_ffn_backward(
        shape, *at[1:4], MoeWeights(*at[8:11]), *at[4:8], MoeWeightGrads(*at[11:]) if len(at) > 11 else None, at[0], ws.nbytes, st))


def moe_combine_backward(shape, dy, y_perm, pair_slot, topk_w, dy_perm, dtopk_w, stream=None):
    _run((dy, y_perm, pair_slot, topk_w, dy_perm, dtopk_w), stream,
         lambda at, st: load().moe_combine_backward(shape, *at, st))


class AdamwTensors:
    """The tensor table of moe_adamw, with references that keep its tensors alive."""

    def __init__(self, array, keep, p_type: str, g_type: str, state: int):
        self.array, self.keep, self.p_type, self.g_type, self.state = array, keep, p_type, g_type, state


def adamw_tensors(p, g, m, v, master=None, m_scale=None, v_scale=None) -> AdamwTensors:
    """Lists of tensors, one entry per parameter; m_scale and v_scale select the E4M3 state (m and v then
    one byte an element). Made once and used for every step on the same tensors."""
    import torch
    lists = [p, g, m, v, m_scale, v_scale, master]
    if (m_scale is None) != (v_scale is None):
        raise ValueError("m_scale and v_scale go together")
    if any(x is not None and len(x) != len(p) for x in lists):
        raise ValueError("every list needs one tensor per parameter")
    q8 = m_scale is not None
    types = {torch.float32: "f32", torch.bfloat16: "bf16"}
    device = p[0].device if len(p) else None
    for i, t in enumerate(p):
        n = t.numel()
        if t.dtype not in types or g[i].dtype not in types or t.dtype != p[0].dtype or g[i].dtype != g[0].dtype:
            raise ValueError("parameters and gradients are float32 or bfloat16, one type each")
        if any(x[i].element_size() != 1 if q8 else x[i].dtype != torch.float32 for x in (m, v)):
            raise ValueError("m and v are float32, or one byte an element with scales")
        if any(x is not None and x[i].dtype != torch.float32 for x in (master, m_scale, v_scale)):
            raise ValueError("master copies and scales are float32")
        if any(x is not None and x[i].numel() != n for x in (g, m, v, master)):
            raise ValueError("tensor %d: sizes differ" % i)
        if q8 and any(x[i].numel() != (n + 255) // 256 for x in (m_scale, v_scale)):
            raise ValueError("tensor %d: one scale per 256 elements" % i)
        if any(x is not None and (not x[i].is_contiguous() or not x[i].is_cuda or x[i].device != device) for x in lists):
            raise ValueError("tensor %d: contiguous tensors of one GPU are needed" % i)
    array = (MoeAdamwTensor * len(p))(*[
        MoeAdamwTensor(*[None if x is None else x[i].data_ptr() for x in lists], n=t.numel()) for i, t in enumerate(p)])
    return AdamwTensors(array, [None if x is None else list(x) for x in lists], types[p[0].dtype] if len(p) else "f32",
                        types[g[0].dtype] if len(p) else "f32", int(q8))


def moe_adamw(tensors: AdamwTensors, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, lr_dev=None,
              step_dev=None, grad_scale=None, seed=0, stream=None):
    """lr_dev, grad_scale (float32) and step_dev (int64): one-element device tensors read in place of lr, 1, step.
    seed: of the E4M3 state's random rounding."""
    c = MoeAdamwConfig(DTYPE[tensors.p_type], DTYPE[tensors.g_type], tensors.state, lr, beta1, beta2, eps, weight_decay,
                       step, seed & 0xFFFFFFFF)
    if not len(tensors.array):
        return
    import torch
    for t, dtype in ((lr_dev, torch.float32), (step_dev, torch.int64), (grad_scale, torch.float32)):
        if t is not None and (t.dtype != dtype or not t.numel()):
            raise ValueError("lr_dev and grad_scale hold a float32, step_dev an int64")

    def call(at, st):
        c.lr_dev, c.step_dev, c.grad_scale = at[1:]
        return load().moe_adamw(c, tensors.array, len(tensors.array), st)
    _run((tensors.keep[0][0], lr_dev, step_dev, grad_scale), stream, call)


def make_gate(score="softmax", groups=1, top_groups=None, group_top=1, renormalize=True, scale=1.0) -> MoeGateRule:
    """The rule of the gate; top_groups: groups where it is None."""
    return MoeGateRule(SCORE[score], groups, groups if top_groups is None else top_groups, group_top, bool(renormalize), scale)


def _sized(*checks):
    """(name, tensor or None, dtype, elements) of each argument."""
    for name, t, dtype, n in checks:
        if t is not None and (t.dtype != dtype or t.numel() != n):
            raise ValueError("%s: %d elements of %s are needed" % (name, n, dtype))


def moe_gate(shape, rule, logits, bias, topk_idx, topk_w, stream=None):
    """logits float32 [T, E], bias float32 [E] or None -> topk_idx int32 [T, k], topk_w float32 [T, k]."""
    import torch
    P = shape.T * shape.k
    _sized(("logits", logits, torch.float32, shape.T * shape.E), ("bias", bias, torch.float32, shape.E),
           ("topk_idx", topk_idx, torch.int32, P), ("topk_w", topk_w, torch.float32, P))
    _run((logits, bias, topk_idx, topk_w), stream, lambda at, st: load().moe_gate(shape, rule, *at, st))


def moe_gate_backward(shape, rule, logits, topk_idx, dtopk_w, dlogits, stream=None):
    """dlogits float32 [T, E], which may be logits, from the gradient of the weights, float32 [T, k]."""
    import torch
    P = shape.T * shape.k
    _sized(("logits", logits, torch.float32, shape.T * shape.E), ("topk_idx", topk_idx, torch.int32, P),
           ("dtopk_w", dtopk_w, torch.float32, P), ("dlogits", dlogits, torch.float32, shape.T * shape.E))
    _run((logits, topk_idx, dtopk_w, dlogits), stream, lambda at, st: load().moe_gate_backward(shape, rule, *at, st))


def moe_route_gated(shape, rule, x, Wr_packed, bias, logits, topk_idx, topk_w, ws, stream=None):
    """logits float32 [T, E] receives the router's scores, or None."""
    import torch
    P = shape.T * shape.k
    _sized(("bias", bias, torch.float32, shape.E), ("logits", logits, torch.float32, shape.T * shape.E),
           ("topk_idx", topk_idx, torch.int32, P), ("topk_w", topk_w, torch.float32, P))
    _run((ws, x, Wr_packed, bias, logits, topk_idx, topk_w), stream,
         lambda at, st: load().moe_route_gated(shape, rule, *at[1:], at[0], ws.nbytes, st))


def moe_layer_forward_gated(shape, rule, x, Wr_packed, bias, routed: dict, shared: dict | None, y, topk_idx=None,
                            topk_w=None, ws=None, stream=None):
    r, s = weights(routed), weights(shared)
    _check(load().moe_layer_forward_gated(ctypes.byref(shape), ctypes.byref(rule), _p(x), _p(Wr_packed), _p(bias),
                                          ctypes.byref(r), None if s is None else ctypes.byref(s), _p(y), _p(topk_idx),
                                          _p(topk_w), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                          _stream(stream)))


NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)  # takes singular values from 0.01 to 1 into 0.68 to 1.2 in five steps


def moe_orthogonalize_workspace_size(type_: str, count: int, rows: int, cols: int) -> int:
    b = ctypes.c_size_t()
    _check(load().moe_orthogonalize_workspace_size(DTYPE[type_], count, rows, cols, ctypes.byref(b)))
    return b.value


def _matrix_type(t):
    import torch
    name = {torch.float32: "f32", torch.bfloat16: "bf16"}.get(t.dtype)
    if name is None:
        raise ValueError("matrices are float32 or bfloat16")
    return name


def moe_orthogonalize(g, o, ws, steps=5, coefficients=NEWTON_SCHULZ, eps=1e-7, stream=None):
    """g, o [count, rows, cols] or [rows, cols], float32 or bfloat16."""
    kind, shape = DTYPE[_matrix_type(g)], tuple(g.shape)
    if len(shape) not in (2, 3) or tuple(o.shape) != shape or o.dtype != g.dtype:
        raise ValueError("g and o are matrices, or stacks of them, of one size and type")
    count, rows, cols = shape if len(shape) == 3 else (1, *shape)
    ns = MoeNewtonSchulz(steps, *coefficients, eps)
    _run((g, o, ws), stream, lambda at, st: load().moe_orthogonalize(ns, kind, count, rows, cols, *at, ws.nbytes, st))


class MuonTensors:
    """The table of moe_muon, with references that keep its tensors alive."""

    def __init__(self, array, keep, p_type: str, g_type: str):
        self.array, self.keep, self.p_type, self.g_type = array, keep, p_type, g_type


def muon_tensors(p, g, m, master=None, scale=None) -> MuonTensors:
    """Lists of tensors, one entry per parameter: matrices [rows, cols] or stacks of them [count, rows, cols]. scale: a
    number each; None: 0.2 sqrt(max(rows, cols)), which gives the update AdamW's usual size. Made once and used for every
    step on the same tensors."""
    import torch
    lists = [p, g, m, master]
    if any(x is not None and len(x) != len(p) for x in lists + [scale]):
        raise ValueError("every list needs one entry per parameter")
    device = p[0].device if len(p) else None
    rows = []
    for i, t in enumerate(p):
        if t.dim() not in (2, 3):
            raise ValueError("tensor %d: a matrix or a stack of matrices is needed" % i)
        if t.dtype != p[0].dtype or g[i].dtype != g[0].dtype:
            raise ValueError("parameters and gradients are of one type each")
        _matrix_type(t), _matrix_type(g[i])
        if any(x is not None and x[i].dtype != torch.float32 for x in (m, master)):
            raise ValueError("momenta and master copies are float32")
        if any(x is not None and x[i].shape != t.shape for x in (g, m, master)):
            raise ValueError("tensor %d: sizes differ" % i)
        if any(x is not None and (not x[i].is_contiguous() or not x[i].is_cuda or x[i].device != device) for x in lists):
            raise ValueError("tensor %d: contiguous tensors of one GPU are needed" % i)
        size = tuple(t.shape) if t.dim() == 3 else (1, *t.shape)
        rows.append(MoeMuonTensor(*[None if x is None else x[i].data_ptr() for x in lists], *size,
                                  0.2 * max(size[1:]) ** 0.5 if scale is None else scale[i]))
    return MuonTensors((MoeMuonTensor * len(p))(*rows), [None if x is None else list(x) for x in lists],
                       _matrix_type(p[0]) if len(p) else "f32", _matrix_type(g[0]) if len(p) else "f32")


def moe_muon_workspace_size(tensors: MuonTensors) -> int:
    b = ctypes.c_size_t()
    _check(load().moe_muon_workspace_size(DTYPE[tensors.p_type], tensors.array, len(tensors.array), ctypes.byref(b)))
    return b.value


def moe_muon(tensors: MuonTensors, ws, lr=1e-3, momentum=0.95, nesterov=True, weight_decay=0.0, steps=5,
             coefficients=NEWTON_SCHULZ, eps=1e-7, lr_dev=None, grad_scale=None, stream=None):
    """lr_dev, grad_scale: one-element float32 device tensors read in place of lr and 1."""
    if not len(tensors.array):
        return
    import torch
    for t in (lr_dev, grad_scale):
        if t is not None and (t.dtype != torch.float32 or not t.numel()):
            raise ValueError("lr_dev and grad_scale hold a float32")
    c = MoeMuonConfig(MoeNewtonSchulz(steps, *coefficients, eps), DTYPE[tensors.p_type], DTYPE[tensors.g_type], lr, momentum,
                      weight_decay, bool(nesterov))

    def call(at, st):
        c.lr_dev, c.grad_scale = at[2:]
        return load().moe_muon(c, tensors.array, len(tensors.array), at[1], ws.nbytes, st)
    _run((tensors.keep[0][0], ws, lr_dev, grad_scale), stream, call)
