"""Torch-tensor binding of the C ABI (include/moe.h), same names as the C calls.

Only argument marshalling happens here: pointers, sizes and the current CUDA
stream are passed to the library; every step of the block runs in its CUDA
kernels.  Torch provides device memory and streams.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
from typing import Optional

import torch

from . import abi
from .abi import check, load

__all__ = [
    "ExpertWeights", "Plan", "moe_workspace_bytes", "moe_workspace_layout", "moe_route", "moe_plan",
    "moe_experts", "moe_forward", "moe_forward_host", "moe_shared_expert", "moe_set_dispatch", "moe_set_combine",
    "moe_device_error",
    "moe_last_error", "moe_version", "new_plan", "new_workspace", "dims", "moe_profile_hook",
    "moe_last_launch_count", "exec_cfg", "moe_experts_ex", "DecodeLayer", "moe_decode_workspace_bytes",
    "moe_linear",
]


def dims(T: int, H: int, E: int, k: int, I: int) -> abi.moe_dims:
    return abi.moe_dims(T, H, E, k, I)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_NO_CONTEXT = contextlib.nullcontext()


def _alloc_on(stream, device: torch.device):
    """Context in which ``stream`` (None: no other) is the current one and new tensors
    belong to it: else the allocator may hand out blocks whose last use, on the current
    stream, is still to come."""
    if stream is None or device.type != "cuda" or _stream(stream) == torch._C._cuda_getCurrentRawStream(device.index):
        return _NO_CONTEXT
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                             else torch.cuda.ExternalStream(_stream(stream), device=device))


@dataclasses.dataclass
class ExpertWeights:
    """Device tensors of the experts (layouts as in include/moe.h)."""
    act: int                          # abi.MOE_ACT_SWIGLU | abi.MOE_ACT_RELU2
    fmt: int                          # abi.MOE_W_BF16 | abi.MOE_W_AFFINE4_G64 | abi.MOE_W_NVFP4
    w1: torch.Tensor
    w2: torch.Tensor
    w1_scale: Optional[torch.Tensor] = None
    w1_bias: Optional[torch.Tensor] = None
    w2_scale: Optional[torch.Tensor] = None
    w2_bias: Optional[torch.Tensor] = None
    swiglu_limit: float = 0.0
    w1_global: Optional[torch.Tensor] = None   # NVFP4: (E,) fp32 global scales
    w2_global: Optional[torch.Tensor] = None

    def c_struct(self) -> abi.moe_experts_w:
        return abi.moe_experts_w(self.fmt, self.act, _ptr(self.w1), _ptr(self.w1_scale), _ptr(self.w1_bias),
                                 _ptr(self.w2), _ptr(self.w2_scale), _ptr(self.w2_bias), self.swiglu_limit,
                                 _ptr(self.w1_global), _ptr(self.w2_global))

    def clone(self) -> "ExpertWeights":
        c = lambda t: None if t is None else t.clone()  # noqa: E731
        return ExpertWeights(act=self.act, fmt=self.fmt, w1=c(self.w1), w2=c(self.w2), w1_scale=c(self.w1_scale),
                             w1_bias=c(self.w1_bias), w2_scale=c(self.w2_scale), w2_bias=c(self.w2_bias),
                             swiglu_limit=self.swiglu_limit, w1_global=c(self.w1_global),
                             w2_global=c(self.w2_global))


def router_cfg(score: str = "sigmoid", norm_topk: bool = True) -> abi.moe_router_cfg:
    return abi.moe_router_cfg({"sigmoid": abi.MOE_SCORE_SIGMOID, "softmax": abi.MOE_SCORE_SOFTMAX}[score],
                              1 if norm_topk else 0)


def exec_cfg(dispatch: Optional[int] = None, combine: Optional[int] = None) -> Optional[abi.moe_exec_cfg]:
    """A per-call execution choice, or None (the library's process-wide
    defaults) when neither is given; a missing one of the two takes the
    library's default value (AUTO dispatch, atomic combine)."""
    if dispatch is None and combine is None:
        return None
    return abi.moe_exec_cfg(abi.MOE_DISPATCH_AUTO if dispatch is None else dispatch,
                            abi.MOE_COMBINE_ATOMIC if combine is None else combine)


def _ref(c):
    return None if c is None else ctypes.byref(c)


@dataclasses.dataclass
class Plan:
    counts: torch.Tensor   # [E] int32
    offsets: torch.Tensor  # [E+1]
    perm: torch.Tensor     # [P]
    inv: torch.Tensor      # [P]
    tiles: torch.Tensor    # [E+1]

    def c_struct(self) -> abi.moe_plan_t:
        return abi.moe_plan_t(_ptr(self.counts), _ptr(self.offsets), _ptr(self.perm), _ptr(self.inv),
                              _ptr(self.tiles))


def new_plan(T: int, E: int, k: int, device="cuda") -> Plan:
    P = max(T * k, 1)
    z = lambda n: torch.empty(n, dtype=torch.int32, device=device)  # noqa: E731
    return Plan(z(E), z(E + 1), z(P), z(P), z(E + 1))


def moe_workspace_bytes(d: abi.moe_dims, fmt: int = abi.MOE_W_BF16, *, dispatch=None, combine=None) -> int:
    return int(load().moe_workspace_bytes_ex(ctypes.byref(d), fmt, _ref(exec_cfg(dispatch, combine))))


def moe_workspace_layout(d: abi.moe_dims, fmt: int = abi.MOE_W_BF16, *, dispatch=None,
                         combine=None) -> abi.moe_ws_layout:
    out = abi.moe_ws_layout()
    check(load().moe_workspace_layout_ex(ctypes.byref(d), fmt, _ref(exec_cfg(dispatch, combine)),
                                         ctypes.byref(out)), "moe_workspace_layout")
    return out


def new_workspace(d: abi.moe_dims, fmt: int = abi.MOE_W_BF16, device="cuda", *, dispatch=None,
                  combine=None) -> torch.Tensor:
    n = moe_workspace_bytes(d, fmt, dispatch=dispatch, combine=combine)
    if n == 0:
        raise ValueError("invalid sizes for a workspace")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_route(x=None, logits=None, w_router=None, expert_bias=None, *, E: int, k: int, eps: float = 1e-6,
              scale: float = 1.0, topk_idx=None, topk_w=None, stream=None, score: str = "sigmoid",
              norm_topk: bool = True):
    src = x if x is not None else logits
    T = src.shape[0]
    H = x.shape[1] if x is not None else (w_router.shape[1] if w_router is not None else 64)
    d = abi.moe_dims(T, H, E, k, 64)
    dev = src.device
    with _alloc_on(stream, dev):
        if topk_idx is None:
            topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        if topk_w is None:
            topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
    rc = router_cfg(score, norm_topk)
    check(load().moe_route_ex(_ptr(x), _ptr(logits), _ptr(w_router), _ptr(expert_bias), ctypes.byref(d),
                              eps, scale, ctypes.byref(rc), _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
          "moe_route")
    return topk_idx, topk_w


def moe_plan(topk_idx, *, E: int, H: int = 64, I: int = 64, plan: Optional[Plan] = None, ws=None,
             stream=None) -> Plan:
    T, k = topk_idx.shape
    d = abi.moe_dims(T, H, E, k, I)
    with _alloc_on(stream, topk_idx.device):
        plan = plan or new_plan(T, E, k, topk_idx.device)
        ws = ws if ws is not None else new_workspace(d, device=topk_idx.device)
    cp = plan.c_struct()
    check(load().moe_plan(_ptr(topk_idx), ctypes.byref(d), ctypes.byref(cp), _ptr(ws), ws.numel(),
                          _stream(stream)), "moe_plan")
    return plan


def moe_experts(x, plan: Plan, topk_w, W: ExpertWeights, *, E: int, I: int, out_scale: float = 1.0, y=None,
                ws=None, stream=None, skip: int = -1, y_shared=None, dispatch=None, combine=None):
    """Grouped experts + combine over a plan of E plan experts; ``skip`` >= 0
    names a plan expert whose pairs are computed nowhere and left out (W then
    holds E - 1 experts when skip == E - 1)."""
    T, H = x.shape
    k = topk_w.shape[1]
    d = abi.moe_dims(T, H, E, k, I)
    ex = exec_cfg(dispatch, combine)
    with _alloc_on(stream, x.device):
        y = y if y is not None else torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
        ws = ws if ws is not None else new_workspace(d, W.fmt, x.device, dispatch=dispatch, combine=combine)
    cp, cw = plan.c_struct(), W.c_struct()
    check(load().moe_experts_ex(_ptr(x), ctypes.byref(cp), _ptr(topk_w), ctypes.byref(d), ctypes.byref(cw),
                                _ref(ex), skip, _ptr(y_shared), out_scale, _ptr(y), _ptr(ws), ws.numel(),
                                _stream(stream)), "moe_experts")
    return y


moe_experts_ex = moe_experts


def moe_forward(x, W: ExpertWeights, w_router=None, expert_bias=None, *, E: int, k: int, I: int,
                logits=None, eps: float = 1e-6, router_scale: float = 1.0, out_scale: float = 1.0,
                topk_idx=None, topk_w=None, plan: Optional[Plan] = None, y=None, ws=None, stream=None,
                score: str = "sigmoid", norm_topk: bool = True, y_shared=None, dispatch=None, combine=None):
    T, H = x.shape
    d = abi.moe_dims(T, H, E, k, I)
    dev = x.device
    ex = exec_cfg(dispatch, combine)
    with _alloc_on(stream, dev):
        topk_idx = topk_idx if topk_idx is not None else torch.empty((T, k), dtype=torch.int32, device=dev)
        topk_w = topk_w if topk_w is not None else torch.empty((T, k), dtype=torch.float32, device=dev)
        plan = plan or new_plan(T, E, k, dev)
        y = y if y is not None else torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        ws = ws if ws is not None else new_workspace(d, W.fmt, dev, dispatch=dispatch, combine=combine)
    cp, cw, rc = plan.c_struct(), W.c_struct(), router_cfg(score, norm_topk)
    check(load().moe_forward_ex(_ptr(x), _ptr(logits), _ptr(w_router), _ptr(expert_bias), ctypes.byref(d), eps,
                                router_scale, out_scale, ctypes.byref(rc), _ref(ex), _ptr(y_shared),
                                ctypes.byref(cw),
                                _ptr(topk_idx), _ptr(topk_w), ctypes.byref(cp), _ptr(y), _ptr(ws), ws.numel(),
                                _stream(stream)), "moe_forward")
    return y, topk_idx, topk_w, plan


def moe_shared_expert(x, Ws: ExpertWeights, *, I: int, y_shared=None, ws=None, stream=None, dispatch=None,
                      combine=None):
    """fp32 (T, H) output of the shared expert (one expert, weight 1, on every token)."""
    T, H = x.shape
    d = abi.moe_dims(T, H, 1, 1, I)
    ex = exec_cfg(dispatch, combine)
    with _alloc_on(stream, x.device):
        y_shared = y_shared if y_shared is not None else torch.empty((T, H), dtype=torch.float32, device=x.device)
        ws = ws if ws is not None else new_workspace(d, Ws.fmt, x.device, dispatch=dispatch, combine=combine)
    cw = Ws.c_struct()
    check(load().moe_shared_expert_ex(_ptr(x), ctypes.byref(cw), ctypes.byref(d), _ref(ex), _ptr(y_shared),
                                      _ptr(ws), ws.numel(), _stream(stream)), "moe_shared_expert")
    return y_shared


def moe_forward_host(x_host: torch.Tensor, x_dev, W: ExpertWeights, w_router, expert_bias, *, E: int, k: int,
                     I: int, y_dev, y_host: torch.Tensor, topk_idx, topk_w, plan: Plan, ws, eps: float = 1e-6,
                     router_scale: float = 1.0, out_scale: float = 1.0, stream=None):
    """Host token rows in, host output rows out (the call synchronises its stream)."""
    T, H = x_host.shape
    if x_host.is_cuda or y_host.is_cuda:
        raise ValueError("x_host and y_host must be host tensors")
    d = abi.moe_dims(T, H, E, k, I)
    cp, cw = plan.c_struct(), W.c_struct()
    check(load().moe_forward_host(x_host.data_ptr(), _ptr(x_dev), _ptr(w_router), _ptr(expert_bias),
                                  ctypes.byref(d), eps, router_scale, out_scale, ctypes.byref(cw),
                                  _ptr(topk_idx), _ptr(topk_w), ctypes.byref(cp), _ptr(y_dev),
                                  y_host.data_ptr(), _ptr(ws), ws.numel(), _stream(stream)), "moe_forward_host")
    return y_host


_LINEAR_ACT = {"none": abi.MOE_ACT_NONE, "relu2": abi.MOE_ACT_RELU2, "swiglu": abi.MOE_ACT_SWIGLU}


_BF16, _FP32, _OUT = (torch.bfloat16,), (torch.float32,), (torch.bfloat16, torch.float32)


def _rows(name: str, t: torch.Tensor, rows: int, cols: int, dtypes, device) -> int:
    """Row stride of a (rows, cols) matrix with unit column stride, or ValueError."""
    if t.device != device or t.dtype not in dtypes or t.shape != (rows, cols):
        raise ValueError(f"{name}: expected ({rows}, {cols}) of {dtypes[0]} on {device}, got {tuple(t.shape)} of "
                         f"{t.dtype} on {t.device}")
    s0, s1 = t.stride()
    if (s1 != 1 and cols > 1) or (s0 < cols and rows > 1):
        raise ValueError(f"{name}: expected unit column stride and rows that do not overlap, got strides {t.stride()}")
    return s0 if rows > 1 else (cols + 7) // 8 * 8   # the stride of a single row means nothing


def moe_linear(x, w, bias=None, residual=None, *, act: str = "none", swiglu_limit: float = 0.0, out_dtype=None, y=None,
               stream=None):
    """y = act(x w^T + bias) + residual (``act``: "none", "relu2" or "swiglu", the
    last with w = [gate; up] of 2N rows).  x (M, K) and w are bf16 with row strides
    that are multiples of 8; bias is fp32; residual and y are bf16 or fp32 with any
    row stride.  y defaults to a new bf16 (or ``out_dtype``) tensor; it may be the
    residual itself, any other overlap with an input is refused."""
    if stream is not None:
        with _alloc_on(stream, x.device):
            return moe_linear(x, w, bias, residual, act=act, swiglu_limit=swiglu_limit, out_dtype=out_dtype, y=y)
    if not x.is_cuda or x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w: expected CUDA matrices")
    dev, (M, K), rows = x.device, x.shape, w.shape[0]
    code = _LINEAR_ACT.get(act)
    if code is None:
        raise ValueError(f"act: expected one of {sorted(_LINEAR_ACT)}, got {act!r}")
    if act == "swiglu" and rows % 2:
        raise ValueError("w: swiglu needs an even number of rows (gate, then up)")
    N = rows // 2 if act == "swiglu" else rows
    ldx = _rows("x", x, M, K, _BF16, dev)
    ldw = _rows("w", w, rows, K, _BF16, dev)
    bias_p = res_p = None
    ldr, res_f32 = N, False
    if bias is not None:
        _want("bias", bias, (rows,), _FP32, dev)
        bias_p = bias.data_ptr()
    if residual is not None:
        ldr = _rows("residual", residual, M, N, _OUT, dev)
        res_p, res_f32 = residual.data_ptr(), residual.dtype is torch.float32
    if y is None:
        y = x.new_empty((M, N), dtype=out_dtype)   # (None: x's bf16)
        if y.dtype not in _OUT:
            raise ValueError(f"out_dtype: expected bfloat16 or float32, got {out_dtype}")
        ldy = N
    else:
        if out_dtype is not None and y.dtype != out_dtype:
            raise ValueError(f"y is {y.dtype}, out_dtype is {out_dtype}")
        ldy = _rows("y", y, M, N, _OUT, dev)
    d = abi.moe_linear_dims(M, N, K, ldx, ldw, ldr, ldy)
    cfg = abi.moe_linear_cfg(code, res_f32, y.dtype is torch.float32, swiglu_limit)
    args = (x.data_ptr(), w.data_ptr(), bias_p, res_p, ctypes.byref(d), ctypes.byref(cfg), y.data_ptr(),
            torch._C._cuda_getCurrentRawStream(dev.index))
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            st = load().moe_linear(*args)
    else:
        st = load().moe_linear(*args)
    if st:
        check(st, "moe_linear")
    return y


def moe_decode_workspace_bytes(d: abi.moe_dims, Is: int = 0) -> int:
    return int(load().moe_decode_workspace_bytes(ctypes.byref(d), Is))


def _want(name: str, t: Optional[torch.Tensor], shape, dtypes, device) -> None:
    """Refuse a tensor that the library would read with another shape or type."""
    if t is None:
        return
    if t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got {t.device}")
    if t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {tuple(shape)} of {dtypes[0]}, got {tuple(t.shape)} of {t.dtype}")


def _check_weights(name: str, W: ExpertWeights, E: int, I: int, H: int, device) -> None:
    n1 = 2 * I if W.act == abi.MOE_ACT_SWIGLU else I
    for i, n, K in ((1, n1, H), (2, H, I)):
        w, sc = getattr(W, f"w{i}"), getattr(W, f"w{i}_scale")
        if W.fmt == abi.MOE_W_BF16:
            _want(f"{name}.w{i}", w, (E, n, K), (torch.bfloat16,), device)
        elif W.fmt == abi.MOE_W_AFFINE4_G64:
            _want(f"{name}.w{i}", w, (E, n, K // 8), (torch.int32, torch.uint32), device)
            _want(f"{name}.w{i}_scale", sc, (E, n, K // 64), (torch.bfloat16,), device)
            _want(f"{name}.w{i}_bias", getattr(W, f"w{i}_bias"), (E, n, K // 64), (torch.bfloat16,), device)
        else:
            _want(f"{name}.w{i}", w, (E, n, K // 2), (torch.uint8,), device)
            _want(f"{name}.w{i}_scale", sc, (E, n, K // 16), (torch.uint8,), device)
            _want(f"{name}.w{i}_global", getattr(W, f"w{i}_global"), (E,), (torch.float32,), device)


class DecodeLayer:
    """A whole MoE layer for a few tokens, one kernel launch a call (``moe_decode``;
    from about 9 tokens with 4-bit experts, 12 with bf16 ones, ``moe_forward`` is faster).

    Holds what stays the same from step to step: the router, the experts, an
    optional shared expert (``Ws`` of width ``Is``, same format and activation),
    the scalars, and a workspace for up to ``max_tokens`` tokens.  ``layer(x)``
    returns ``(y, topk_idx, topk_w)``.  The workspace is the layer's own: its
    calls must not overlap on the GPU (calls on several streams, or graphs that
    replay at once, each need a layer of their own).  The tensors given here are
    kept, not copied: new values in them count from the next call on, other tensors
    set as fields of ``W`` or ``Ws`` do not.  Where a bounded wait of a call runs out
    (``moe_device_error`` 2), its outputs are undefined; the next call is not affected.
    """

    def __init__(self, W: ExpertWeights, w_router=None, expert_bias=None, *, E: int, k: int, I: int,
                 Ws: Optional[ExpertWeights] = None, Is: int = 0, eps: float = 1e-6, router_scale: float = 1.0,
                 out_scale: float = 1.0, score: str = "sigmoid", norm_topk: bool = True,
                 max_tokens: int = abi.MOE_DECODE_MAX_T):
        if W.w2.dim() != 3 or not W.w2.is_cuda:
            raise ValueError("w2: expected (E, H, ...) on a CUDA device")
        self.device = dev = W.w2.device
        self.H, self.E, self.k, self.I = W.w2.shape[1], E, k, I
        if (Ws is None) != (Is == 0):
            raise ValueError("give Ws and Is together")
        _want("w_router", w_router, (E, self.H), (torch.float32,), dev)
        _want("expert_bias", expert_bias, (E,), (torch.float32,), dev)
        _check_weights("W", W, E, I, self.H, dev)
        if Ws is not None:
            _check_weights("Ws", Ws, 1, Is, self.H, dev)
        # the tensors themselves: W's and Ws' fields may be set to others later
        given = [w_router, expert_bias] + [getattr(w, f.name) for w in (W, Ws) if w for f in dataclasses.fields(w)]
        self._tensors = [t for t in given if isinstance(t, torch.Tensor)]
        self.max_tokens = max_tokens
        d = abi.moe_dims(max_tokens, self.H, E, k, I)
        n = moe_decode_workspace_bytes(d, Is)
        if n == 0:
            raise ValueError(f"sizes of the layer: {moe_last_error()}")
        self.ws = torch.zeros(n, dtype=torch.uint8, device=dev)   # counts in the first 1 KB start at zero
        with torch.cuda.device(dev):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()         # the first call may be on any stream
        self._seen = set()                                        # streams that the allocator knows of
        self._layer = abi.moe_layer(_ptr(w_router), _ptr(expert_bias), W.c_struct(),
                                    Ws.c_struct() if Ws is not None else abi.moe_experts_w(), Is, eps, router_scale,
                                    out_scale, router_cfg(score, norm_topk))
        self._plans = {}
        self._run = load().moe_decode_run
        self._plan(max_tokens)

    def _plan(self, T: int):
        """The prepared call for T tokens: (plan, reference to it, templates of the outputs)."""
        plan = abi.moe_decode_plan()
        d = abi.moe_dims(T, self.H, self.E, self.k, self.I)
        with torch.cuda.device(self.device):
            check(load().moe_decode_prepare(ctypes.byref(self._layer), ctypes.byref(d), ctypes.byref(plan)), "moe_decode")
            idx = torch.empty((T, self.k), dtype=torch.int32, device=self.device)
        self._plans[T] = (plan, ctypes.byref(plan), idx, idx.view(torch.float32))
        return self._plans[T]

    def __call__(self, x, *, residual=None, logits=None, y=None, topk_idx=None, topk_w=None, stream=None):
        if stream is not None:
            with _alloc_on(stream, self.device):
                return self(x, residual=residual, logits=logits, y=y, topk_idx=topk_idx, topk_w=topk_w)
        dev, T = self.device, x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens, but the layer was made for max_tokens = {self.max_tokens}")
        _want("x", x, (T, self.H), (torch.bfloat16,), dev)
        if residual is not None:
            _want("residual", residual, (T, self.H), (torch.bfloat16,), dev)
        if logits is not None:
            _want("logits", logits, (T, self.E), (torch.float32,), dev)
        _, plan, like_idx, like_w = self._plans.get(T) or self._plan(T)
        if y is None:
            y = torch.empty_like(x)
        else:
            _want("y", y, (T, self.H), (torch.bfloat16,), dev)
        if topk_idx is None:
            topk_idx = torch.empty_like(like_idx)
        else:
            _want("topk_idx", topk_idx, (T, self.k), (torch.int32,), dev)
        if topk_w is None:
            topk_w = torch.empty_like(like_w)
        else:
            _want("topk_w", topk_w, (T, self.k), (torch.float32,), dev)
        if torch.cuda.current_device() != dev.index:
            with torch.cuda.device(dev):
                st = self._go(plan, x, logits, residual, topk_idx, topk_w, y)
        else:
            st = self._go(plan, x, logits, residual, topk_idx, topk_w, y)
        if st:
            check(st, "moe_decode")
        return y, topk_idx, topk_w

    def _go(self, plan, x, logits, residual, topk_idx, topk_w, y):
        raw = torch._C._cuda_getCurrentRawStream(self.device.index)   # (3 us faster than through a Stream object)
        if raw not in self._seen:                                 # a dropped layer's memory waits for this stream
            s = torch.cuda.ExternalStream(raw, device=self.device)
            for t in (self.ws, *self._tensors):
                t.record_stream(s)
            self._seen.add(raw)
        return self._run(plan, x.data_ptr(), None if logits is None else logits.data_ptr(),
                         None if residual is None else residual.data_ptr(), topk_idx.data_ptr(), topk_w.data_ptr(),
                         y.data_ptr(), self.ws.data_ptr(), self.ws.numel(), raw)


def moe_profile_hook(ev_begin, ev_end, stage: int) -> None:
    """One-shot: the next forward/experts call on this thread records the two
    torch.cuda.Events around `stage`'s kernel (None, None clears)."""
    b = ev_begin.cuda_event if ev_begin is not None else None
    e = ev_end.cuda_event if ev_end is not None else None
    check(load().moe_profile_hook(b, e, stage), "moe_profile_hook")


def moe_last_launch_count() -> int:
    return int(load().moe_last_launch_count())


def moe_set_dispatch(mode: int) -> int:
    return int(load().moe_set_dispatch(mode))


def moe_set_combine(mode: int) -> int:
    return int(load().moe_set_combine(mode))


def moe_device_error(stream=None) -> int:
    code = ctypes.c_int32(0)
    st = load().moe_device_error(ctypes.byref(code), _stream(stream))
    if st not in (abi.MOE_OK, abi.MOE_ERR_DEVICE):
        check(st, "moe_device_error")
    return int(code.value)


def moe_last_error() -> str:
    return load().moe_last_error().decode(errors="replace")


def moe_version() -> str:
    return load().moe_version().decode()
