"""On-GPU MoE token route / layout / dispatch / combine for NVIDIA B200 (sm_100a).

Python binding over the C ABI in include/moe_route07.h.  The functions carry
the ABI's names and only marshal arguments: they check that tensors are CUDA,
contiguous and of the right dtype, allocate outputs with torch when the caller
passes none, and forward data pointers plus torch's current stream.  Every
step of the path runs in the library's kernels.

    shape = MoeShape(tokens=T, hidden=H, experts=E, k=k, ranks=R)
    ws = Workspace(shape)                       # zero-filled device workspace
    ids, gates = moe_route(shape, logits, bias, ws=ws)
    lay = moe_layout(shape, ids, ws=ws)
    xd = moe_dispatch(shape, x, lay.dst_pos, ws=ws)
    ...  experts turn xd into y (same rows) ...
    out = moe_combine(shape, y, lay.dst_pos, gates, ws=ws, residual=x)
    moe_check(ws)                               # raises on a device-side error

The rest of an expert layer, and what a training step takes back through it:

    rule = ScoreRule(func="sigmoid", groups=8, top_groups=4, group_top=2, scale=2.5)
    ids, gates = moe_route_scored(shape, logits, rule, bias, ws=ws)
    h = moe_expert_matmul(shape, xd, w1, lay.counts, lay.expert_off, ws=ws, act="swiglu")
    y = moe_expert_matmul(shape, h, w2, lay.counts, lay.expert_off, ws=ws)
    g = moe_expert_matmul_backward(shape, grad_y, h, w2, lay.counts, lay.expert_off, ws=ws)
    grad_y, grad_gates = moe_combine_backward(shape, grad_out, y, lay.dst_pos, gates, ws=ws)
    grad_logits = moe_route_scored_backward(shape, logits, rule, ids, grad_gates, ws=ws)
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import Optional

import torch

from . import _binding
from ._binding import MoeError, MOE_F_FP8, MOE_F_RENORM, MOE_F_SRC_LAYOUT

__all__ = ["MoeShape", "Workspace", "Layout", "LayoutSrc", "MoeError", "moe_route", "moe_layout",
           "moe_layout_src", "moe_route_limited", "moe_bias_update",
           "moe_layout_remote_first", "moe_route_round_robin",
           "moe_route_layout", "moe_route_layout_dispatch",
           "moe_dispatch", "moe_combine", "moe_get_device_error", "moe_check",
           "moe_layout_rows", "moe_workspace_bytes", "ScoreRule", "ExpertGrads",
           "moe_route_scored", "moe_route_scored_backward", "moe_expert_matmul",
           "moe_expert_matmul_backward", "moe_combine_backward"]


@dataclasses.dataclass(frozen=True)
class MoeShape:
    tokens: int
    hidden: int
    experts: int
    k: int
    ranks: int
    capacity: int = 0
    align: int = 1
    renorm: bool = True
    fp8: bool = False
    src_layout: bool = False  # rows follow the per-source-rank layout (moe_layout_src)

    @property
    def flags(self) -> int:
        return ((MOE_F_RENORM if self.renorm else 0) | (MOE_F_FP8 if self.fp8 else 0)
                | (MOE_F_SRC_LAYOUT if self.src_layout else 0))

    @functools.cached_property
    def _c(self) -> _binding.MoeShapeC:
        return _binding.MoeShapeC(self.tokens, self.hidden, self.experts, self.k, self.ranks,
                                  self.capacity, self.align, self.flags)

    def c(self) -> _binding.MoeShapeC:
        return self._c

    @functools.cached_property
    def rows(self) -> int:
        return moe_layout_rows(self)


def moe_layout_rows(shape: MoeShape) -> int:
    n = _binding.lib().moe_layout_rows(ctypes.byref(shape.c()))
    if n < 0:
        raise MoeError(_binding.MOE_ERR_INVALID_ARG, "moe_layout_rows")
    return int(n)


def moe_workspace_bytes(shape: MoeShape) -> int:
    n = _binding.lib().moe_workspace_bytes(ctypes.byref(shape.c()))
    if n == 0:
        raise MoeError(_binding.MOE_ERR_INVALID_ARG, "moe_workspace_bytes")
    return int(n)


# The current stream's handle without building a torch.cuda.Stream (2 us of a call
# that takes 8); torch builds without it go through the object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device=None) -> int:
    if _raw_stream is None or not isinstance(device, torch.device):
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(torch.cuda.current_device() if device.index is None else device.index)


def _ptr(t: Optional[torch.Tensor], name: str, dtype=None, shape=None) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _check(status: int, what: str):
    if status != _binding.MOE_OK:
        raise MoeError(status, what)


class Workspace:
    """Zero-filled device workspace for the calls of `shape` (or any shape whose
    requirement is not larger)."""

    def __init__(self, shape: MoeShape, device=None):
        self.nbytes = moe_workspace_bytes(shape)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8,
                               device=device if device is not None else "cuda")
        _check(_binding.lib().moe_workspace_init(self.buf.data_ptr(), self.nbytes,
                                                 _stream(self.buf.device)),
               "moe_workspace_init")

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()


@dataclasses.dataclass
class Layout:
    counts: torch.Tensor       # int32 [E]
    expert_off: torch.Tensor   # int32 [E+1]
    rank_off: torch.Tensor     # int32 [R+1]
    rank_counts: torch.Tensor  # int32 [R]
    dst_pos: torch.Tensor      # int32 [T,k]
    src_idx: torch.Tensor      # int32 [N]


def moe_route(shape: MoeShape, logits: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
              ws: Workspace, ids: Optional[torch.Tensor] = None,
              gates: Optional[torch.Tensor] = None):
    T, E, k = shape.tokens, shape.experts, shape.k
    dev = logits.device
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if gates is None:
        gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    st = _binding.lib().moe_route(
        ctypes.byref(shape.c()), _ptr(logits, "logits", torch.float32, (T, E)),
        _ptr(bias, "bias", torch.float32, (E,)), _ptr(ids, "ids", torch.int32, (T, k)),
        _ptr(gates, "gates", torch.float32, (T, k)), ws.ptr, ws.nbytes, _stream(dev))
    _check(st, "moe_route")
    return ids, gates


def moe_route_limited(shape: MoeShape, logits: torch.Tensor, max_ranks: int,
                      bias: Optional[torch.Tensor] = None, *, ws: Workspace,
                      ids: Optional[torch.Tensor] = None, gates: Optional[torch.Tensor] = None):
    """moe_route with each token's experts taken from at most `max_ranks` ranks."""
    T, E, k = shape.tokens, shape.experts, shape.k
    dev = logits.device
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if gates is None:
        gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    st = _binding.lib().moe_route_limited(
        ctypes.byref(shape.c()), _ptr(logits, "logits", torch.float32, (T, E)),
        _ptr(bias, "bias", torch.float32, (E,)), int(max_ranks),
        _ptr(ids, "ids", torch.int32, (T, k)), _ptr(gates, "gates", torch.float32, (T, k)),
        ws.ptr, ws.nbytes, _stream(dev))
    _check(st, "moe_route_limited")
    return ids, gates


def moe_layout_remote_first(shape: MoeShape, ids: torch.Tensor, home_rank: int, *,
                            ws: Workspace, out: Optional[Layout] = None,
                            tile_expert: Optional[torch.Tensor] = None):
    """Layout with the rank slices ordered home+1, ..., home (remote first);
    returns (Layout, tile_expert int32 [N/align])."""
    T, E, k, R = shape.tokens, shape.experts, shape.k, shape.ranks
    N = shape.rows
    dev = ids.device
    i32 = dict(dtype=torch.int32, device=dev)
    if out is None:
        out = Layout(torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(R + 1, **i32),
                     torch.empty(R, **i32), torch.empty((T, k), **i32), torch.empty(N, **i32))
    if tile_expert is None:
        tile_expert = torch.empty(N // shape.align, **i32)
    st = _binding.lib().moe_layout_remote_first(
        ctypes.byref(shape.c()), _ptr(ids, "ids", torch.int32, (T, k)), int(home_rank),
        _ptr(out.counts, "counts", torch.int32, (E,)),
        _ptr(out.expert_off, "expert_off", torch.int32, (E + 1,)),
        _ptr(out.rank_off, "rank_off", torch.int32, (R + 1,)),
        _ptr(out.rank_counts, "rank_counts", torch.int32, (R,)),
        _ptr(out.dst_pos, "dst_pos", torch.int32, (T, k)),
        _ptr(out.src_idx, "src_idx", torch.int32, (N,)),
        _ptr(tile_expert, "tile_expert", torch.int32, (N // shape.align,)),
        ws.ptr, ws.nbytes, _stream(dev))
    _check(st, "moe_layout_remote_first")
    return out, tile_expert


def moe_route_round_robin(shape: MoeShape, *, device=None, ids: Optional[torch.Tensor] = None,
                          gates: Optional[torch.Tensor] = None):
    """The round-robin router: ids[t,j] = (t*k + j) mod E, gates 1/k."""
    T, k = shape.tokens, shape.k
    dev = device if device is not None else (ids.device if ids is not None else "cuda")
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if gates is None:
        gates = torch.empty((T, k), dtype=torch.float32, device=ids.device)
    st = _binding.lib().moe_route_round_robin(
        ctypes.byref(shape.c()), _ptr(ids, "ids", torch.int32, (T, k)),
        _ptr(gates, "gates", torch.float32, (T, k)), _stream(ids.device))
    _check(st, "moe_route_round_robin")
    return ids, gates


def moe_bias_update(shape: MoeShape, counts: torch.Tensor, gamma: float,
                    bias: torch.Tensor) -> torch.Tensor:
    """bias[e] += gamma * sign(T*k/E - counts[e]), in place; returns bias."""
    E = shape.experts
    st = _binding.lib().moe_bias_update(
        ctypes.byref(shape.c()), _ptr(counts, "counts", torch.int32, (E,)), float(gamma),
        _ptr(bias, "bias", torch.float32, (E,)), _stream(bias.device))
    _check(st, "moe_bias_update")
    return bias


def moe_layout(shape: MoeShape, ids: torch.Tensor, *, ws: Workspace,
               out: Optional[Layout] = None) -> Layout:
    T, E, k, R = shape.tokens, shape.experts, shape.k, shape.ranks
    N = shape.rows
    dev = ids.device
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = Layout(torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(R + 1, **i32),
                     torch.empty(R, **i32), torch.empty((T, k), **i32), torch.empty(N, **i32))
    st = _binding.lib().moe_layout(
        ctypes.byref(shape.c()), _ptr(ids, "ids", torch.int32, (T, k)),
        _ptr(out.counts, "counts", torch.int32, (E,)),
        _ptr(out.expert_off, "expert_off", torch.int32, (E + 1,)),
        _ptr(out.rank_off, "rank_off", torch.int32, (R + 1,)),
        _ptr(out.rank_counts, "rank_counts", torch.int32, (R,)),
        _ptr(out.dst_pos, "dst_pos", torch.int32, (T, k)),
        _ptr(out.src_idx, "src_idx", torch.int32, (N,)), ws.ptr, ws.nbytes, _stream(dev))
    _check(st, "moe_layout")
    return out


@dataclasses.dataclass
class LayoutSrc:
    src_counts: torch.Tensor   # int32 [R,E]   per (source shard, expert)
    seg_off: torch.Tensor      # int32 [R*E+1] segments in (rank, shard, expert) order
    pair_counts: torch.Tensor  # int32 [R,R]   [source shard][destination rank]
    rank_off: torch.Tensor     # int32 [R+1]
    rank_counts: torch.Tensor  # int32 [R]
    dst_pos: torch.Tensor      # int32 [T,k]
    src_idx: torch.Tensor      # int32 [N]


def moe_layout_src(shape: MoeShape, ids: torch.Tensor, *, ws: Workspace,
                   out: Optional[LayoutSrc] = None) -> LayoutSrc:
    """Per-source-rank layout (shape.src_layout must be set)."""
    T, E, k, R = shape.tokens, shape.experts, shape.k, shape.ranks
    N = shape.rows
    dev = ids.device
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = LayoutSrc(torch.empty((R, E), **i32), torch.empty(R * E + 1, **i32),
                        torch.empty((R, R), **i32), torch.empty(R + 1, **i32),
                        torch.empty(R, **i32), torch.empty((T, k), **i32),
                        torch.empty(N, **i32))
    st = _binding.lib().moe_layout_src(
        ctypes.byref(shape.c()), _ptr(ids, "ids", torch.int32, (T, k)),
        _ptr(out.src_counts, "src_counts", torch.int32, (R, E)),
        _ptr(out.seg_off, "seg_off", torch.int32, (R * E + 1,)),
        _ptr(out.pair_counts, "pair_counts", torch.int32, (R, R)),
        _ptr(out.rank_off, "rank_off", torch.int32, (R + 1,)),
        _ptr(out.rank_counts, "rank_counts", torch.int32, (R,)),
        _ptr(out.dst_pos, "dst_pos", torch.int32, (T, k)),
        _ptr(out.src_idx, "src_idx", torch.int32, (N,)), ws.ptr, ws.nbytes, _stream(dev))
    _check(st, "moe_layout_src")
    return out


def moe_route_layout(shape: MoeShape, logits: torch.Tensor, bias: Optional[torch.Tensor] = None,
                     *, ws: Workspace, ids: Optional[torch.Tensor] = None,
                     gates: Optional[torch.Tensor] = None, out: Optional[Layout] = None):
    """moe_route then moe_layout in one launch; returns (ids, gates, Layout)."""
    T, E, k, R = shape.tokens, shape.experts, shape.k, shape.ranks
    N = shape.rows
    dev = logits.device
    i32 = dict(dtype=torch.int32, device=dev)
    if ids is None:
        ids = torch.empty((T, k), **i32)
    if gates is None:
        gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    if out is None:
        out = Layout(torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(R + 1, **i32),
                     torch.empty(R, **i32), torch.empty((T, k), **i32), torch.empty(N, **i32))
    st = _binding.lib().moe_route_layout(
        ctypes.byref(shape.c()), _ptr(logits, "logits", torch.float32, (T, E)),
        _ptr(bias, "bias", torch.float32, (E,)), _ptr(ids, "ids", torch.int32, (T, k)),
        _ptr(gates, "gates", torch.float32, (T, k)),
        _ptr(out.counts, "counts", torch.int32, (E,)),
        _ptr(out.expert_off, "expert_off", torch.int32, (E + 1,)),
        _ptr(out.rank_off, "rank_off", torch.int32, (R + 1,)),
        _ptr(out.rank_counts, "rank_counts", torch.int32, (R,)),
        _ptr(out.dst_pos, "dst_pos", torch.int32, (T, k)),
        _ptr(out.src_idx, "src_idx", torch.int32, (N,)), ws.ptr, ws.nbytes, _stream(dev))
    _check(st, "moe_route_layout")
    return ids, gates, out


def _dispatch_out(shape: MoeShape, dev, out, scales):
    N, H = shape.rows, shape.hidden
    if shape.fp8:
        if out is None:
            out = torch.empty((N, H), dtype=torch.float8_e4m3fn, device=dev)
        if scales is None:
            scales = torch.empty((N, H // 128), dtype=torch.float32, device=dev)
        return out, scales, _ptr(out, "out", torch.float8_e4m3fn, (N, H)), \
            _ptr(scales, "scales", torch.float32, (N, H // 128))
    if out is None:
        out = torch.empty((N, H), dtype=torch.bfloat16, device=dev)
    return out, None, _ptr(out, "out", torch.bfloat16, (N, H)), None


def moe_route_layout_dispatch(shape: MoeShape, logits: torch.Tensor, x: torch.Tensor,
                              bias: Optional[torch.Tensor] = None, *, ws: Workspace,
                              ids: Optional[torch.Tensor] = None,
                              gates: Optional[torch.Tensor] = None, lay: Optional[Layout] = None,
                              out: Optional[torch.Tensor] = None,
                              scales: Optional[torch.Tensor] = None):
    """Steps 1-4 in one call.  Returns (ids, gates, Layout, dispatched) where
    dispatched is as moe_dispatch returns it."""
    T, E, k, R, H = shape.tokens, shape.experts, shape.k, shape.ranks, shape.hidden
    N = shape.rows
    dev = logits.device
    i32 = dict(dtype=torch.int32, device=dev)
    if ids is None:
        ids = torch.empty((T, k), **i32)
    if gates is None:
        gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    if lay is None:
        lay = Layout(torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(R + 1, **i32),
                     torch.empty(R, **i32), torch.empty((T, k), **i32), torch.empty(N, **i32))
    out, scales, optr, sptr = _dispatch_out(shape, dev, out, scales)
    st = _binding.lib().moe_route_layout_dispatch(
        ctypes.byref(shape.c()), _ptr(logits, "logits", torch.float32, (T, E)),
        _ptr(bias, "bias", torch.float32, (E,)), _ptr(x, "x", torch.bfloat16, (T, H)),
        _ptr(ids, "ids", torch.int32, (T, k)), _ptr(gates, "gates", torch.float32, (T, k)),
        _ptr(lay.counts, "counts", torch.int32, (E,)),
        _ptr(lay.expert_off, "expert_off", torch.int32, (E + 1,)),
        _ptr(lay.rank_off, "rank_off", torch.int32, (R + 1,)),
        _ptr(lay.rank_counts, "rank_counts", torch.int32, (R,)),
        _ptr(lay.dst_pos, "dst_pos", torch.int32, (T, k)),
        _ptr(lay.src_idx, "src_idx", torch.int32, (N,)), optr, sptr, ws.ptr, ws.nbytes,
        _stream(dev))
    _check(st, "moe_route_layout_dispatch")
    return ids, gates, lay, ((out, scales) if shape.fp8 else out)


def moe_dispatch(shape: MoeShape, x: torch.Tensor, dst_pos: torch.Tensor, *, ws: Workspace,
                 out: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """bf16: returns out [N,H] bf16.  FP8: returns (codes [N,H] float8_e4m3fn,
    scales [N,H/128] fp32).  Rows no assignment maps to are left as allocated."""
    T, H, k = shape.tokens, shape.hidden, shape.k
    N = shape.rows
    dev = x.device
    if shape.fp8:
        if out is None:
            out = torch.empty((N, H), dtype=torch.float8_e4m3fn, device=dev)
        if scales is None:
            scales = torch.empty((N, H // 128), dtype=torch.float32, device=dev)
        optr = _ptr(out, "out", torch.float8_e4m3fn, (N, H))
        sptr = _ptr(scales, "scales", torch.float32, (N, H // 128))
    else:
        if out is None:
            out = torch.empty((N, H), dtype=torch.bfloat16, device=dev)
        optr = _ptr(out, "out", torch.bfloat16, (N, H))
        sptr = None
    st = _binding.lib().moe_dispatch(
        ctypes.byref(shape.c()), _ptr(x, "x", torch.bfloat16, (T, H)),
        _ptr(dst_pos, "dst_pos", torch.int32, (T, k)), optr, sptr, ws.ptr, ws.nbytes,
        _stream(dev))
    _check(st, "moe_dispatch")
    return (out, scales) if shape.fp8 else out


def moe_combine(shape: MoeShape, y: torch.Tensor, dst_pos: torch.Tensor, gates: torch.Tensor, *,
                ws: Workspace, shared: Optional[torch.Tensor] = None,
                residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    T, H, k = shape.tokens, shape.hidden, shape.k
    N = shape.rows
    dev = y.device
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    st = _binding.lib().moe_combine(
        ctypes.byref(shape.c()), _ptr(y, "y", torch.bfloat16, (N, H)),
        _ptr(dst_pos, "dst_pos", torch.int32, (T, k)),
        _ptr(gates, "gates", torch.float32, (T, k)),
        _ptr(shared, "shared", torch.bfloat16, (T, H)),
        _ptr(residual, "residual", torch.bfloat16, (T, H)),
        _ptr(out, "out", torch.bfloat16, (T, H)), ws.ptr, ws.nbytes, _stream(dev))
    _check(st, "moe_combine")
    return out


def _run(what: str, ws: Workspace, tensors, call):
    """call(stream) on the workspace's device, which every tensor must be on; that
    device is made current for the launch where it is not already."""
    dev = ws.buf.device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"every tensor must be on the workspace's device {dev}, got {t.device}")
    if dev.index == torch.cuda.current_device():
        st = call(_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = call(_stream(dev))
    if st != _binding.MOE_OK:
        raise MoeError(st, what)


@dataclasses.dataclass(frozen=True)
class ScoreRule:
    """How moe_route_scored scores and chooses: `func` "softmax" or "sigmoid";
    each token keeps the `top_groups` best of `groups` groups of experts, a
    group scored by the sum of its `group_top` (1 or 2) largest keys; the gates
    are multiplied by `scale`."""
    func: str = "softmax"
    groups: int = 1
    top_groups: int = 1
    group_top: int = 1
    scale: float = 1.0

    @functools.cached_property
    def _c(self) -> _binding.MoeScoreC:
        if self.func not in _binding.MOE_SCORES:
            raise ValueError(f"func must be one of {sorted(_binding.MOE_SCORES)}, got {self.func!r}")
        return _binding.MoeScoreC(_binding.MOE_SCORES[self.func], self.groups, self.top_groups,
                                  self.group_top, self.scale)

    def c(self) -> _binding.MoeScoreC:
        return self._c


def moe_route_scored(shape: MoeShape, logits: torch.Tensor, rule: ScoreRule,
                     bias: Optional[torch.Tensor] = None, *, ws: Workspace,
                     ids: Optional[torch.Tensor] = None, gates: Optional[torch.Tensor] = None):
    """Top-k by sigmoid or softmax scores plus bias, among the best groups of
    experts; returns (ids int32 [T,k], gates fp32 [T,k])."""
    T, E, k = shape.tokens, shape.experts, shape.k
    dev = logits.device
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if gates is None:
        gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    _run("moe_route_scored", ws, (logits, bias, ids, gates),
         lambda stream: _binding.lib().moe_route_scored(
             ctypes.byref(shape.c()), _ptr(logits, "logits", torch.float32, (T, E)),
             _ptr(bias, "bias", torch.float32, (E,)), ctypes.byref(rule.c()),
             _ptr(ids, "ids", torch.int32, (T, k)), _ptr(gates, "gates", torch.float32, (T, k)),
             ws.ptr, ws.nbytes, stream))
    return ids, gates


def moe_route_scored_backward(shape: MoeShape, logits: torch.Tensor, rule: ScoreRule,
                              ids: torch.Tensor, grad_gates: torch.Tensor, *, ws: Workspace,
                              grad_logits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the logits through moe_route_scored's gates, fp32 [T,E]."""
    T, E, k = shape.tokens, shape.experts, shape.k
    if grad_logits is None:
        grad_logits = torch.empty((T, E), dtype=torch.float32, device=logits.device)
    _run("moe_route_scored_backward", ws, (logits, ids, grad_gates, grad_logits),
         lambda stream: _binding.lib().moe_route_scored_backward(
             ctypes.byref(shape.c()), _ptr(logits, "logits", torch.float32, (T, E)),
             ctypes.byref(rule.c()), _ptr(ids, "ids", torch.int32, (T, k)),
             _ptr(grad_gates, "grad_gates", torch.float32, (T, k)),
             _ptr(grad_logits, "grad_logits", torch.float32, (T, E)), ws.ptr, ws.nbytes, stream))
    return grad_logits


def _act(act: str) -> int:
    if act not in _binding.MOE_ACTS:
        raise ValueError(f"act must be one of {sorted(_binding.MOE_ACTS)}, got {act!r}")
    return _binding.MOE_ACTS[act]


def _features(w: torch.Tensor, E: int, act: str):
    """(in_features, out_features, Wd) of a weight tensor [E, Wd, in_features]."""
    if w.dim() != 3 or w.shape[0] != E:
        raise ValueError(f"w must have shape [{E}, features, in_features], got {tuple(w.shape)}")
    wide = w.shape[1]
    if act == "swiglu":
        if wide % 2:
            raise ValueError("swiglu needs w with gate and up halves: an even number of rows")
        return w.shape[2], wide // 2, wide
    return w.shape[2], wide, wide


def moe_expert_matmul(shape: MoeShape, x: torch.Tensor, w: torch.Tensor,
                      counts: Optional[torch.Tensor] = None,
                      expert_off: Optional[torch.Tensor] = None, *, ws: Workspace,
                      bias: Optional[torch.Tensor] = None, act: str = "none",
                      residual: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None,
                      pre: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act(x[p] W_e^T + bias_e) + residual[p] for every row p that holds a token
    of expert e, bf16 [N, F].  x bf16 [N, K]; w bf16 [E, F, K], or [E, 2F, K]
    with act "swiglu" (gate rows, then up rows); counts and expert_off from the
    layout, or neither for a dense product (one expert, every row).  `pre` bf16
    [N, F or 2F] receives the pre-activations that the backward call reads.
    Rows that hold no token are left as they are."""
    a = _act(act)
    E, N = shape.experts, shape.rows
    K, F, wide = _features(w, E, act)
    bf16 = torch.bfloat16
    if out is None:
        out = torch.empty((N, F), dtype=bf16, device=x.device)
    _run("moe_expert_matmul", ws, (x, w, counts, expert_off, bias, residual, out, pre),
         lambda stream: _binding.lib().moe_expert_matmul(
             ctypes.byref(shape.c()), K, F, a, _ptr(x, "x", bf16, (N, K)), _ptr(w, "w", bf16),
             _ptr(bias, "bias", torch.float32, (E, wide)),
             _ptr(counts, "counts", torch.int32, (E,)),
             _ptr(expert_off, "expert_off", torch.int32, (E + 1,)),
             _ptr(residual, "residual", bf16, (N, F)), _ptr(out, "out", bf16, (N, F)),
             _ptr(pre, "pre", bf16, (N, wide)), ws.ptr, ws.nbytes, stream))
    return out


@dataclasses.dataclass
class ExpertGrads:
    grad_x: Optional[torch.Tensor]     # bf16 [N, K]
    grad_w: Optional[torch.Tensor]     # bf16 [E, Wd, K]
    grad_bias: Optional[torch.Tensor]  # fp32 [E, Wd]
    grad_pre: Optional[torch.Tensor]   # bf16 [N, Wd] (None with act "none")


def moe_expert_matmul_backward(shape: MoeShape, grad_out: torch.Tensor, x: torch.Tensor,
                               w: torch.Tensor, counts: Optional[torch.Tensor] = None,
                               expert_off: Optional[torch.Tensor] = None, *, ws: Workspace,
                               act: str = "none", pre: Optional[torch.Tensor] = None,
                               need_x: bool = True, need_w: bool = True, need_bias: bool = False,
                               grad_pre: Optional[torch.Tensor] = None,
                               grad_x: Optional[torch.Tensor] = None,
                               grad_w: Optional[torch.Tensor] = None,
                               grad_bias: Optional[torch.Tensor] = None) -> ExpertGrads:
    """Gradients of moe_expert_matmul: of x, w and the bias (each where asked
    for, or where a buffer is given), with `pre` as the forward call wrote it.
    The residual's gradient is grad_out.  Rows of grad_x and grad_pre that hold
    no token are left as they are."""
    a = _act(act)
    E, N = shape.experts, shape.rows
    K, F, wide = _features(w, E, act)
    dev, bf16 = x.device, torch.bfloat16
    if grad_x is None and need_x:
        grad_x = torch.empty((N, K), dtype=bf16, device=dev)
    if grad_w is None and need_w:
        grad_w = torch.empty((E, wide, K), dtype=bf16, device=dev)
    if grad_bias is None and need_bias:
        grad_bias = torch.empty((E, wide), dtype=torch.float32, device=dev)
    if act == "none":
        pre = grad_pre = None
    elif grad_pre is None:
        grad_pre = torch.empty((N, wide), dtype=bf16, device=dev)
    scratch, nbytes = None, 0
    if grad_bias is not None:
        nbytes = _binding.lib().moe_expert_matmul_backward_scratch_bytes(ctypes.byref(shape.c()),
                                                                         F, a)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _run("moe_expert_matmul_backward", ws,
         (grad_out, x, w, counts, expert_off, pre, grad_pre, grad_x, grad_w, grad_bias),
         lambda stream: _binding.lib().moe_expert_matmul_backward(
             ctypes.byref(shape.c()), K, F, a, _ptr(grad_out, "grad_out", bf16, (N, F)),
             _ptr(x, "x", bf16, (N, K)), _ptr(w, "w", bf16), _ptr(pre, "pre", bf16, (N, wide)),
             _ptr(counts, "counts", torch.int32, (E,)),
             _ptr(expert_off, "expert_off", torch.int32, (E + 1,)),
             _ptr(grad_pre, "grad_pre", bf16, (N, wide)), _ptr(grad_x, "grad_x", bf16, (N, K)),
             _ptr(grad_w, "grad_w", bf16, (E, wide, K)),
             _ptr(grad_bias, "grad_bias", torch.float32, (E, wide)),
             None if scratch is None else scratch.data_ptr(), nbytes, ws.ptr, ws.nbytes, stream))
    return ExpertGrads(grad_x, grad_w, grad_bias, grad_pre)


def moe_combine_backward(shape: MoeShape, grad_out: torch.Tensor, y: torch.Tensor,
                         dst_pos: torch.Tensor, gates: torch.Tensor, *, ws: Workspace,
                         grad_y: Optional[torch.Tensor] = None,
                         grad_gates: Optional[torch.Tensor] = None):
    """Gradients of moe_combine: (grad_y bf16 [N,H], grad_gates fp32 [T,k]).
    Rows of grad_y that no slot maps to are left as they are; the gradients of
    shared and residual are grad_out.  (The gradient of moe_dispatch is
    moe_combine with gates of one.)"""
    T, H, k = shape.tokens, shape.hidden, shape.k
    N = shape.rows
    if grad_y is None:
        grad_y = torch.empty((N, H), dtype=torch.bfloat16, device=y.device)
    if grad_gates is None:
        grad_gates = torch.empty((T, k), dtype=torch.float32, device=y.device)
    _run("moe_combine_backward", ws, (grad_out, y, dst_pos, gates, grad_y, grad_gates),
         lambda stream: _binding.lib().moe_combine_backward(
             ctypes.byref(shape.c()), _ptr(grad_out, "grad_out", torch.bfloat16, (T, H)),
             _ptr(y, "y", torch.bfloat16, (N, H)), _ptr(dst_pos, "dst_pos", torch.int32, (T, k)),
             _ptr(gates, "gates", torch.float32, (T, k)),
             _ptr(grad_y, "grad_y", torch.bfloat16, (N, H)),
             _ptr(grad_gates, "grad_gates", torch.float32, (T, k)), ws.ptr, ws.nbytes, stream))
    return grad_y, grad_gates


def moe_get_device_error(ws: Workspace):
    """Synchronise the current stream; return (status, detail) of the first
    device-side error since the last read, and clear it."""
    detail = ctypes.c_int32(0)
    st = _binding.lib().moe_get_device_error(ws.ptr, ctypes.byref(detail),
                                             _stream(ws.buf.device))
    return int(st), int(detail.value)


def moe_check(ws: Workspace):
    st, detail = moe_get_device_error(ws)
    if st != _binding.MOE_OK:
        raise MoeError(st, "device", detail)
