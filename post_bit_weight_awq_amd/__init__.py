"""MI355X (gfx950) AWQ per-layer search: thin Python binding of libawq_mi355x.

The functions below only marshal torch tensors into the C ABI declared in
include/awq_mi355x.h; every step of the path runs in the library's HIP
kernels on the tensors' device, on torch's current stream.  torch provides
device memory and streams, nothing else.  There is no CPU fallback: without
the built library the calls raise.

    sal = awq_act_stats(X)                          # step 1
    res = awq_search_layer(X, W, sal)               # steps 2-5: losses, i*, s*
    qweight, step, zero = awq_pack(W, res.s_best)   # codes of W diag(s*)
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import operator
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import AwqConfig, AwqError, AwqKv4Cache, AwqSearchPlan, check, load  # noqa: F401
from ._lib import STAGE_ALL, STAGE_GRID, STAGE_PREPARE, STAGE_SELECT  # noqa: F401

__all__ = ["AwqConfig", "AwqError", "default_config", "awq_act_stats", "awq_act_stats_noalloc",
           "awq_act_stats_workspace_size", "awq_search_plan", "awq_search_workspace_size",
           "awq_search_layer", "awq_pack", "awq_w4a16_matmul", "awq_fold_inverse_scale", "awq_select_top_channels", "awq_weight_saliency",
           "awq_w4a16_linear", "awq_w4a16_gated", "awq_w4a16_input_grad", "awq_w4a16_gated_backward",
           "awq_w4a16_param_grad", "awq_w4a16_adapted", "awq_w4a16_adapted_backward", "Kv4Cache", "awq_kv4_cache", "awq_kv4_append", "awq_kv4_gather",
           "awq_kv4_attention", "SearchResult", "load"]


def default_config(n_grid: int = 20, sal_floor: float = 1e-4, *, group_size: int = 128,
                   w_bit: int = 4, zero_point: bool = True) -> AwqConfig:
    """The method's settings (4-bit, groups of 128, zero point, 20 grid points,
    floor 1e-4); the keywords select the ablation variants the library has."""
    cfg = AwqConfig()
    load().awq_default_config(ctypes.byref(cfg))
    cfg.n_grid = n_grid
    cfg.sal_floor = sal_floor
    cfg.group_size = group_size
    cfg.w_bit = w_bit
    cfg.zero_point = 1 if zero_point else 0
    return cfg


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _on(stream):
    """Context in which the binding allocates its outputs and workspaces: the
    stream the kernels run on, so torch's caching allocator hands the memory
    to no other stream while they may still be pending."""
    return torch.cuda.stream(stream) if stream is not None else _NOTHING


_NOTHING = contextlib.nullcontext()


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype, shape) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# ------------------------------------------------------------------- stats
def awq_act_stats_workspace_size(n_tokens: int, in_features: int) -> int:
    n = load().awq_act_stats_workspace_size(n_tokens, in_features)
    if n == 0:
        raise AwqError(_lib.AWQ_ERR_INVALID_ARG, f"bad shape ({n_tokens}, {in_features})")
    return n


def awq_act_stats(X: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """sal[k] = mean_t |X[t, k]| as fp32, exact sum (X: [tokens, in] fp16)."""
    if X.dim() != 2:
        raise ValueError("X must be [tokens, in_features]")
    n, k = X.shape
    with _on(stream):
        if out is None:
            out = torch.empty(k, dtype=torch.float32, device=X.device)
        if workspace is None:
            workspace = torch.empty(awq_act_stats_workspace_size(n, k), dtype=torch.uint8,
                                    device=X.device)
    check(load().awq_act_stats(
        ctypes.c_void_p(_dev(X, "X", torch.float16, (n, k))), n, k,
        ctypes.c_void_p(_dev(out, "out", torch.float32, (k,))),
        ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return out


def awq_act_stats_noalloc(X: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """The same saliency through the entry point that allocates nothing (its
    partials go to a fixed per-GPU scratch; overlapping calls on one GPU race).
    Only ``out``, when not given, is allocated here."""
    if X.dim() != 2:
        raise ValueError("X must be [tokens, in_features]")
    n, k = X.shape
    with _on(stream):
        if out is None:
            out = torch.empty(k, dtype=torch.float32, device=X.device)
    check(load().awq_act_stats_noalloc(
        ctypes.c_void_p(_dev(X, "X", torch.float16, (n, k))), n, k,
        ctypes.c_void_p(_dev(out, "out", torch.float32, (k,))), _stream(stream)))
    return out


# ------------------------------------------------------------------ search
def awq_search_plan(n_tokens: int, in_features: int, out_features: int,
                    cfg: Optional[AwqConfig] = None) -> AwqSearchPlan:
    cfg = cfg or default_config()
    plan = AwqSearchPlan()
    check(load().awq_search_plan_query(n_tokens, in_features, out_features, ctypes.byref(cfg),
                                       ctypes.byref(plan)))
    return plan


def awq_search_workspace_size(n_tokens: int, in_features: int, out_features: int,
                              cfg: Optional[AwqConfig] = None) -> int:
    return awq_search_plan(n_tokens, in_features, out_features, cfg).workspace_bytes


@dataclass
class SearchResult:
    losses: torch.Tensor     # [n_grid] float64 (device)
    best_idx: torch.Tensor   # [1] int32 (device); -1 when no loss is finite
    s_best: torch.Tensor     # [in] float32 (device)
    workspace: torch.Tensor  # uint8 workspace (tile partial sums, scale table, group parameters)
    plan: AwqSearchPlan

    def best(self) -> int:
        """The chosen grid index after synchronizing with the search's stream;
        raises AwqError(AWQ_ERR_NONFINITE) when no loss was finite."""
        b = int(self.best_idx.item())
        if b < 0:
            raise AwqError(_lib.AWQ_ERR_NONFINITE, "no grid point gave a finite loss")
        return b


def awq_search_layer(X: torch.Tensor, W: torch.Tensor, sal: torch.Tensor,
                     cfg: Optional[AwqConfig] = None, *, workspace: Optional[torch.Tensor] = None,
                     losses: Optional[torch.Tensor] = None, best_idx: Optional[torch.Tensor] = None,
                     s_best: Optional[torch.Tensor] = None, stream=None,
                     stages: int = _lib.STAGE_ALL) -> SearchResult:
    """Alpha-grid search of one layer (X: [tokens, in] fp16, W: [out, in] fp16).

    ``stages`` selects a subset of the prepare / grid / select stages (an OR
    of STAGE_PREPARE, STAGE_GRID, STAGE_SELECT); the stages of one search run
    in that order on one workspace."""
    cfg = cfg or default_config()
    if X.dim() != 2 or W.dim() != 2:
        raise ValueError("X and W must be 2-D")
    n, k = X.shape
    o = W.shape[0]
    plan = awq_search_plan(n, k, o, cfg)
    dev = X.device
    with _on(stream):
        if workspace is None:
            workspace = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=dev)
        if losses is None:
            losses = torch.empty(cfg.n_grid, dtype=torch.float64, device=dev)
        if best_idx is None:
            best_idx = torch.empty(1, dtype=torch.int32, device=dev)
        if s_best is None:
            s_best = torch.empty(k, dtype=torch.float32, device=dev)
    check(load().awq_search_layer_stages(
        stages, ctypes.c_void_p(_dev(X, "X", torch.float16, (n, k))),
        ctypes.c_void_p(_dev(W, "W", torch.float16, (o, k))),
        ctypes.c_void_p(_dev(sal, "sal", torch.float32, (k,))), n, k, o, ctypes.byref(cfg),
        ctypes.c_void_p(_dev(losses, "losses", torch.float64, (cfg.n_grid,))),
        ctypes.c_void_p(_dev(best_idx, "best_idx", torch.int32, (1,))),
        ctypes.c_void_p(_dev(s_best, "s_best", torch.float32, (k,))),
        ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return SearchResult(losses, best_idx, s_best, workspace, plan)


# -------------------------------------------------------------------- pack
def awq_pack(W: torch.Tensor, s: torch.Tensor, cfg: Optional[AwqConfig] = None, *,
             qweight: Optional[torch.Tensor] = None, step: Optional[torch.Tensor] = None,
             zero: Optional[torch.Tensor] = None, stream=None):
    """Codes of W diag(s): (qweight [out, in/8] int32, step [out, in/128] fp16,
    zero [out, in/128] fp16)."""
    cfg = cfg or default_config()
    if W.dim() != 2:
        raise ValueError("W must be [out_features, in_features]")
    o, k = W.shape
    g = cfg.group_size
    dev = W.device
    if k % 8 or k % g:
        raise ValueError(f"in_features={k} must be a multiple of {g}")
    with _on(stream):
        if qweight is None:
            qweight = torch.empty((o, k // 8), dtype=torch.int32, device=dev)
        if step is None:
            step = torch.empty((o, k // g), dtype=torch.float16, device=dev)
        if zero is None:
            zero = torch.empty((o, k // g), dtype=torch.float16, device=dev)
    check(load().awq_pack(
        ctypes.c_void_p(_dev(W, "W", torch.float16, (o, k))),
        ctypes.c_void_p(_dev(s, "s", torch.float32, (k,))), k, o, ctypes.byref(cfg),
        ctypes.c_void_p(_dev(qweight, "qweight", torch.int32, (o, k // 8))),
        ctypes.c_void_p(_dev(step, "step", torch.float16, (o, k // g))),
        ctypes.c_void_p(_dev(zero, "zero", torch.float16, (o, k // g))),
        _stream(stream)))
    return qweight, step, zero


def awq_w4a16_matmul(X: torch.Tensor, qweight: torch.Tensor, step: torch.Tensor,
                     zero: torch.Tensor, *, out: Optional[torch.Tensor] = None, stream=None):
    """Y [n_tokens, out_features] fp32 = X (q - zero) step, with (qweight, step,
    zero) as awq_pack returns them and X [n_tokens, in_features] fp16."""
    if X.dim() != 2 or qweight.dim() != 2:
        raise ValueError("X must be [n_tokens, in_features], qweight [out_features, in_features/8]")
    n, k = X.shape
    o = qweight.shape[0]
    if k % 128:
        raise ValueError(f"in_features={k} must be a multiple of 128")
    with _on(stream):
        if out is None:
            out = torch.empty((n, o), dtype=torch.float32, device=X.device)
    check(load().awq_w4a16_matmul(
        ctypes.c_void_p(_dev(X, "X", torch.float16, (n, k))), n, k, o,
        ctypes.c_void_p(_dev(qweight, "qweight", torch.int32, (o, k // 8))),
        ctypes.c_void_p(_dev(step, "step", torch.float16, (o, k // 128))),
        ctypes.c_void_p(_dev(zero, "zero", torch.float16, (o, k // 128))),
        ctypes.c_void_p(_dev(out, "out", torch.float32, (n, o))),
        _stream(stream)))
    return out


# -------------------------------------------------- packed-weight operators
# A decode call runs for about ten microseconds, so these bindings keep to the
# cheap checks: an argument that is as expected costs a few attribute reads,
# and only one that is not goes through _dev, which says what is wrong.
_DTYPES = {torch.float16: _lib.DTYPE_F16, torch.bfloat16: _lib.DTYPE_BF16}
#: "gelu" is the tanh form here, another name of "gelu_tanh"; the erf form, which torch calls
#: "gelu" (its tanh form is approximate="tanh"), is up to 5e-4 away and not offered
_ACTS = {"silu": _lib.ACT_SILU, "gelu": _lib.ACT_GELU_TANH, "gelu_tanh": _lib.ACT_GELU_TANH}
_REFUSED = ctypes.c_size_t(-1).value


def _w4_tracked(name: str):
    raise RuntimeError(
        f"{name} requires a gradient, and these calls record none: a result would silently be cut "
        "off from it. Call them under torch.no_grad() or inside a torch.autograd.Function, whose "
        "backward calls awq_w4a16_input_grad, awq_w4a16_gated_backward, awq_w4a16_adapted_backward and "
        "awq_w4a16_param_grad")


def _w4_ptr(t, name: str, dtype: torch.dtype, shape, dev: int) -> int:
    """_dev's checks, and that the tensor is on GPU ``dev`` and needs no gradient recorded."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.shape == shape
            and t.is_contiguous()):
        _dev(t, name, dtype, shape)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}: all tensors must be on one device, "
                         f"the current one (cuda:{dev})")
    if t.requires_grad and torch.is_grad_enabled():
        _w4_tracked(name)
    return t.data_ptr()


def _w4_layer(lead: torch.Tensor, name: str, qweight, step, zero):
    """Checks a packed layer against the activations or gradients ``lead`` and
    returns (dtype code, tokens, in_features, rows, group size, the layer's
    pointers, device index)."""
    if not isinstance(lead, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dt = _DTYPES.get(lead.dtype)
    if dt is None:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {lead.dtype}")
    if lead.requires_grad and torch.is_grad_enabled():
        _w4_tracked(name)
    if lead.dim() != 2 or qweight.dim() != 2 or step.dim() != 2:
        raise ValueError(f"{name}, qweight and step must be 2-D")
    o, words = qweight.shape
    k, ng = 8 * words, step.shape[1]
    if ng == 0 or k % ng:
        raise ValueError(f"step has {ng} groups for in_features={k}")
    if not lead.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    dev = torch._C._cuda_getDevice()
    if lead.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{lead.get_device()}, the current device is cuda:{dev}")
    ptrs = (_w4_ptr(qweight, "qweight", torch.int32, (o, words), dev),
            _w4_ptr(step, "step", torch.float16, (o, ng), dev),
            _w4_ptr(zero, "zero", torch.float16, (o, ng), dev))
    return dt, lead.shape[0], k, o, k // ng, ptrs, dev


def _w4_out(t, name: str, dtype: torch.dtype, shape, lead, dev: int):
    """(tensor, pointer) of an output, allocated where the caller gave none."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=lead.device)
        return t, t.data_ptr()
    return t, _w4_ptr(t, name, dtype, shape, dev)


def _w4_workspace(query, sizes, lead, workspace):
    """(tensor, pointer, bytes) of the workspace, allocated where the call needs one."""
    if workspace is None:
        need = query(*sizes)
        if need == 0 or need == _REFUSED:  # the call itself says what it refuses
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=lead.device)
    elif workspace.device != lead.device:
        raise ValueError(f"workspace must be on {lead.device}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _w4_stream(stream, dev: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on cuda:{dev}")
    return stream.cuda_stream


def awq_w4a16_linear(X: torch.Tensor, qweight: torch.Tensor, step: torch.Tensor,
                     zero: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                     out_dtype: Optional[torch.dtype] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = X W^T with the packed layer (qweight, step, zero) of awq_pack, any of
    its group sizes; X [n_tokens, in_features] fp16 or bf16, Y in out_dtype
    (X's type by default, or torch.float32).  awq_w4a16_matmul takes groups of
    128 in fp16 alone; of the two it is faster for one token through up to
    about 5000 rows."""
    lib = load()
    dt, n, k, o, group, layer, dev = _w4_layer(X, "X", qweight, step, zero)
    if out_dtype is None:
        out_dtype = X.dtype if out is None else out.dtype
    if out_dtype is not X.dtype and out_dtype is not torch.float32:
        raise TypeError(f"out_dtype must be {X.dtype} or torch.float32, got {out_dtype}")
    x = _w4_ptr(X, "X", X.dtype, (n, k), dev)
    with _on(stream):
        out, y = _w4_out(out, "out", out_dtype, (n, o), X, dev)
        workspace, ws, size = _w4_workspace(lib.awq_w4a16_linear_workspace_size, (n, k, o, group, dt),
                                            X, workspace)
    rc = lib.awq_w4a16_linear(x, dt, n, k, o, group, *layer, y,
                              _lib.DTYPE_F32 if out_dtype is torch.float32 else dt, ws, size,
                              _w4_stream(stream, dev))
    if rc:
        check(rc)
    return out


def _w4_half(o: int) -> int:
    if o % 2:
        raise ValueError(f"a gated layer has the gate's rows and as many up rows, got {o}")
    return o // 2


def _w4_act(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return _ACTS[act]


def awq_w4a16_gated(X: torch.Tensor, qweight: torch.Tensor, step: torch.Tensor,
                    zero: torch.Tensor, *, act: str = "silu", keep_pre: bool = False,
                    out: Optional[torch.Tensor] = None, pre: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """H = act(X Wg^T) * (X Wu^T) in one kernel; the packed layer holds the
    gate's rows and then the up rows.  act is "silu" or "gelu_tanh",
    g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))), torch's gelu with
    approximate="tanh"; "gelu" is another name of that form, not the erf one.
    With keep_pre (or a pre buffer) returns (H, pre), pre = [G | U] in X's
    type, which the backward pass reads."""
    lib = load()
    dt, n, k, o, group, layer, dev = _w4_layer(X, "X", qweight, step, zero)
    f, code = _w4_half(o), _w4_act(act)
    x = _w4_ptr(X, "X", X.dtype, (n, k), dev)
    p = None
    with _on(stream):
        out, h = _w4_out(out, "out", X.dtype, (n, f), X, dev)
        if keep_pre or pre is not None:
            pre, p = _w4_out(pre, "pre", X.dtype, (n, o), X, dev)
        workspace, ws, size = _w4_workspace(lib.awq_w4a16_gated_workspace_size, (n, k, f, group, dt),
                                            X, workspace)
    rc = lib.awq_w4a16_gated(x, dt, n, k, f, group, code, *layer, h, p, ws, size,
                             _w4_stream(stream, dev))
    if rc:
        check(rc)
    return out if pre is None else (out, pre)


def awq_w4a16_input_grad(dY: torch.Tensor, qweight: torch.Tensor, step: torch.Tensor,
                         zero: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dX = dY W [n_tokens, in_features] in dY's type, the packed codes frozen."""
    lib = load()
    dt, n, k, o, group, layer, dev = _w4_layer(dY, "dY", qweight, step, zero)
    d = _w4_ptr(dY, "dY", dY.dtype, (n, o), dev)
    with _on(stream):
        out, dx = _w4_out(out, "out", dY.dtype, (n, k), dY, dev)
        workspace, ws, size = _w4_workspace(lib.awq_w4a16_input_grad_workspace_size,
                                            (n, k, o, group, dt), dY, workspace)
    rc = lib.awq_w4a16_input_grad(d, dt, n, k, o, group, *layer, dx, ws, size,
                                  _w4_stream(stream, dev))
    if rc:
        check(rc)
    return out


def awq_w4a16_gated_backward(dH: torch.Tensor, pre: torch.Tensor, qweight: torch.Tensor,
                             step: torch.Tensor, zero: torch.Tensor, *, act: str = "silu",
                             out: Optional[torch.Tensor] = None,
                             dpre: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None, stream=None):
    """(dX, dpre) of awq_w4a16_gated (act as there) from the gradient of H and the kept pre;
    dpre = [dG | dU] is what awq_w4a16_param_grad takes as dY."""
    lib = load()
    dt, n, k, o, group, layer, dev = _w4_layer(dH, "dH", qweight, step, zero)
    f, code = _w4_half(o), _w4_act(act)
    d = _w4_ptr(dH, "dH", dH.dtype, (n, f), dev)
    p = _w4_ptr(pre, "pre", dH.dtype, (n, o), dev)
    with _on(stream):
        out, dx = _w4_out(out, "out", dH.dtype, (n, k), dH, dev)
        dpre, dp = _w4_out(dpre, "dpre", dH.dtype, (n, o), dH, dev)
        workspace, ws, size = _w4_workspace(lib.awq_w4a16_gated_backward_workspace_size,
                                            (n, k, f, group, dt), dH, workspace)
    rc = lib.awq_w4a16_gated_backward(d, p, dt, n, k, f, group, code, *layer, dp, dx, ws, size,
                                      _w4_stream(stream, dev))
    if rc:
        check(rc)
    return out, dpre


def awq_w4a16_param_grad(dY: torch.Tensor, X: torch.Tensor, qweight: torch.Tensor,
                         step: torch.Tensor, zero: torch.Tensor, *,
                         dstep: Optional[torch.Tensor] = None,
                         dzero: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """(dstep, dzero), fp32 in step's shape: gradients of the group parameters
    of Y = X W^T for the output gradient dY, the packed codes frozen."""
    lib = load()
    dt, n, k, o, group, layer, dev = _w4_layer(dY, "dY", qweight, step, zero)
    d = _w4_ptr(dY, "dY", dY.dtype, (n, o), dev)
    x = _w4_ptr(X, "X", dY.dtype, (n, k), dev)
    with _on(stream):
        dstep, ds = _w4_out(dstep, "dstep", torch.float32, tuple(step.shape), dY, dev)
        dzero, dz = _w4_out(dzero, "dzero", torch.float32, tuple(step.shape), dY, dev)
        workspace, ws, size = _w4_workspace(lib.awq_w4a16_param_grad_workspace_size,
                                            (n, k, o, group, dt), dY, workspace)
    rc = lib.awq_w4a16_param_grad(d, x, dt, n, k, o, group, *layer, ds, dz, ws, size,
                                  _w4_stream(stream, dev))
    if rc:
        check(rc)
    return dstep, dzero


def _w4_adapters(A, B, scale, adapter, lead, n: int, k: int, o: int, dev: int):
    """Checks a stack of adapters; (count, rank, pointers)."""
    if A.dim() != 3:
        raise ValueError("A must be [adapters, rank, in_features]")
    count, rank = A.shape[0], A.shape[1]
    return count, rank, (_w4_ptr(A, "A", lead.dtype, (count, rank, k), dev),
                         _w4_ptr(B, "B", lead.dtype, (count, o, rank), dev),
                         _w4_ptr(scale, "scale", torch.float32, (count,), dev)), \
        _w4_ptr(adapter, "adapter", torch.int32, (n,), dev)


def awq_w4a16_adapted(X: torch.Tensor, qweight: torch.Tensor, step: torch.Tensor, zero: torch.Tensor,
                      A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor, adapter: torch.Tensor, *,
                      keep_low: bool = False, low: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """Y = X W^T plus each token's own adapter: scale[a] (X A[a]^T) B[a]^T with
    a = adapter[t].  The packed layer and X as awq_w4a16_linear takes them; A
    [adapters, rank, in], B [adapters, out, rank] in X's type, scale [adapters] fp32,
    adapter [tokens] int32 (a negative one: none); rank a multiple of 8 up to 128.
    With keep_low (or a low buffer) returns (Y, low), low = X A^T [tokens, rank] fp32,
    which the backward pass reads."""
    lib = load()
    dt, n, k, o, group, layer, dev = _w4_layer(X, "X", qweight, step, zero)
    if out_dtype is None:
        out_dtype = X.dtype if out is None else out.dtype
    if out_dtype is not X.dtype and out_dtype is not torch.float32:
        raise TypeError(f"out_dtype must be {X.dtype} or torch.float32, got {out_dtype}")
    x = _w4_ptr(X, "X", X.dtype, (n, k), dev)
    count, rank, stack, ids = _w4_adapters(A, B, scale, adapter, X, n, k, o, dev)
    yt = _lib.DTYPE_F32 if out_dtype is torch.float32 else dt
    p = None
    with _on(stream):
        out, y = _w4_out(out, "out", out_dtype, (n, o), X, dev)
        if keep_low or low is not None:
            low, p = _w4_out(low, "low", torch.float32, (n, rank), X, dev)
        workspace, ws, size = _w4_workspace(lib.awq_w4a16_adapted_workspace_size,
                                            (n, k, o, group, dt, yt, count, rank, p is not None), X,
                                            workspace)
    rc = lib.awq_w4a16_adapted(x, dt, n, k, o, group, *layer, *stack, count, rank, ids, y, yt, p, ws,
                               size, _w4_stream(stream, dev))
    if rc:
        check(rc)
    return out if low is None else (out, low)


def awq_w4a16_adapted_backward(dY: torch.Tensor, X: torch.Tensor, low: torch.Tensor,
                               qweight: torch.Tensor, step: torch.Tensor, zero: torch.Tensor,
                               A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                               adapter: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                               dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None, stream=None):
    """(dX, dA, dB) of awq_w4a16_adapted from the gradient of Y and the kept low; dX
    in dY's type, dA and dB fp32 in A's and B's shapes (zeros for an adapter without
    tokens).  The packed layer and the scales are frozen."""
    lib = load()
    dt, n, k, o, group, layer, dev = _w4_layer(dY, "dY", qweight, step, zero)
    d = _w4_ptr(dY, "dY", dY.dtype, (n, o), dev)
    x = _w4_ptr(X, "X", dY.dtype, (n, k), dev)
    count, rank, stack, ids = _w4_adapters(A, B, scale, adapter, dY, n, k, o, dev)
    p = _w4_ptr(low, "low", torch.float32, (n, rank), dev)
    with _on(stream):
        out, dx = _w4_out(out, "out", dY.dtype, (n, k), dY, dev)
        dA, da = _w4_out(dA, "dA", torch.float32, (count, rank, k), dY, dev)
        dB, db = _w4_out(dB, "dB", torch.float32, (count, o, rank), dY, dev)
        workspace, ws, size = _w4_workspace(lib.awq_w4a16_adapted_backward_workspace_size,
                                            (n, k, o, group, dt, count, rank), dY, workspace)
    rc = lib.awq_w4a16_adapted_backward(d, x, p, dt, n, k, o, group, *layer, *stack, count, rank, ids,
                                        dx, da, db, ws, size, _w4_stream(stream, dev))
    if rc:
        check(rc)
    return out, dA, dB


# ------------------------------------------------- key/value cache in 4 bits
class Kv4Cache:
    """The arrays of a 4-bit key/value cache (include/awq_mi355x.h has their
    order): k_codes [n_pages, n_heads, page_size, head_dim / 8] and v_codes
    [n_pages, n_heads, page_size / 16, head_dim / 8, 16] int32, k_params and
    v_params [n_pages, n_heads, page_size, head_dim / group_size, 2] fp16.
    awq_kv4_cache makes one; a program may bring its own memory.  Place
    p * page_size + i is token i of page p.  The arrays are checked here and not
    by each call, so they and the sizes are read-only: a larger cache is another
    object.  Arrays that were resized or replaced in place are refused."""
    __slots__ = ("_k_codes", "_v_codes", "_k_params", "_v_params", "_n_pages", "_n_heads", "_page_size",
                 "_head_dim", "_group_size", "_device", "_ref", "_at")

    k_codes = property(operator.attrgetter("_k_codes"))
    v_codes = property(operator.attrgetter("_v_codes"))
    k_params = property(operator.attrgetter("_k_params"))
    v_params = property(operator.attrgetter("_v_params"))
    n_pages = property(operator.attrgetter("_n_pages"))
    n_heads = property(operator.attrgetter("_n_heads"))
    page_size = property(operator.attrgetter("_page_size"))
    head_dim = property(operator.attrgetter("_head_dim"))
    group_size = property(operator.attrgetter("_group_size"))

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_params: torch.Tensor,
                 v_params: torch.Tensor):
        p, h, s, w = k_codes.shape
        if k_params.dim() != 5 or not k_params.shape[3] or 8 * w % k_params.shape[3]:
            raise ValueError(f"k_params {tuple(k_params.shape)} does not fit k_codes {tuple(k_codes.shape)}")
        g = k_params.shape[3]
        device = k_codes.device
        for name, t, dtype, shape in (("k_codes", k_codes, torch.int32, (p, h, s, w)),
                                      ("v_codes", v_codes, torch.int32, (p, h, s // 16, w, 16)),
                                      ("k_params", k_params, torch.float16, (p, h, s, g, 2)),
                                      ("v_params", v_params, torch.float16, (p, h, s, g, 2))):
            if t.dtype is not dtype:
                raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
            if t.shape != shape:
                raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if t.device != device:
                raise ValueError(f"{name} is on {t.device}, k_codes on {device}")
        self._k_codes, self._v_codes, self._k_params, self._v_params = k_codes, v_codes, k_params, v_params
        self._n_pages, self._n_heads, self._page_size = p, h, s
        self._head_dim, self._group_size = 8 * w, 8 * w // g
        self._device = device.index if device.type == "cuda" else -1
        self._at = (k_codes.data_ptr(), v_codes.data_ptr(), k_params.data_ptr(), v_params.data_ptr())
        self._ref = ctypes.byref(AwqKv4Cache(*self._at, p, h, s, 8 * w, 8 * w // g))


def awq_kv4_cache(n_pages: int, n_heads: int, page_size: int, head_dim: int, group_size: int = 64,
                  *, device="cuda") -> Kv4Cache:
    """An empty cache: page_size 16, 32, 64 or 128; head_dim 64 or 128; groups of
    32, 64 or 128 columns.  0.5 + 4 / group_size bytes for each key and value."""
    if page_size not in (16, 32, 64, 128) or head_dim not in (64, 128) \
            or group_size not in (32, 64, 128) or group_size > head_dim:
        raise AwqError(_lib.AWQ_ERR_UNSUPPORTED, f"page_size={page_size} (16, 32, 64, 128), head_dim="
                       f"{head_dim} (64, 128), group_size={group_size} (32, 64, 128, at most head_dim)")
    if n_pages < 1 or n_heads < 1 or n_heads > 1024 or n_pages * page_size >= 2 ** 31:
        raise AwqError(_lib.AWQ_ERR_INVALID_ARG, f"n_pages={n_pages}, n_heads={n_heads}")
    w, g = head_dim // 8, head_dim // group_size
    return Kv4Cache(
        torch.zeros((n_pages, n_heads, page_size, w), dtype=torch.int32, device=device),
        torch.zeros((n_pages, n_heads, page_size // 16, w, 16), dtype=torch.int32, device=device),
        torch.zeros((n_pages, n_heads, page_size, g, 2), dtype=torch.float16, device=device),
        torch.zeros((n_pages, n_heads, page_size, g, 2), dtype=torch.float16, device=device))


def _kv4(cache: Kv4Cache, dev: int):
    """The C struct of a cache on GPU ``dev``."""
    if not isinstance(cache, Kv4Cache):
        raise TypeError("cache must be a Kv4Cache")
    if cache._device != dev:
        if cache._device < 0:
            raise ValueError("cache must be on the GPU")
        raise ValueError(f"cache is on cuda:{cache._device}, the current device is cuda:{dev}")
    if (cache._k_codes.data_ptr(), cache._v_codes.data_ptr(), cache._k_params.data_ptr(),
            cache._v_params.data_ptr()) != cache._at:
        raise ValueError("the cache's arrays have moved since it was made: make another Kv4Cache of them")
    return cache._ref


def _kv4_rows(t, name: str, heads, dim: int, dtype, dev: int):
    """(pointer, tokens, heads, token stride, head stride) of [tokens, heads, dim]
    rows, whose strides may be a slice's; heads None: any number."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype is not dtype):
        raise TypeError(f"{name} must be {dtype or 'torch.float16 or torch.bfloat16'}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {dim}], got {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")
    if t.requires_grad and torch.is_grad_enabled():
        _w4_tracked(name)
    n, h, _ = shape
    ts, hs, ds = t.stride()
    if ds != 1:
        raise ValueError(f"{name}'s last dimension must be dense")
    # a dimension of one row has no stride of its own
    return t.data_ptr(), n, h, ts if n > 1 else 0, hs if h > 1 else 0


def _kv4_device(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    return torch._C._cuda_getDevice()


@functools.lru_cache(maxsize=1024)
def _kv4_attention_need(pages: int, heads: int, page: int, dim: int, group: int, n: int, h: int, seqs: int,
                        per: int, ragged: bool) -> int:
    """awq_kv4_attention_workspace_size, which depends on the sizes alone."""
    c = AwqKv4Cache(None, None, None, None, pages, heads, page, dim, group)
    return load().awq_kv4_attention_workspace_size(ctypes.byref(c), n, h, seqs, per, ragged)


def awq_kv4_append(k: torch.Tensor, v: torch.Tensor, cache: Kv4Cache, slots: torch.Tensor, *,
                   stream=None) -> None:
    """Quantizes the keys and values of some tokens ([tokens, n_heads, head_dim]
    fp16 or bf16, slices of a fused projection's output too) into their places,
    slots [tokens] int32.  A token with a negative slot is left out; no two may
    have the same slot."""
    lib, dev = load(), _kv4_device(k, "k")
    c = _kv4(cache, dev)
    dtype = k.dtype
    kp, n, h, kt, kh = _kv4_rows(k, "k", cache.n_heads, cache.head_dim, None, dev)
    vp, m, h, vt, vh = _kv4_rows(v, "v", cache.n_heads, cache.head_dim, dtype, dev)
    if m != n:
        raise ValueError(f"k has {n} tokens, v {m}")
    sp = _w4_ptr(slots, "slots", torch.int32, (n,), dev)
    rc = lib.awq_kv4_append(c, kp, vp, _DTYPES[dtype], n, kt, kh, vt, vh, sp, _w4_stream(stream, dev))
    if rc:
        check(rc)


def awq_kv4_gather(cache: Kv4Cache, slots: torch.Tensor, *, dtype: torch.dtype = torch.float16,
                   k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None, stream=None):
    """(k, v), [tokens, n_heads, head_dim] in dtype: the values that the places
    slots [tokens] int32 hold, zeros for a negative slot."""
    lib, dev = load(), _kv4_device(slots, "slots")
    c = _kv4(cache, dev)
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be torch.float16 or torch.bfloat16, got {dtype}")
    n = slots.numel()
    sp = _w4_ptr(slots, "slots", torch.int32, (n,), dev)
    shape = (n, cache.n_heads, cache.head_dim)
    with _on(stream):
        k, kp = _w4_out(k, "k", dtype, shape, slots, dev)
        v, vp = _w4_out(v, "v", dtype, shape, slots, dev)
    rc = lib.awq_kv4_gather(c, sp, n, kp, vp, _DTYPES[dtype], _w4_stream(stream, dev))
    if rc:
        check(rc)
    return k, v


def awq_kv4_attention(q: torch.Tensor, cache: Kv4Cache, table: torch.Tensor, lens: torch.Tensor, *,
                      starts: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                      out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """softmax(scale Q K^T) V over the 4-bit cache, [tokens, heads, head_dim] in
    q's type.  q [tokens, heads, head_dim] fp16 or bf16 may be a slice; heads is a
    multiple of the cache's, neighbours share a kv head.  table [seqs, max_pages]
    int32 has each sequence's pages, lens [seqs] int32 its keys, its newest tokens
    among them (append them first).  Without starts every sequence has one query
    token; with it, [seqs + 1] int32, sequence s has rows starts[s] ..
    starts[s + 1] - 1 of q, its last tokens, each of which sees the keys up to its
    own.  scale is 1 / sqrt(head_dim) by default.  A row without keys gets zeros,
    rows behind the last sequence are left as they are."""
    lib, dev = load(), _kv4_device(q, "q")
    c = _kv4(cache, dev)
    d = cache.head_dim
    qp, n, h, qt, qh = _kv4_rows(q, "q", None, d, None, dev)
    if table.dim() != 2:
        raise ValueError("table must be [seqs, max_pages]")
    b, pages = table.shape
    tp = _w4_ptr(table, "table", torch.int32, (b, pages), dev)
    lp = _w4_ptr(lens, "lens", torch.int32, (b,), dev)
    sp = None if starts is None else _w4_ptr(starts, "starts", torch.int32, (b + 1,), dev)
    sizes = (cache.n_pages, cache.n_heads, cache.page_size, d, cache.group_size, n, h, b, pages, starts is not None)
    with _on(stream):
        out, op = _w4_out(out, "out", q.dtype, (n, h, d), q, dev)
        workspace, ws, size = _w4_workspace(_kv4_attention_need, sizes, q, workspace)
    rc = lib.awq_kv4_attention(c, qp, _DTYPES[q.dtype], n, h, qt, qh, b, sp, tp, pages, lp,
                               d ** -0.5 if scale is None else scale, op, ws, size,
                               _w4_stream(stream, dev))
    if rc:
        check(rc)
    return out


def awq_fold_inverse_scale(src: torch.Tensor, s: torch.Tensor, *,
                           out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Row j of the fp16 array src ([n] or [n, cols]) divided by s[j], in fp16:
    the gain or bias of the norm, or the weight or bias of the linear, that
    feeds the layer whose columns were scaled by s."""
    if src.dim() not in (1, 2):
        raise ValueError("src must be [n] or [n, cols]")
    rows = src.shape[0]
    cols = 1 if src.dim() == 1 else src.shape[1]
    with _on(stream):
        if out is None:
            out = torch.empty_like(src)
    check(load().awq_fold_inverse_scale(
        ctypes.c_void_p(_dev(src, "src", torch.float16, tuple(src.shape))),
        ctypes.c_void_p(_dev(s, "s", torch.float32, (rows,))), rows, cols,
        ctypes.c_void_p(_dev(out, "out", torch.float16, tuple(src.shape))),
        _stream(stream)))
    return out


def awq_weight_saliency(W: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """mean_o |W[o, k]| (weight-magnitude saliency): awq_act_stats over W's rows."""
    return awq_act_stats(W, out=out, stream=stream)


def awq_select_top_channels(sal: torch.Tensor, n_keep: int, *,
                            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """sal with every channel outside the n_keep most salient set to 1."""
    if sal.dim() != 1:
        raise ValueError("sal must be [in_features]")
    n = sal.shape[0]
    with _on(stream):
        if out is None:
            out = torch.empty_like(sal)
    check(load().awq_select_top_channels(
        ctypes.c_void_p(_dev(sal, "sal", torch.float32, (n,))), n, int(n_keep),
        ctypes.c_void_p(_dev(out, "out", torch.float32, (n,))), _stream(stream)))
    return out
