"""Torch-facing wrapper of the libcq C ABI.

PyTorch supplies device memory and the current stream; every step of the
path runs in libcq's CUDA kernels. Output tensors are allocated here (or
passed in) and handed to the C entry points as raw pointers.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import asdict, dataclass, fields
from typing import NamedTuple, Optional

import torch

from . import _lib


@dataclass(frozen=True)
class Config:
    """Operator attributes (pages' parameter names). See include/cq.h."""
    ep_world_size: int
    moe_expert_num: int
    shared_expert_num: int = 0
    shared_expert_rank_num: int = 0
    zero_expert_num: int = 0
    copy_expert_num: int = 0
    const_expert_num: int = 0
    max_bs: int = 1
    topk: int = 1
    hidden: int = 1024
    global_bs: int = 0
    quant_mode: int = 0
    expert_token_nums_type: int = 1
    mask_ndim: int = 0
    x_dtype: int = 0       # 0 bf16, 1 fp16
    smooth_kind: int = 0   # 0 per-expert rows, 1 one row for all experts, 2 one scalar
    y_dtype: int = 0       # fp8 codes of modes 3-5: 0 e4m3fn, 1 e5m2

    @classmethod
    def from_dict(cls, d: dict) -> "Config":
        names = {f.name for f in fields(cls)}
        return cls(**{k: int(v) for k, v in d.items() if k in names})

    def as_c(self) -> _lib.CqConfig:
        return _c_config(self)

    def _q(self, name):
        c = self.as_c()
        return getattr(_lib.load(), name)(ctypes.byref(c))

    def check(self) -> int:
        return self._q("cq_check_config")

    @property
    def local_expert_num(self) -> int:
        return self._q("cq_local_expert_num")

    @property
    def num_slots(self) -> int:
        return self._q("cq_num_slots")

    @property
    def max_rows(self) -> int:
        return self._q("cq_max_rows")

    @property
    def scale_cols(self) -> int:
        return self._q("cq_scale_cols")

    @property
    def assist_info_size(self) -> int:
        return self._q("cq_assist_info_size")

    @property
    def workspace_size(self) -> int:
        return self._q("cq_workspace_size")

    @property
    def token_dtype(self) -> torch.dtype:
        return torch.float16 if self.x_dtype == 1 else torch.bfloat16

    @property
    def group_cols(self) -> int:
        return (self.hidden + 127) // 128

    def code_dtype(self) -> torch.dtype:
        return {0: self.token_dtype, 1: torch.int8, 2: torch.int8, 3: torch.uint8,
                4: torch.uint8, 5: torch.uint8}[self.quant_mode]  # fp8 codes as raw bytes


@functools.lru_cache(maxsize=256)
def _c_config(cfg: Config) -> _lib.CqConfig:
    """The C struct of a config, built once per distinct config (treat as read-only)."""
    return _lib.CqConfig(**asdict(cfg))


@dataclass(frozen=True)
class ExpertConfig:
    """Attributes of the expert products (cq_expert_config in include/cq.h)."""
    experts: int
    rows: int
    n: int
    k: int
    x_dtype: int = 0       # 0 bf16, 1 fp16, 2 mx fp8 e4m3, 3 mx fp8 e5m2
    w_dtype: int = 0       # mx weight codes: 0 e4m3, 1 e5m2
    out_dtype: int = -1    # -1 the token type, 0 bf16, 1 fp16, 2 f32 (expert_matmul_dw)
    act: int = 0           # 1: SwiGLU, weights with 2n rows
    group: int = 0         # 4-bit weights: inner elements per scale
    rows_type: int = 1     # group_rows: 1 counts, 0 running sums per rank
    experts_per_rank: int = 1

    def as_c(self) -> _lib.CqExpertConfig:
        return _c_expert_config(self)

    def check(self) -> int:
        return _lib.load().cq_check_expert_config(ctypes.byref(self.as_c()))

    @property
    def weight_rows(self) -> int:
        return 2 * self.n if self.act == 1 else self.n

    @property
    def scale_cols(self) -> int:
        """Scale columns of mx rows: Align2(k / 32), as Config.scale_cols."""
        return (self.k // 32 + 1) // 2 * 2

    @property
    def mx(self) -> bool:
        return self.x_dtype in (2, 3)

    @property
    def in_dtype(self) -> torch.dtype:
        return {0: torch.bfloat16, 1: torch.float16}.get(self.x_dtype, torch.uint8)

    @property
    def result_dtype(self) -> torch.dtype:
        d = self.out_dtype if self.out_dtype >= 0 else int(self.x_dtype == 1)
        return {0: torch.bfloat16, 1: torch.float16}.get(d, torch.float32)


@functools.lru_cache(maxsize=256)
def _c_expert_config(cfg: ExpertConfig) -> _lib.CqExpertConfig:
    """The C struct of an expert config, built once per distinct config (treat as read-only)."""
    return _lib.CqExpertConfig(**asdict(cfg))


class _ExpertPlan:
    """What the calls derive from an expert config, kept per distinct config."""

    def __init__(self, cfg: ExpertConfig):
        R, G, WN, K = cfg.rows, cfg.experts, cfg.weight_rows, cfg.k
        self.struct = cfg.as_c()
        self.ref = ctypes.byref(self.struct)
        self.experts, self.act, self.mx = G, cfg.act, cfg.mx
        self.dtype, self.result = cfg.in_dtype, cfg.result_dtype
        self.x, self.w, self.y, self.dy = (R, K), (G, WN, K), (R, cfg.n), (R, WN)
        self.pre_k = (R, 2 * K)  # SwiGLU's products when the input was its result
        self.x_scales, self.w_scales = (R, cfg.scale_cols), (G, WN, cfg.scale_cols)
        self.codes = (G, WN, K // 2)
        self.groups = (G, WN, K // cfg.group if cfg.group > 0 else 0)


@functools.lru_cache(maxsize=256)
def _plan_of(*fields) -> _ExpertPlan:
    return _ExpertPlan(ExpertConfig(*fields))


def _expert_plan(cfg: ExpertConfig) -> _ExpertPlan:
    return _plan_of(*vars(cfg).values())  # half the time of hashing and comparing the config itself


class DispatchResult(NamedTuple):
    expand_x: torch.Tensor          # [R_max, H] bf16 / int8 / uint8 (e4m3 bytes)
    dynamic_scales: Optional[torch.Tensor]  # f32 [R_max] or uint8 [R_max, SC]
    assist_info: torch.Tensor       # int32, opaque (pass to combine)
    ep_recv_count: torch.Tensor     # int32 [W, W*L]
    expert_token_nums: torch.Tensor  # int64 [W, L]
    expand_scales: Optional[torch.Tensor]  # f32 [R_max]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t, name, dtype, shape=None, device=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def alloc_workspace(cfg: Config, device) -> torch.Tensor:
    """A zero-filled workspace (torch allocations are 512-byte aligned)."""
    n = cfg.workspace_size
    if n == 0:
        raise _lib.CqError(_lib.CQ_ERR_ARG, "workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_dispatch_outputs(cfg: Config, device, with_expand_scales: bool = True) -> DispatchResult:
    W, H, R = cfg.ep_world_size, cfg.hidden, cfg.max_rows
    L = cfg.local_expert_num
    if cfg.quant_mode == 2:
        dyn = torch.empty(R, dtype=torch.float32, device=device)
    elif cfg.quant_mode == 3:
        dyn = torch.empty(R, cfg.group_cols, dtype=torch.float32, device=device)
    elif cfg.quant_mode in (4, 5):
        dyn = torch.empty(R, cfg.scale_cols, dtype=torch.uint8, device=device)
    else:
        dyn = None
    return DispatchResult(
        torch.empty(R, H, dtype=cfg.code_dtype(), device=device), dyn,
        torch.empty(cfg.assist_info_size, dtype=torch.int32, device=device),
        torch.empty(W, W * L, dtype=torch.int32, device=device),
        torch.empty(W, L, dtype=torch.int64, device=device),
        torch.empty(R, dtype=torch.float32, device=device) if with_expand_scales else None)


def _check_outputs(cfg: Config, out: DispatchResult, dev, rows: bool = True,
                   route: bool = True) -> None:
    """The caller's output buffers must have the config's shapes and types:
    the kernels write through raw pointers and cannot check sizes. `rows`:
    the permute outputs are written; `route`: the routing outputs are."""
    W, H, R = cfg.ep_world_size, cfg.hidden, cfg.max_rows
    L = cfg.local_expert_num
    if out.assist_info is None:
        raise ValueError("assist_info is required")
    _need(out.assist_info, "assist_info", torch.int32, (cfg.assist_info_size,), dev)
    if route:
        if out.ep_recv_count is None or out.expert_token_nums is None:
            raise ValueError("ep_recv_count and expert_token_nums are required")
        _need(out.ep_recv_count, "ep_recv_count", torch.int32, (W, W * L), dev)
        _need(out.expert_token_nums, "expert_token_nums", torch.int64, (W, L), dev)
    if rows:
        if out.expand_x is None:
            raise ValueError("expand_x is required")
        _need(out.expand_x, "expand_x", cfg.code_dtype(), (R, H), dev)
        if cfg.quant_mode == 2:
            _need(out.dynamic_scales, "dynamic_scales", torch.float32, (R,), dev)
        elif cfg.quant_mode == 3:
            _need(out.dynamic_scales, "dynamic_scales", torch.float32, (R, cfg.group_cols), dev)
        elif cfg.quant_mode in (4, 5):
            _need(out.dynamic_scales, "dynamic_scales", torch.uint8, (R, cfg.scale_cols), dev)
        _need(out.expand_scales, "expand_scales", torch.float32, (R,), dev)


def _check_workspace(workspace: torch.Tensor, dev) -> None:
    _need(workspace, "workspace", torch.uint8, None, dev)


def _check_inputs(cfg, x, expert_ids, smooth_scales, x_active_mask, bs_per_rank, expert_scales):
    W, BS, K, H = cfg.ep_world_size, cfg.max_bs, cfg.topk, cfg.hidden
    dev = expert_ids.device
    _need(expert_ids, "expert_ids", torch.int32, (W, BS, K))
    if x is not None:
        _need(x, "x", cfg.token_dtype, (W, BS, H), dev)
    if smooth_scales is not None:
        s_eff = cfg.shared_expert_num if cfg.shared_expert_rank_num > 0 else 0
        shape = {0: (s_eff + cfg.moe_expert_num, H), 1: (H,), 2: (1,)}[cfg.smooth_kind]
        _need(smooth_scales, "smooth_scales", torch.float32, shape, dev)
    if cfg.mask_ndim == 1:
        _need(x_active_mask, "x_active_mask", torch.uint8, (W, BS), dev)
    elif cfg.mask_ndim == 2:
        _need(x_active_mask, "x_active_mask", torch.uint8, (W, BS, K), dev)
    _need(bs_per_rank, "bs_per_rank", torch.int32, (W,), dev)
    _need(expert_scales, "expert_scales", torch.float32, (W, BS, K), dev)
    return dev


def dispatch(cfg: Config, x: torch.Tensor, expert_ids: torch.Tensor,
             smooth_scales: Optional[torch.Tensor] = None,
             x_active_mask: Optional[torch.Tensor] = None,
             bs_per_rank: Optional[torch.Tensor] = None,
             expert_scales: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None,
             out: Optional[DispatchResult] = None) -> DispatchResult:
    """MoE dispatch of every logical rank's tokens (cq_dispatch)."""
    dev = _check_inputs(cfg, x, expert_ids, smooth_scales, x_active_mask, bs_per_rank,
                        expert_scales)
    if workspace is None:
        workspace = alloc_workspace(cfg, dev)
    _check_workspace(workspace, dev)
    if out is None:
        out = alloc_dispatch_outputs(cfg, dev, expert_scales is not None)
    _check_outputs(cfg, out, dev)
    c = cfg.as_c()
    with torch.cuda.device(dev):  # the library looks up the current device
        rc = _lib.load().cq_dispatch(
            ctypes.byref(c), _ptr(x), _ptr(expert_ids), _ptr(smooth_scales), _ptr(x_active_mask),
            _ptr(bs_per_rank), _ptr(expert_scales), _ptr(out.expand_x), _ptr(out.dynamic_scales),
            _ptr(out.assist_info), _ptr(out.ep_recv_count), _ptr(out.expert_token_nums),
            _ptr(out.expand_scales), _ptr(workspace), workspace.numel(), _stream(dev))
    _lib.check(rc, "cq_dispatch")
    return out


def dispatch_noalloc(cfg: Config, x: torch.Tensor, expert_ids: torch.Tensor,
                     smooth_scales: Optional[torch.Tensor] = None,
                     x_active_mask: Optional[torch.Tensor] = None,
                     bs_per_rank: Optional[torch.Tensor] = None,
                     expert_scales: Optional[torch.Tensor] = None,
                     out: Optional[DispatchResult] = None) -> DispatchResult:
    """Dispatch through cq_dispatch_noalloc: no workspace, the library's own
    fixed scratch instead (for callers that cannot allocate device memory;
    calls must not overlap on the GPU). `out` may be preallocated."""
    dev = _check_inputs(cfg, x, expert_ids, smooth_scales, x_active_mask, bs_per_rank,
                        expert_scales)
    if out is None:
        out = alloc_dispatch_outputs(cfg, dev, expert_scales is not None)
    _check_outputs(cfg, out, dev)
    c = cfg.as_c()
    with torch.cuda.device(dev):  # the library looks up the current device
        rc = _lib.load().cq_dispatch_noalloc(
            ctypes.byref(c), _ptr(x), _ptr(expert_ids), _ptr(smooth_scales), _ptr(x_active_mask),
            _ptr(bs_per_rank), _ptr(expert_scales), _ptr(out.expand_x), _ptr(out.dynamic_scales),
            _ptr(out.assist_info), _ptr(out.ep_recv_count), _ptr(out.expert_token_nums),
            _ptr(out.expand_scales), _stream(dev))
    _lib.check(rc, "cq_dispatch_noalloc")
    return out


def dispatch_route(cfg: Config, expert_ids, x_active_mask=None, bs_per_rank=None, *,
                   workspace, out: DispatchResult) -> None:
    """First half of dispatch (scan, counts, prefix sums)."""
    dev = _check_inputs(cfg, None, expert_ids, None, x_active_mask, bs_per_rank, None)
    _check_workspace(workspace, dev)
    _check_outputs(cfg, out, dev, rows=False)
    c = cfg.as_c()
    with torch.cuda.device(dev):  # the library looks up the current device
        rc = _lib.load().cq_dispatch_route(
            ctypes.byref(c), _ptr(expert_ids), _ptr(x_active_mask), _ptr(bs_per_rank),
            _ptr(out.assist_info), _ptr(out.ep_recv_count), _ptr(out.expert_token_nums),
            _ptr(workspace), workspace.numel(), _stream(dev))
    _lib.check(rc, "cq_dispatch_route")


def dispatch_permute(cfg: Config, x, expert_ids, smooth_scales=None, expert_scales=None,
                     x_active_mask=None, bs_per_rank=None, *, workspace,
                     out: DispatchResult) -> None:
    """Second half of dispatch (placement and quantisation). The mask and
    per-rank BS, as given to dispatch_route, only let the kernel skip
    prefetching rows of inactive tokens."""
    dev = _check_inputs(cfg, x, expert_ids, smooth_scales, x_active_mask, bs_per_rank,
                        expert_scales)
    _check_workspace(workspace, dev)
    _check_outputs(cfg, out, dev, route=False)
    c = cfg.as_c()
    with torch.cuda.device(dev):  # the library looks up the current device
        rc = _lib.load().cq_dispatch_permute(
            ctypes.byref(c), _ptr(x), _ptr(expert_ids), _ptr(smooth_scales), _ptr(x_active_mask),
            _ptr(bs_per_rank), _ptr(expert_scales), _ptr(out.expand_x), _ptr(out.dynamic_scales),
            _ptr(out.assist_info), _ptr(out.expand_scales), _ptr(workspace), workspace.numel(),
            _stream(dev))
    _lib.check(rc, "cq_dispatch_permute")


def combine(cfg: Config, expand_x_ffn: torch.Tensor, assist_info: torch.Tensor,
            expert_scales: torch.Tensor, ep_recv_count: Optional[torch.Tensor] = None,
            ori_x: Optional[torch.Tensor] = None,
            const_alpha1: Optional[torch.Tensor] = None,
            const_alpha2: Optional[torch.Tensor] = None,
            const_v: Optional[torch.Tensor] = None,
            out_dtype: Optional[torch.dtype] = None,
            y: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """MoE combine (cq_combine): y [W, BS, H] in the token dtype (default) or
    float32. With `workspace` (the dispatch workspace of the same config) the
    call is cq_combine_ws: its status goes to that workspace (read_status)."""
    W, BS, K, H = cfg.ep_world_size, cfg.max_bs, cfg.topk, cfg.hidden
    dev = assist_info.device
    if workspace is not None:
        _check_workspace(workspace, dev)
    _need(expand_x_ffn, "expand_x_ffn", cfg.token_dtype, (cfg.max_rows, H), dev)
    _need(assist_info, "assist_info", torch.int32, (cfg.assist_info_size,), dev)
    _need(expert_scales, "expert_scales", torch.float32, (W, BS, K), dev)
    _need(ep_recv_count, "ep_recv_count", torch.int32,
          (W, W * cfg.local_expert_num), dev)
    _need(ori_x, "ori_x", cfg.token_dtype, (W, BS, H), dev)
    Q = cfg.const_expert_num
    _need(const_alpha1, "const_alpha1", torch.float32, (Q,), dev)
    _need(const_alpha2, "const_alpha2", torch.float32, (Q,), dev)
    _need(const_v, "const_v", cfg.token_dtype, (Q, H), dev)
    if out_dtype is None:
        out_dtype = cfg.token_dtype
    if out_dtype not in (cfg.token_dtype, torch.float32):
        raise ValueError("out_dtype must be the token dtype or float32")
    if y is None:
        y = torch.empty(W, BS, H, dtype=out_dtype, device=dev)
    _need(y, "y", out_dtype, (W, BS, H), dev)
    c = cfg.as_c()
    args = (ctypes.byref(c), _ptr(expand_x_ffn), _ptr(assist_info), _ptr(ep_recv_count),
            _ptr(expert_scales), _ptr(ori_x), _ptr(const_alpha1), _ptr(const_alpha2),
            _ptr(const_v), 0 if out_dtype != torch.float32 else 1, _ptr(y))
    with torch.cuda.device(dev):  # the library looks up the current device
        if workspace is None:
            rc = _lib.load().cq_combine(*args, _stream(dev))
        else:
            rc = _lib.load().cq_combine_ws(*args, _ptr(workspace), workspace.numel(), _stream(dev))
    _lib.check(rc, "cq_combine" if workspace is None else "cq_combine_ws")
    return y


def combine_ws(cfg: Config, expand_x_ffn: torch.Tensor, assist_info: torch.Tensor,
               expert_scales: torch.Tensor, workspace: torch.Tensor, **kw) -> torch.Tensor:
    """cq_combine_ws: combine whose status goes to `workspace` (read_status)."""
    return combine(cfg, expand_x_ffn, assist_info, expert_scales, workspace=workspace, **kw)


def combine_quant(cfg: Config, expand_x_ffn: torch.Tensor, assist_info: torch.Tensor,
                  codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """Expert-side int8 block quantisation of the FFN outputs (cq_combine_quant).
    Returns (codes int8 [R_max, H], scales f32 [R_max, H/8])."""
    R, H = cfg.max_rows, cfg.hidden
    dev = assist_info.device
    _need(expand_x_ffn, "expand_x_ffn", cfg.token_dtype, (R, H), dev)
    _need(assist_info, "assist_info", torch.int32, (cfg.assist_info_size,), dev)
    if codes is None:
        codes = torch.empty(R, H, dtype=torch.int8, device=dev)
    if scales is None:
        scales = torch.empty(R, H // 8, dtype=torch.float32, device=dev)
    _need(codes, "codes", torch.int8, (R, H), dev)
    _need(scales, "scales", torch.float32, (R, H // 8), dev)
    c = cfg.as_c()
    with torch.cuda.device(dev):  # the library looks up the current device
        rc = _lib.load().cq_combine_quant(ctypes.byref(c), _ptr(expand_x_ffn), _ptr(assist_info),
                                          _ptr(codes), _ptr(scales), _stream(dev))
    _lib.check(rc, "cq_combine_quant")
    return codes, scales


def combine_q8(cfg: Config, codes: torch.Tensor, scales: torch.Tensor, assist_info: torch.Tensor,
               expert_scales: torch.Tensor, ep_recv_count: Optional[torch.Tensor] = None,
               ori_x: Optional[torch.Tensor] = None,
               const_alpha1: Optional[torch.Tensor] = None,
               const_alpha2: Optional[torch.Tensor] = None,
               const_v: Optional[torch.Tensor] = None,
               out_dtype: Optional[torch.dtype] = None,
               y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """MoE combine from int8 expert outputs (cq_combine_q8)."""
    W, BS, K, H = cfg.ep_world_size, cfg.max_bs, cfg.topk, cfg.hidden
    dev = assist_info.device
    _need(codes, "codes", torch.int8, (cfg.max_rows, H), dev)
    _need(scales, "scales", torch.float32, (cfg.max_rows, H // 8), dev)
    _need(assist_info, "assist_info", torch.int32, (cfg.assist_info_size,), dev)
    _need(expert_scales, "expert_scales", torch.float32, (W, BS, K), dev)
    _need(ep_recv_count, "ep_recv_count", torch.int32,
          (W, W * cfg.local_expert_num), dev)
    _need(ori_x, "ori_x", cfg.token_dtype, (W, BS, H), dev)
    Q = cfg.const_expert_num
    _need(const_alpha1, "const_alpha1", torch.float32, (Q,), dev)
    _need(const_alpha2, "const_alpha2", torch.float32, (Q,), dev)
    _need(const_v, "const_v", cfg.token_dtype, (Q, H), dev)
    if out_dtype is None:
        out_dtype = cfg.token_dtype
    if out_dtype not in (cfg.token_dtype, torch.float32):
        raise ValueError("out_dtype must be the token dtype or float32")
    if y is None:
        y = torch.empty(W, BS, H, dtype=out_dtype, device=dev)
    _need(y, "y", out_dtype, (W, BS, H), dev)
    c = cfg.as_c()
    with torch.cuda.device(dev):  # the library looks up the current device
        rc = _lib.load().cq_combine_q8(
            ctypes.byref(c), _ptr(codes), _ptr(scales), _ptr(assist_info), _ptr(ep_recv_count),
            _ptr(expert_scales), _ptr(ori_x), _ptr(const_alpha1), _ptr(const_alpha2), _ptr(const_v),
            0 if out_dtype != torch.float32 else 1, _ptr(y), _stream(dev))
    _lib.check(rc, "cq_combine_q8")
    return y


def _arg(t, name, dtype, shape, dev: torch.device):
    """The address of a tensor argument after _need's checks (which raise); None
    for None. One pass over the common case: these calls may take only microseconds
    on the GPU."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _need(t, name, dtype, shape, dev)
    return t.data_ptr()


def _result(t, name, dtype, shape, dev: torch.device):
    """A result tensor, the caller's (checked) or a new one, and its address."""
    if t is not None:
        return t, _arg(t, name, dtype, shape, dev)
    t = torch.empty(shape, dtype=dtype, device=dev)
    return t, t.data_ptr()


def _group_rows(p: _ExpertPlan, group_rows: torch.Tensor) -> torch.device:
    """Checks the counts; returns the device that the other tensors must be on."""
    _need(group_rows, "group_rows", torch.int64)
    if group_rows.numel() != p.experts:
        raise ValueError(f"group_rows must have {p.experts} entries, got {group_rows.numel()}")
    return group_rows.device


# The handle of the current stream, without building a torch.cuda.Stream around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _expert_call(name: str, dev: torch.device, *args) -> None:
    fn = getattr(_lib.load(), name)
    if _current_device() == dev.index:  # the library looks up the current device
        rc = fn(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev.index))
    if rc != _lib.CQ_OK:
        _lib.check(rc, name)


def expert_matmul(cfg: ExpertConfig, x: torch.Tensor, w: torch.Tensor, group_rows: torch.Tensor,
                  x_scales: Optional[torch.Tensor] = None,
                  w_scales: Optional[torch.Tensor] = None,
                  pre: Optional[torch.Tensor] = None,
                  y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Grouped matrix product over the experts' rows (cq_expert_matmul):
    y [rows, n], with act 1 SwiGLU of the gate and up products (`pre`
    [rows, 2n] receives them). `group_rows` is dispatch's expert_token_nums."""
    p = _expert_plan(cfg)
    dev = _group_rows(p, group_rows)
    if x is None or w is None:
        raise ValueError("x and w are required")
    px, pw = _arg(x, "x", p.dtype, p.x, dev), _arg(w, "w", p.dtype, p.w, dev)
    pxs = pws = None
    if p.mx:
        if x_scales is None or w_scales is None:
            raise ValueError("x_scales and w_scales are required with mx types")
        pxs = _arg(x_scales, "x_scales", torch.uint8, p.x_scales, dev)
        pws = _arg(w_scales, "w_scales", torch.uint8, p.w_scales, dev)
    elif x_scales is not None or w_scales is not None:
        raise ValueError("x_scales and w_scales go with mx types only")
    if pre is not None and p.act != 1:
        raise ValueError("pre goes with act 1 only")
    ppre = _arg(pre, "pre", p.result, p.dy, dev)
    y, py = _result(y, "y", p.result, p.y, dev)
    _expert_call("cq_expert_matmul", dev, p.ref, px, pxs, pw, pws, group_rows.data_ptr(), py, ppre)
    return y


def expert_matmul_dx(cfg: ExpertConfig, dy: torch.Tensor, w: torch.Tensor,
                     group_rows: torch.Tensor, pre: Optional[torch.Tensor] = None,
                     dx: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of expert_matmul's input (cq_expert_matmul_dx): [rows, k], or
    with `pre` [rows, 2k] (the input was SwiGLU of pre) the gradient of pre."""
    p = _expert_plan(cfg)
    dev = _group_rows(p, group_rows)
    if dy is None or w is None:
        raise ValueError("dy and w are required")
    pdy, pw = _arg(dy, "dy", p.dtype, p.dy, dev), _arg(w, "w", p.dtype, p.w, dev)
    ppre = _arg(pre, "pre", p.dtype, p.pre_k, dev)
    shape = p.x if pre is None else p.pre_k
    dx, pdx = _result(dx, "dx", p.dtype, shape, dev)
    _expert_call("cq_expert_matmul_dx", dev, p.ref, pdy, pw, group_rows.data_ptr(), ppre, pdx)
    return dx


def expert_matmul_dw(cfg: ExpertConfig, dy: torch.Tensor, x: torch.Tensor,
                     group_rows: torch.Tensor, dw: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of expert_matmul's weights (cq_expert_matmul_dw), in the
    config's out_dtype: the token type (default) or f32."""
    p = _expert_plan(cfg)
    dev = _group_rows(p, group_rows)
    if dy is None or x is None:
        raise ValueError("dy and x are required")
    pdy, px = _arg(dy, "dy", p.dtype, p.dy, dev), _arg(x, "x", p.dtype, p.x, dev)
    dw, pdw = _result(dw, "dw", p.result, p.w, dev)
    _expert_call("cq_expert_matmul_dw", dev, p.ref, pdy, px, group_rows.data_ptr(), pdw)
    return dw


def expert_matmul_w4(cfg: ExpertConfig, x: torch.Tensor, codes: torch.Tensor,
                     scales: torch.Tensor, group_rows: torch.Tensor,
                     zeros: Optional[torch.Tensor] = None,
                     y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """expert_matmul with 4-bit weights (cq_expert_matmul_w4), for few rows per
    expert: codes uint8 [G, n or 2n, k/2], scales (and uint8 zeros)
    [G, n or 2n, k/group]."""
    p = _expert_plan(cfg)
    dev = _group_rows(p, group_rows)
    if x is None or codes is None or scales is None:
        raise ValueError("x, codes and scales are required")
    px = _arg(x, "x", p.dtype, p.x, dev)
    pc = _arg(codes, "codes", torch.uint8, p.codes, dev)
    ps = _arg(scales, "scales", p.dtype, p.groups, dev)
    pz = _arg(zeros, "zeros", torch.uint8, p.groups, dev)
    y, py = _result(y, "y", p.dtype, p.y, dev)
    _expert_call("cq_expert_matmul_w4", dev, p.ref, px, pc, ps, pz, group_rows.data_ptr(), py)
    return y


def read_expert_status(device=None) -> int:
    """Synchronise the current stream of `device`, return and clear the expert
    products' status bits (CQ_ST_BAD_ROWS, CQ_ST_TIMEOUT) of that device."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    st = ctypes.c_uint32(0)
    with torch.cuda.device(dev):
        rc = _lib.load().cq_read_expert_status(ctypes.byref(st), _stream(dev))
    _lib.check(rc, "cq_read_expert_status")
    return int(st.value)


def read_status(workspace: torch.Tensor) -> int:
    """Synchronise the current stream, return and clear the sticky status bits."""
    st = ctypes.c_uint32(0)
    with torch.cuda.device(workspace.device):
        rc = _lib.load().cq_read_status(_ptr(workspace), ctypes.byref(st),
                                        _stream(workspace.device))
    _lib.check(rc, "cq_read_status")
    return int(st.value)


def read_combine_status(device=None) -> int:
    """Synchronise the current stream of `device`, return and clear the
    combine kernels' status bits (CQ_ST_TIMEOUT) of that device."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    st = ctypes.c_uint32(0)
    with torch.cuda.device(dev):
        rc = _lib.load().cq_read_combine_status(ctypes.byref(st), _stream(dev))
    _lib.check(rc, "cq_read_combine_status")
    return int(st.value)


def _bounded_check(name: str, device) -> tuple[int, float]:
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    value, secs = ctypes.c_uint32(0), ctypes.c_double(0.0)
    with torch.cuda.device(dev):
        rc = getattr(_lib.load(), name)(ctypes.byref(value), ctypes.byref(secs), _stream(dev))
    _lib.check(rc, name)
    return int(value.value), float(secs.value)


def check_bounded_wait(device=None) -> tuple[int, float]:
    """Run the library's bounded wait on a barrier nothing completes
    (cq_check_bounded_wait): returns (gave_up, seconds)."""
    return _bounded_check("cq_check_bounded_wait", device)


def check_bounded_meet(device=None) -> tuple[int, float]:
    """Sixteen warps that wait apart and meet, one of which gives up
    (cq_check_bounded_meet): returns (threads that left, seconds)."""
    return _bounded_check("cq_check_bounded_meet", device)


def assist_views(cfg: Config, assist_info: torch.Tensor):
    """Views into assist_info: rows [R_max, 4], inv [W, BS, NS], rank_row_base [W+1]."""
    R, W, BS, NS = cfg.max_rows, cfg.ep_world_size, cfg.max_bs, cfg.num_slots
    rows = assist_info[:4 * R].view(R, 4)
    inv = assist_info[4 * R:4 * R + W * BS * NS].view(W, BS, NS)
    base = assist_info[4 * R + W * BS * NS:]
    return rows, inv, base


# The C ABI's names (include/cq.h) for the same calls.
def dispatch_workspace_size(cfg: Config) -> int:
    """Bytes of the dispatch workspace (cq_dispatch_workspace_size, the same
    as Config.workspace_size)."""
    return int(_lib.load().cq_dispatch_workspace_size(ctypes.byref(cfg.as_c())))


def dispatch_one_kernel(cfg: Config, with_smooth_scales: bool = False) -> bool:
    """Whether cq_dispatch runs this config's routing and permute as one
    kernel (cq_dispatch_one_kernel; host only)."""
    rc = _lib.load().cq_dispatch_one_kernel(ctypes.byref(cfg.as_c()), int(bool(with_smooth_scales)))
    if rc < 0:
        _lib.check(rc, "cq_dispatch_one_kernel")
    return rc == 1


cq_dispatch = moe_dispatch = dispatch
cq_dispatch_workspace_size = dispatch_workspace_size
cq_dispatch_one_kernel = dispatch_one_kernel
cq_dispatch_route = dispatch_route
cq_dispatch_permute = dispatch_permute
cq_dispatch_noalloc = dispatch_noalloc
cq_combine = moe_combine = combine
cq_combine_ws = combine_ws
cq_combine_quant = combine_quant
cq_combine_q8 = combine_q8
cq_expert_matmul = expert_matmul
cq_expert_matmul_dx = expert_matmul_dx
cq_expert_matmul_dw = expert_matmul_dw
cq_expert_matmul_w4 = expert_matmul_w4
cq_read_expert_status = read_expert_status
cq_read_status = read_status
cq_read_combine_status = read_combine_status
cq_check_bounded_wait = check_bounded_wait
cq_check_bounded_meet = check_bounded_meet
