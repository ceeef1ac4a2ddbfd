"""MoE expert-parallel layout / dispatch / combine on one MI355X rank.

Thin Python binding of ``libepl.so`` (C ABI in ``include/epl.h``). The
functions named ``epl_*`` mirror the C entry points one to one and do only
argument marshalling: they check tensor dtypes, shapes and devices, pass raw
pointers and the current HIP stream, and turn status codes into exceptions.
Every step of the path runs in the library's HIP kernels; there is no CPU or
PyTorch fallback, and using the package without the built library raises.

``dispatch`` and ``combine`` are tensor-level conveniences on top of them:
they allocate outputs with ``torch.empty`` and call the same entry points.
With ``stream=`` they run as under ``with torch.cuda.stream(stream)``: memory
is taken from that stream's pool.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple, Optional

from . import build as _build

__all__ = [
    "EplError", "Problem", "lib_path", "load", "is_built", "ensure_built",
    "epl_validate", "epl_workspace_bytes", "epl_capacity_rows", "epl_layout", "epl_scan",
    "epl_scatter", "epl_dispatch", "epl_combine", "epl_expert_scale", "epl_status", "epl_total",
    "epl_strerror", "epl_version", "dispatch", "combine", "expert_scale", "DispatchResult",
    "EPL_OK", "EPL_EINVAL", "EPL_ERANGE", "EPL_ECAPACITY", "EPL_EHIP", "EPL_OUT_F32",
    "EPL_OUT_BF16", "prepare", "epl_scatter_fp8", "epl_dispatch_fp8", "EPL_SCALE_NONE",
    "EPL_SCALE_F32", "EPL_SCALE_UE8M0", "epl_dispatch_static", "StaticWorkspace",
    "EPL_STATIC_WORKSPACE_BYTES", "Router", "Product", "epl_router_validate", "epl_route",
    "epl_route_backward", "epl_product_validate", "epl_product_workspace_bytes",
    "epl_weight_grad_workspace_bytes", "epl_expert_product", "epl_expert_weight_grad",
    "epl_combine_backward", "route", "route_backward", "expert_product", "expert_weight_grad",
    "combine_backward", "dispatch_backward", "EPL_SCORE_SOFTMAX", "EPL_SCORE_SIGMOID",
    "EPL_ACT_NONE", "EPL_ACT_SILU", "EPL_ACT_GELU", "EPL_ACT_SWIGLU", "EPL_ACT_SILU_GRAD",
    "EPL_ACT_GELU_GRAD", "EPL_ACT_SWIGLU_GRAD", "EPL_WEIGHT_OUT_IN", "EPL_WEIGHT_IN_OUT",
    "EPL_SCALE_F32_RECT", "Cast", "WeightCast", "ProductFp8", "epl_cast_validate",
    "epl_weight_cast_validate", "epl_product_fp8_validate", "epl_product_fp8_workspace_bytes",
    "epl_quantize", "epl_dequantize", "epl_quantize_weight", "epl_expert_product_fp8", "quantize",
    "dequantize", "quantize_weight", "expert_product_fp8", "gated_block_fp8",
    "gated_block_fp8_backward",
]

EPL_OK = 0
EPL_EINVAL = -1
EPL_ERANGE = -2
EPL_ECAPACITY = -3
EPL_EHIP = -4
EPL_OUT_F32 = 0
EPL_OUT_BF16 = 1
EPL_SCALE_NONE = 0
EPL_SCALE_F32 = 1
EPL_SCALE_UE8M0 = 2
EPL_SCALE_F32_RECT = 3
EPL_STATIC_WORKSPACE_BYTES = 8 << 20
EPL_SCORE_SOFTMAX = 0
EPL_SCORE_SIGMOID = 1
EPL_ACT_NONE = 0
EPL_ACT_SILU = 1
EPL_ACT_GELU = 2
EPL_ACT_SWIGLU = 3
EPL_ACT_SILU_GRAD = 4
EPL_ACT_GELU_GRAD = 5
EPL_ACT_SWIGLU_GRAD = 6
EPL_WEIGHT_OUT_IN = 0
EPL_WEIGHT_IN_OUT = 1

# Every function include/epl.h declares; tests check the library exports them.
C_ENTRY_POINTS = (
    "epl_validate", "epl_workspace_bytes", "epl_capacity_rows", "epl_layout", "epl_scan",
    "epl_scatter", "epl_dispatch", "epl_scatter_fp8", "epl_dispatch_fp8", "epl_combine",
    "epl_expert_scale", "epl_status", "epl_total", "epl_strerror", "epl_version",
    "epl_ll_workspace_bytes", "epl_ll_dispatch", "epl_dispatch_static",
    "epl_router_validate", "epl_route", "epl_route_backward", "epl_product_validate",
    "epl_expert_product", "epl_expert_weight_grad", "epl_combine_backward",
    "epl_product_workspace_bytes", "epl_weight_grad_workspace_bytes",
    "epl_cast_validate", "epl_quantize", "epl_dequantize", "epl_weight_cast_validate",
    "epl_quantize_weight", "epl_product_fp8_validate", "epl_product_fp8_workspace_bytes",
    "epl_expert_product_fp8",
)


class EplError(RuntimeError):
    """A non-zero status code from libepl."""

    def __init__(self, code: int, where: str):
        self.code = code
        msg = epl_strerror(code) if _LIB is not None else f"code {code}"
        super().__init__(f"{where}: {msg} ({code})")


class Problem(ctypes.Structure):
    """epl_problem: T, K, E, R, H, S, a, G (see include/epl.h)."""

    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("num_topk", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("num_ranks", ctypes.c_int32),
        ("hidden", ctypes.c_int32),
        ("scale_cols", ctypes.c_int32),
        ("expert_alignment", ctypes.c_int32),
        ("ranks_per_node", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]

    @classmethod
    def make(cls, num_tokens, num_topk, num_experts, num_ranks, hidden, scale_cols=0,
             expert_alignment=0, ranks_per_node=0):
        return cls(int(num_tokens), int(num_topk), int(num_experts), int(num_ranks), int(hidden),
                   int(scale_cols), int(expert_alignment), int(ranks_per_node), 0)

    @property
    def num_nodes(self) -> int:
        """Entries of num_tokens_per_rdma_rank (0 when it is not produced)."""
        G, R = self.ranks_per_node, self.num_ranks
        return R // G if 0 < G < R else 0

    def __repr__(self):
        return (f"Problem(T={self.num_tokens}, K={self.num_topk}, E={self.num_experts}, "
                f"R={self.num_ranks}, H={self.hidden}, S={self.scale_cols}, "
                f"a={self.expert_alignment}, G={self.ranks_per_node})")


class Router(ctypes.Structure):
    """epl_router: sizes and rules of the routing (see include/epl.h)."""

    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("num_topk", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("topk_groups", ctypes.c_int32),
        ("group_top", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("logits_type", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("reserved", ctypes.c_int32),
    ]


class Product(ctypes.Structure):
    """epl_product_desc: sizes and epilogue of an experts' product (see
    include/epl.h)."""

    _fields_ = [
        ("num_rows", ctypes.c_int64),
        ("expected_rows", ctypes.c_int64),
        ("num_experts", ctypes.c_int32),
        ("in_cols", ctypes.c_int32),
        ("out_cols", ctypes.c_int32),
        ("weight_layout", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("out_type", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class Cast(ctypes.Structure):
    """epl_cast_desc: sizes and formats of a cast of rows (see include/epl.h)."""

    _fields_ = [
        ("num_rows", ctypes.c_int64),
        ("num_experts", ctypes.c_int32),
        ("cols", ctypes.c_int32),
        ("value_type", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("scale_format", ctypes.c_int32),
        ("rows_per_expert", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("reserved2", ctypes.c_int32),
    ]


class WeightCast(ctypes.Structure):
    """epl_weight_cast_desc: sizes of a cast of weights (see include/epl.h)."""

    _fields_ = [
        ("num_experts", ctypes.c_int32),
        ("out_cols", ctypes.c_int32),
        ("in_cols", ctypes.c_int32),
        ("value_type", ctypes.c_int32),
        ("scale_format", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class ProductFp8(ctypes.Structure):
    """epl_product_fp8_desc: sizes, formats and epilogue of an experts'
    product on 8-bit rows (see include/epl.h)."""

    _fields_ = [
        ("num_rows", ctypes.c_int64),
        ("expected_rows", ctypes.c_int64),
        ("num_experts", ctypes.c_int32),
        ("in_cols", ctypes.c_int32),
        ("out_cols", ctypes.c_int32),
        ("weight_layout", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("out_type", ctypes.c_int32),
        ("scale_format", ctypes.c_int32),
        ("rows_per_expert", ctypes.c_int32),
        ("weight_scale_format", ctypes.c_int32),
        ("codes_scale_format", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("reserved2", ctypes.c_int32),
    ]


_LIB: Optional[ctypes.CDLL] = None
_P = ctypes.c_void_p
_PP = ctypes.POINTER(Problem)


def lib_path() -> str:
    return _build.LIB


def is_built() -> bool:
    return os.path.exists(_build.LIB)


def ensure_built(verbose: bool = False) -> str:
    """Build libepl.so if it is missing or older than its sources."""
    if _build.needs_build():
        _build.build(verbose=verbose)
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libepl.so (or the build named by EPL_LIB, e.g. the test suite's
    host-sanitizer build); raises if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = os.environ.get("EPL_LIB") or _build.LIB
    if not os.path.exists(path):
        raise ImportError(
            f"libepl.so is not built ({path}); run `python -m permute_ep_layout_amd.build` "
            "or __graft_entry__.build() first. There is no fallback implementation.")
    try:
        import torch  # noqa: F401  (share torch's HIP runtime if it is loaded)
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    i64, i32 = ctypes.c_int64, ctypes.c_int
    lib.epl_validate.argtypes = [_PP]
    lib.epl_validate.restype = i32
    lib.epl_workspace_bytes.argtypes = [_PP]
    lib.epl_workspace_bytes.restype = ctypes.c_size_t
    lib.epl_capacity_rows.argtypes = [_PP]
    lib.epl_capacity_rows.restype = i64
    lib.epl_layout.argtypes = [_PP, _P, _P, _P, _P, _P, _P, _P]
    lib.epl_layout.restype = i32
    lib.epl_scan.argtypes = [_PP, _P, _P, _P, _P, _P]
    lib.epl_scan.restype = i32
    lib.epl_scatter.argtypes = [_PP, _P, _P, _P, _P, _P, i64, _P, _P, _P, _P, _P]
    lib.epl_scatter.restype = i32
    lib.epl_dispatch.argtypes = [_PP, _P, _P, _P, i64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                 _P]
    lib.epl_dispatch.restype = i32
    lib.epl_scatter_fp8.argtypes = [_PP, _P, _P, i32, _P, _P, _P, i64, _P, _P, _P, _P, _P]
    lib.epl_scatter_fp8.restype = i32
    lib.epl_dispatch_fp8.argtypes = [_PP, _P, _P, _P, i32, i64, _P, _P, _P, _P, _P, _P, _P, _P,
                                     _P, _P, _P, _P]
    lib.epl_dispatch_fp8.restype = i32
    lib.epl_dispatch_static.argtypes = [_PP, _P, _P, _P, i64, _P, _P, _P, _P, _P, _P, _P, _P,
                                        _P, _P, ctypes.POINTER(ctypes.c_void_p), _P]
    lib.epl_dispatch_static.restype = i32
    lib.epl_ll_workspace_bytes.argtypes = [_PP, i32]
    lib.epl_ll_workspace_bytes.restype = ctypes.c_size_t
    lib.epl_ll_dispatch.argtypes = [_PP, i32, i64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]
    lib.epl_ll_dispatch.restype = i32
    lib.epl_combine.argtypes = [_PP, _P, i64, _P, _P, i32, _P, _P, _P]
    lib.epl_combine.restype = i32
    lib.epl_expert_scale.argtypes = [_PP, _P, _P, i64, _P, _P, _P]
    lib.epl_expert_scale.restype = i32
    pr, pp = ctypes.POINTER(Router), ctypes.POINTER(Product)
    lib.epl_router_validate.argtypes = [pr]
    lib.epl_router_validate.restype = i32
    lib.epl_route.argtypes = [pr, _P, _P, _P, _P, _P, _P]
    lib.epl_route.restype = i32
    lib.epl_route_backward.argtypes = [pr, _P, _P, _P, _P, _P]
    lib.epl_route_backward.restype = i32
    lib.epl_product_validate.argtypes = [pp]
    lib.epl_product_validate.restype = i32
    lib.epl_expert_product.argtypes = [pp, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]
    lib.epl_expert_product.restype = i32
    lib.epl_expert_weight_grad.argtypes = [pp, _P, _P, _P, _P, i32, _P, _P, _P, _P]
    lib.epl_expert_weight_grad.restype = i32
    for name in ("epl_product_workspace_bytes", "epl_weight_grad_workspace_bytes"):
        getattr(lib, name).argtypes = [pp]
        getattr(lib, name).restype = ctypes.c_size_t
    pc, pw, p8 = ctypes.POINTER(Cast), ctypes.POINTER(WeightCast), ctypes.POINTER(ProductFp8)
    for name, kind in (("epl_cast_validate", pc), ("epl_weight_cast_validate", pw),
                       ("epl_product_fp8_validate", p8)):
        getattr(lib, name).argtypes = [kind]
        getattr(lib, name).restype = i32
    for name in ("epl_quantize", "epl_dequantize"):
        getattr(lib, name).argtypes = [pc, _P, _P, _P, _P, _P, _P]
        getattr(lib, name).restype = i32
    lib.epl_quantize_weight.argtypes = [pw, _P, _P, _P, _P]
    lib.epl_quantize_weight.restype = i32
    lib.epl_product_fp8_workspace_bytes.argtypes = [p8]
    lib.epl_product_fp8_workspace_bytes.restype = ctypes.c_size_t
    lib.epl_expert_product_fp8.argtypes = [p8, *[_P] * 14]
    lib.epl_expert_product_fp8.restype = i32
    lib.epl_combine_backward.argtypes = [_PP, i32, _P, _P, i64, _P, _P, _P, _P, _P, _P]
    lib.epl_combine_backward.restype = i32
    lib.epl_status.argtypes = [_P, _P]
    lib.epl_status.restype = i32
    lib.epl_total.argtypes = [_P, _P]
    lib.epl_total.restype = i64
    lib.epl_strerror.argtypes = [i32]
    lib.epl_strerror.restype = ctypes.c_char_p
    lib.epl_version.argtypes = []
    lib.epl_version.restype = i32
    _LIB = lib
    return lib


# ----------------------------------------------------------- marshalling --

_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream, device=None) -> Optional[int]:
    if stream is None:
        torch = _torch()
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _need(t, name, dtype, shape=None, device=None, allow_none=False):
    torch = _torch()
    if t is None:
        if allow_none:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


WS_HEADER_BYTES = 256   # status word and total: all that combine / expert_scale / status touch


class StaticWorkspace:
    """The library's static workspace on one GPU (epl_dispatch_static): a
    device address, not a tensor. It can be passed wherever a workspace is
    taken after the dispatch that used it (epl_status, epl_total,
    epl_combine, epl_expert_scale)."""

    def __init__(self, address: int, device):
        self.address, self.device = int(address), device

    def data_ptr(self) -> int:
        return self.address

    def numel(self) -> int:
        return EPL_STATIC_WORKSPACE_BYTES

    def __repr__(self):
        return f"StaticWorkspace({self.address:#x}, {self.device})"


def _need_ws_arg(workspace, dev, allow_none=False):
    """A workspace argument: a uint8 tensor on `dev`, or the static workspace."""
    if isinstance(workspace, StaticWorkspace):
        if dev is not None and workspace.device != dev:
            raise ValueError(f"workspace is on {workspace.device}, expected {dev}")
        return
    _need(workspace, "workspace", _torch().uint8, None, dev, allow_none=allow_none)


def _need_workspace(workspace, need: int, where: str):
    """The C ABI takes the workspace as a bare pointer, so its size is checked
    here, before any launch: a workspace smaller than the problem needs would
    be written past its end."""
    if need <= 0:
        raise EplError(EPL_EINVAL, where)
    if workspace.numel() < need:
        raise ValueError(f"{where}: workspace holds {workspace.numel()} bytes, the problem needs "
                         f"{need} (epl_workspace_bytes)")


def _check(rc: int, where: str):
    if rc != EPL_OK:
        raise EplError(rc, where)


def _prob(p: Problem):
    return ctypes.byref(p)


# ------------------------------------------------------- C entry points --

def epl_version() -> int:
    return load().epl_version()


def epl_strerror(code: int) -> str:
    return load().epl_strerror(int(code)).decode()


def epl_validate(p: Problem) -> int:
    return load().epl_validate(_prob(p))


def epl_workspace_bytes(p: Problem) -> int:
    return int(load().epl_workspace_bytes(_prob(p)))


def epl_capacity_rows(p: Problem) -> int:
    return int(load().epl_capacity_rows(_prob(p)))


def _need_per_node(p: Problem, t, dev):
    """num_tokens_per_rdma_rank: [R / G] int32 when the problem spans several
    nodes; otherwise None (ignored by the library)."""
    if p.num_nodes:
        _need(t, "num_tokens_per_rdma_rank", _torch().int32, (p.num_nodes,), dev)


def epl_layout(p: Problem, topk_idx, num_tokens_per_expert, num_tokens_per_rank,
               num_tokens_per_rdma_rank, is_token_in_rank, workspace, stream=None):
    torch = _torch()
    T, K, E, R = p.num_tokens, p.num_topk, p.num_experts, p.num_ranks
    _need(topk_idx, "topk_idx", torch.int64, (T, K))
    dev = topk_idx.device
    _need(num_tokens_per_expert, "num_tokens_per_expert", torch.int32, (E,), dev)
    _need(num_tokens_per_rank, "num_tokens_per_rank", torch.int32, (R,), dev)
    _need_per_node(p, num_tokens_per_rdma_rank, dev)
    _need(is_token_in_rank, "is_token_in_rank", torch.uint8, (T, R), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    _need_workspace(workspace, epl_workspace_bytes(p), "epl_layout")
    _check(load().epl_layout(_prob(p), _ptr(topk_idx), _ptr(num_tokens_per_expert),
                             _ptr(num_tokens_per_rank), _ptr(num_tokens_per_rdma_rank),
                             _ptr(is_token_in_rank), _ptr(workspace), _stream(stream, dev)),
           "epl_layout")


def epl_scan(p: Problem, num_tokens_per_expert, expert_start_loc, total_host, workspace,
             stream=None):
    torch = _torch()
    E = p.num_experts
    _need(num_tokens_per_expert, "num_tokens_per_expert", torch.int32, (E,))
    dev = num_tokens_per_expert.device
    _need(expert_start_loc, "expert_start_loc", torch.int32, (E,), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    _need_workspace(workspace, epl_workspace_bytes(p), "epl_scan")
    if total_host is not None:
        if total_host.device.type != "cpu" or not total_host.is_pinned() or \
                total_host.dtype != torch.int32 or total_host.numel() < 1:
            raise ValueError("total_host must be a pinned CPU int32 tensor")
    _check(load().epl_scan(_prob(p), _ptr(num_tokens_per_expert), _ptr(expert_start_loc),
                           _ptr(total_host), _ptr(workspace), _stream(stream, dev)), "epl_scan")


def _check_scatter_args(p, x, x_scale, topk_idx, capacity_rows, out, out_scale, m_indices,
                        output_index):
    torch = _torch()
    T, K, H, S = p.num_tokens, p.num_topk, p.hidden, p.scale_cols
    _need(topk_idx, "topk_idx", torch.int64, (T, K))
    dev = topk_idx.device
    _need(x, "x", torch.bfloat16, (T, H), dev)
    _need(out, "out", torch.bfloat16, (capacity_rows, H), dev)
    _need(m_indices, "m_indices", torch.int32, (capacity_rows,), dev)
    _need(output_index, "output_index", torch.int32, (T, K), dev)
    if S > 0:
        _need(x_scale, "x_scale", torch.float32, (T, S), dev)
        _need(out_scale, "out_scale", torch.float32, (capacity_rows, S), dev)
    elif x_scale is not None or out_scale is not None:
        raise ValueError("scale tensors given but the problem has scale_cols == 0")
    return dev


def epl_scatter(p: Problem, x, x_scale, topk_idx, expert_start_loc, workspace, capacity_rows,
                out, out_scale, m_indices, output_index, stream=None):
    torch = _torch()
    dev = _check_scatter_args(p, x, x_scale, topk_idx, capacity_rows, out, out_scale, m_indices,
                              output_index)
    _need(expert_start_loc, "expert_start_loc", torch.int32, (p.num_experts,), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    _need_workspace(workspace, epl_workspace_bytes(p), "epl_scatter")
    _check(load().epl_scatter(_prob(p), _ptr(x), _ptr(x_scale), _ptr(topk_idx),
                              _ptr(expert_start_loc), _ptr(workspace), int(capacity_rows),
                              _ptr(out), _ptr(out_scale), _ptr(m_indices), _ptr(output_index),
                              _stream(stream, dev)), "epl_scatter")


def epl_dispatch(p: Problem, topk_idx, x, x_scale, capacity_rows, num_tokens_per_expert,
                 num_tokens_per_rank, num_tokens_per_rdma_rank, is_token_in_rank,
                 expert_start_loc, total_host, out, out_scale, m_indices, output_index, workspace,
                 stream=None):
    torch = _torch()
    dev = _check_scatter_args(p, x, x_scale, topk_idx, capacity_rows, out, out_scale, m_indices,
                              output_index)
    E, R, T = p.num_experts, p.num_ranks, p.num_tokens
    _need(num_tokens_per_expert, "num_tokens_per_expert", torch.int32, (E,), dev)
    _need(num_tokens_per_rank, "num_tokens_per_rank", torch.int32, (R,), dev)
    _need_per_node(p, num_tokens_per_rdma_rank, dev)
    _need(is_token_in_rank, "is_token_in_rank", torch.uint8, (T, R), dev)
    _need(expert_start_loc, "expert_start_loc", torch.int32, (E,), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    _need_workspace(workspace, epl_workspace_bytes(p), "epl_dispatch")
    if total_host is not None and (total_host.device.type != "cpu" or not total_host.is_pinned()
                                   or total_host.dtype != torch.int32):
        raise ValueError("total_host must be a pinned CPU int32 tensor")
    _check(load().epl_dispatch(_prob(p), _ptr(topk_idx), _ptr(x), _ptr(x_scale),
                               int(capacity_rows), _ptr(num_tokens_per_expert),
                               _ptr(num_tokens_per_rank), _ptr(num_tokens_per_rdma_rank),
                               _ptr(is_token_in_rank),
                               _ptr(expert_start_loc), _ptr(total_host), _ptr(out),
                               _ptr(out_scale), _ptr(m_indices), _ptr(output_index),
                               _ptr(workspace), _stream(stream, dev)), "epl_dispatch")


def epl_dispatch_static(p: Problem, topk_idx, x, x_scale, capacity_rows, num_tokens_per_expert,
                        num_tokens_per_rank, num_tokens_per_rdma_rank, is_token_in_rank,
                        expert_start_loc, total_host, out, out_scale, m_indices, output_index,
                        stream=None) -> StaticWorkspace:
    """epl_dispatch without a workspace argument, for callers that cannot
    allocate: the library's static workspace on the current GPU is used
    (EPL_STATIC_WORKSPACE_BYTES, shared by every such call on that GPU, so
    calls that overlap on one GPU race). Returns that workspace, for
    epl_status / epl_total / epl_combine / epl_expert_scale. Problems that
    need a larger workspace are rejected."""
    torch = _torch()
    dev = _check_scatter_args(p, x, x_scale, topk_idx, capacity_rows, out, out_scale, m_indices,
                              output_index)
    E, R, T = p.num_experts, p.num_ranks, p.num_tokens
    _need(num_tokens_per_expert, "num_tokens_per_expert", torch.int32, (E,), dev)
    _need(num_tokens_per_rank, "num_tokens_per_rank", torch.int32, (R,), dev)
    _need_per_node(p, num_tokens_per_rdma_rank, dev)
    _need(is_token_in_rank, "is_token_in_rank", torch.uint8, (T, R), dev)
    _need(expert_start_loc, "expert_start_loc", torch.int32, (E,), dev)
    need = epl_workspace_bytes(p)
    if need <= 0 or need > EPL_STATIC_WORKSPACE_BYTES:
        raise ValueError(f"epl_dispatch_static: the problem needs {need} bytes of workspace, "
                         f"the static workspace holds {EPL_STATIC_WORKSPACE_BYTES}")
    if total_host is not None and (total_host.device.type != "cpu" or not total_host.is_pinned()
                                   or total_host.dtype != torch.int32):
        raise ValueError("total_host must be a pinned CPU int32 tensor")
    addr = ctypes.c_void_p()
    _check(load().epl_dispatch_static(_prob(p), _ptr(topk_idx), _ptr(x), _ptr(x_scale),
                                      int(capacity_rows), _ptr(num_tokens_per_expert),
                                      _ptr(num_tokens_per_rank), _ptr(num_tokens_per_rdma_rank),
                                      _ptr(is_token_in_rank), _ptr(expert_start_loc),
                                      _ptr(total_host), _ptr(out), _ptr(out_scale),
                                      _ptr(m_indices), _ptr(output_index), ctypes.byref(addr),
                                      _stream(stream, dev)), "epl_dispatch_static")
    return StaticWorkspace(addr.value, dev)


def _check_fp8_args(p, x, x_scale, scale_format, topk_idx, capacity_rows, out, out_scale,
                    m_indices, output_index):
    torch = _torch()
    T, K, H, S = p.num_tokens, p.num_topk, p.hidden, p.scale_cols
    _need(topk_idx, "topk_idx", torch.int64, (T, K))
    dev = topk_idx.device
    _need(x, "x", torch.uint8, (T, H), dev)
    _need(out, "out", torch.uint8, (capacity_rows, H), dev)
    _need(m_indices, "m_indices", torch.int32, (capacity_rows,), dev)
    _need(output_index, "output_index", torch.int32, (T, K), dev)
    if scale_format == EPL_SCALE_F32:
        _need(x_scale, "x_scale", torch.float32, (T, S), dev)
        _need(out_scale, "out_scale", torch.float32, (capacity_rows, S), dev)
    elif scale_format == EPL_SCALE_UE8M0:
        W = (S + 3) // 4
        _need(x_scale, "x_scale", torch.int32, (T, W), dev)
        _need(out_scale, "out_scale (column-major storage [W, capacity])", torch.int32,
              (W, capacity_rows), dev)
    elif scale_format != EPL_SCALE_NONE:
        raise ValueError(f"unknown scale format {scale_format}")
    return dev


def epl_scatter_fp8(p: Problem, x, x_scale, scale_format, topk_idx, expert_start_loc, workspace,
                    capacity_rows, out, out_scale, m_indices, output_index, stream=None):
    """FP8 rows as uint8 [T, H] (view a float8_e4m3fn tensor as uint8); the
    UE8M0 output scale buffer is int32 [W, capacity] (its transpose is the
    [capacity, W] view the grouped GEMM reads)."""
    torch = _torch()
    dev = _check_fp8_args(p, x, x_scale, scale_format, topk_idx, capacity_rows, out, out_scale,
                          m_indices, output_index)
    _need(expert_start_loc, "expert_start_loc", torch.int32, (p.num_experts,), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    _need_workspace(workspace, epl_workspace_bytes(p), "epl_scatter_fp8")
    _check(load().epl_scatter_fp8(_prob(p), _ptr(x), _ptr(x_scale), int(scale_format),
                                  _ptr(topk_idx), _ptr(expert_start_loc), _ptr(workspace),
                                  int(capacity_rows), _ptr(out), _ptr(out_scale), _ptr(m_indices),
                                  _ptr(output_index), _stream(stream, dev)), "epl_scatter_fp8")


def epl_dispatch_fp8(p: Problem, topk_idx, x, x_scale, scale_format, capacity_rows,
                     num_tokens_per_expert, num_tokens_per_rank, num_tokens_per_rdma_rank,
                     is_token_in_rank, expert_start_loc, total_host, out, out_scale, m_indices,
                     output_index, workspace, stream=None):
    torch = _torch()
    dev = _check_fp8_args(p, x, x_scale, scale_format, topk_idx, capacity_rows, out, out_scale,
                          m_indices, output_index)
    E, R, T = p.num_experts, p.num_ranks, p.num_tokens
    _need(num_tokens_per_expert, "num_tokens_per_expert", torch.int32, (E,), dev)
    _need(num_tokens_per_rank, "num_tokens_per_rank", torch.int32, (R,), dev)
    _need_per_node(p, num_tokens_per_rdma_rank, dev)
    _need(is_token_in_rank, "is_token_in_rank", torch.uint8, (T, R), dev)
    _need(expert_start_loc, "expert_start_loc", torch.int32, (E,), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    _need_workspace(workspace, epl_workspace_bytes(p), "epl_dispatch_fp8")
    if total_host is not None and (total_host.device.type != "cpu" or not total_host.is_pinned()
                                   or total_host.dtype != torch.int32):
        raise ValueError("total_host must be a pinned CPU int32 tensor")
    _check(load().epl_dispatch_fp8(_prob(p), _ptr(topk_idx), _ptr(x), _ptr(x_scale),
                                   int(scale_format), int(capacity_rows),
                                   _ptr(num_tokens_per_expert), _ptr(num_tokens_per_rank),
                                   _ptr(num_tokens_per_rdma_rank), _ptr(is_token_in_rank),
                                   _ptr(expert_start_loc),
                                   _ptr(total_host), _ptr(out), _ptr(out_scale), _ptr(m_indices),
                                   _ptr(output_index), _ptr(workspace), _stream(stream, dev)),
           "epl_dispatch_fp8")


def epl_ll_workspace_bytes(p: Problem, tokens_per_segment: int) -> int:
    return int(load().epl_ll_workspace_bytes(_prob(p), int(tokens_per_segment)))


def epl_ll_dispatch(p: Problem, tokens_per_segment, rows_per_expert, topk_idx, x, out, out_scale,
                    recv_count, src_info, layout_range, output_index, workspace, stream=None):
    """Fixed-rectangle (low-latency) dispatch; shapes as in include/epl.h:
    out uint8 [E, cap, H], out_scale f32 [E, S, cap], recv_count i32 [E],
    src_info i32 [E, cap], layout_range i32 [E, T/M, 2], output_index i32
    [T, K]; x bf16 [T, H]."""
    torch = _torch()
    T, K, E, H = p.num_tokens, p.num_topk, p.num_experts, p.hidden
    M, cap = int(tokens_per_segment), int(rows_per_expert)
    if M < 1 or T % M:
        raise ValueError("num_tokens must be a multiple of tokens_per_segment")
    _need(topk_idx, "topk_idx", torch.int64, (T, K))
    dev = topk_idx.device
    _need(x, "x", torch.bfloat16, (T, H), dev)
    _need(out, "out", torch.uint8, (E, cap, H), dev)
    _need(out_scale, "out_scale", torch.float32, (E, H // 128, cap), dev)
    _need(recv_count, "recv_count", torch.int32, (E,), dev)
    _need(src_info, "src_info", torch.int32, (E, cap), dev)
    _need(layout_range, "layout_range", torch.int32, (E, T // M, 2), dev)
    _need(output_index, "output_index", torch.int32, (T, K), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    _need_workspace(workspace, epl_ll_workspace_bytes(p, M), "epl_ll_dispatch")
    _check(load().epl_ll_dispatch(_prob(p), M, cap, _ptr(topk_idx), _ptr(x), _ptr(out),
                                  _ptr(out_scale), _ptr(recv_count), _ptr(src_info),
                                  _ptr(layout_range), _ptr(output_index), _ptr(workspace),
                                  _stream(stream, dev)), "epl_ll_dispatch")


def epl_combine(p: Problem, expert_out, expert_rows, output_index, topk_weights, out_dtype, y,
                workspace=None, stream=None):
    torch = _torch()
    T, K, H = p.num_tokens, p.num_topk, p.hidden
    _need(output_index, "output_index", torch.int32, (T, K))
    dev = output_index.device
    _need(expert_out, "expert_out", torch.bfloat16, (expert_rows, H), dev)
    _need(topk_weights, "topk_weights", torch.float32, (T, K), dev)
    ydt = torch.bfloat16 if out_dtype == EPL_OUT_BF16 else torch.float32
    _need(y, "y", ydt, (T, H), dev)
    _need_ws_arg(workspace, dev, allow_none=True)
    if workspace is not None:
        _need_workspace(workspace, WS_HEADER_BYTES, "epl_combine")
    _check(load().epl_combine(_prob(p), _ptr(expert_out), int(expert_rows), _ptr(output_index),
                              _ptr(topk_weights), int(out_dtype), _ptr(y), _ptr(workspace),
                              _stream(stream, dev)), "epl_combine")


def epl_expert_scale(p: Problem, rows_in, m_indices, capacity_rows, rows_out, workspace,
                     stream=None):
    torch = _torch()
    H = p.hidden
    _need(rows_in, "rows_in", torch.bfloat16, (capacity_rows, H))
    dev = rows_in.device
    _need(m_indices, "m_indices", torch.int32, (capacity_rows,), dev)
    _need(rows_out, "rows_out", torch.bfloat16, (capacity_rows, H), dev)
    _need_ws_arg(workspace, dev)
    _need_workspace(workspace, WS_HEADER_BYTES, "epl_expert_scale")
    _check(load().epl_expert_scale(_prob(p), _ptr(rows_in), _ptr(m_indices), int(capacity_rows),
                                   _ptr(rows_out), _ptr(workspace), _stream(stream, dev)),
           "epl_expert_scale")


def _raw_stream(index: int) -> int:
    """torch's current stream on GPU `index`, without the Stream object
    around it (1.9 us) where torch offers that."""
    torch = _torch()
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(index) if get is not None else torch.cuda.current_stream(index).cuda_stream


def _launch(name: str, dev, stream, *args):
    """Call C entry point `name` with `dev` as the current device (kernels are
    launched on the current device, which need not be the tensors') and the
    stream last."""
    torch = _torch()
    fn = getattr(_LIB or load(), name)
    current = torch.cuda.current_device()
    index = current if dev.index is None else dev.index
    raw = _raw_stream(index) if stream is None else _stream(stream)
    if index == current:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc != EPL_OK:
        raise EplError(rc, name)


def _need_same(t, name, dtype, shape, dev):
    """_need with every condition given; the common case in one expression."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous() \
                and t.is_cuda:
            return
    except AttributeError:
        pass
    _need(t, name, dtype, shape, dev)


def _type_code(dtype, name) -> int:
    torch = _torch()
    if dtype == torch.float32:
        return EPL_OUT_F32
    if dtype == torch.bfloat16:
        return EPL_OUT_BF16
    raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {dtype}")


def epl_router_validate(p: Router) -> int:
    return load().epl_router_validate(ctypes.byref(p))


def _router_dtype(p: Router):
    return _torch().bfloat16 if p.logits_type == EPL_OUT_BF16 else _torch().float32


def epl_route(p: Router, logits, bias, token_mask, topk_idx, topk_weights, stream=None):
    torch = _torch()
    T, K = p.num_tokens, p.num_topk
    dev = getattr(logits, "device", None)
    _need_same(topk_idx, "topk_idx", torch.int64, (T, K), dev)
    _need_same(topk_weights, "topk_weights", torch.float32, (T, K), dev)
    _route(p, logits, bias, token_mask, topk_idx, topk_weights, stream)


def _route(p: Router, logits, bias, token_mask, topk_idx, topk_weights, stream):
    """epl_route with outputs that are known to fit."""
    torch = _torch()
    T, E = p.num_tokens, p.num_experts
    dev = getattr(logits, "device", None)
    _need_same(logits, "logits", _router_dtype(p), (T, E), dev)
    if bias is not None:
        _need_same(bias, "bias", torch.float32, (E,), dev)
    if token_mask is not None:
        _need_same(token_mask, "token_mask", torch.uint8, (T,), dev)
    _launch("epl_route", dev, stream, ctypes.byref(p), _ptr(logits), _ptr(bias), _ptr(token_mask),
            _ptr(topk_idx), _ptr(topk_weights))


def epl_route_backward(p: Router, logits, topk_idx, grad_weights, grad_logits, stream=None):
    torch = _torch()
    T, K, E = p.num_tokens, p.num_topk, p.num_experts
    dt = _router_dtype(p)
    dev = getattr(logits, "device", None)
    _need_same(logits, "logits", dt, (T, E), dev)
    _need_same(topk_idx, "topk_idx", torch.int64, (T, K), dev)
    _need_same(grad_weights, "grad_weights", torch.float32, (T, K), dev)
    _need_same(grad_logits, "grad_logits", dt, (T, E), dev)
    _launch("epl_route_backward", dev, stream, ctypes.byref(p), _ptr(logits), _ptr(topk_idx),
            _ptr(grad_weights), _ptr(grad_logits))


def epl_product_validate(p: Product) -> int:
    return load().epl_product_validate(ctypes.byref(p))


def _blocks(p: Product, expert_start_loc, num_tokens_per_expert, dev):
    torch = _torch()
    _need_same(expert_start_loc, "expert_start_loc", torch.int32, (p.num_experts,), dev)
    _need_same(num_tokens_per_expert, "num_tokens_per_expert", torch.int32, (p.num_experts,), dev)


def epl_product_workspace_bytes(p: Product) -> int:
    return int(load().epl_product_workspace_bytes(ctypes.byref(p)))


def epl_weight_grad_workspace_bytes(p: Product) -> int:
    return int(load().epl_weight_grad_workspace_bytes(ctypes.byref(p)))


def _need_split_ws(workspace, dev, need, where):
    """The optional workspace of the products: None, or all of it."""
    _need(workspace, "workspace", _torch().uint8, None, dev, allow_none=True)
    if workspace is not None and workspace.numel() < need:
        raise ValueError(f"{where}: workspace holds {workspace.numel()} bytes, the product needs "
                         f"{need}")


def epl_expert_product(p: Product, x, weight, bias, residual, expert_start_loc,
                       num_tokens_per_expert, pre, y, workspace=None, stream=None):
    torch = _torch()
    rows, E, K, N = p.num_rows, p.num_experts, p.in_cols, p.out_cols
    bf16 = torch.bfloat16
    dev = getattr(x, "device", None)
    _need_same(x, "x", bf16, (rows, K), dev)
    _need_same(weight, "weight", bf16,
               (E, K, N) if p.weight_layout == EPL_WEIGHT_IN_OUT else (E, N, K), dev)
    if bias is not None:
        _need_same(bias, "bias", torch.float32, (E, N), dev)
    grad = p.activation >= EPL_ACT_SILU_GRAD
    cols = N // 2 if p.activation == EPL_ACT_SWIGLU else \
        2 * N if p.activation == EPL_ACT_SWIGLU_GRAD else N
    if residual is not None:
        _need_same(residual, "residual", bf16, (rows, cols), dev)
    if pre is not None or grad:
        _need_same(pre, "pre", bf16, (rows, cols if grad else N), dev)
    _need_same(y, "y", bf16 if p.out_type == EPL_OUT_BF16 else torch.float32, (rows, cols), dev)
    _blocks(p, expert_start_loc, num_tokens_per_expert, dev)
    if workspace is not None:
        _need_split_ws(workspace, dev, epl_product_workspace_bytes(p), "epl_expert_product")
    _launch("epl_expert_product", dev, stream, ctypes.byref(p), _ptr(x), _ptr(weight), _ptr(bias),
            _ptr(residual), _ptr(expert_start_loc), _ptr(num_tokens_per_expert), _ptr(pre),
            _ptr(y), _ptr(workspace))


def epl_expert_weight_grad(p: Product, grad, x, expert_start_loc, num_tokens_per_expert,
                           accumulate, grad_weight, grad_bias=None, workspace=None, stream=None):
    torch = _torch()
    rows, E, K, N = p.num_rows, p.num_experts, p.in_cols, p.out_cols
    dev = getattr(grad, "device", None)
    _need_same(grad, "grad", torch.bfloat16, (rows, N), dev)
    _need_same(x, "x", torch.bfloat16, (rows, K), dev)
    _need_same(grad_weight, "grad_weight",
               torch.bfloat16 if p.out_type == EPL_OUT_BF16 else torch.float32, (E, N, K), dev)
    if grad_bias is not None:
        _need_same(grad_bias, "grad_bias", torch.float32, (E, N), dev)
    _blocks(p, expert_start_loc, num_tokens_per_expert, dev)
    if workspace is not None:
        _need_split_ws(workspace, dev, epl_weight_grad_workspace_bytes(p),
                       "epl_expert_weight_grad")
    _launch("epl_expert_weight_grad", dev, stream, ctypes.byref(p), _ptr(grad), _ptr(x),
            _ptr(expert_start_loc), _ptr(num_tokens_per_expert), int(bool(accumulate)),
            _ptr(grad_weight), _ptr(grad_bias), _ptr(workspace))


def epl_cast_validate(p: Cast) -> int:
    return load().epl_cast_validate(ctypes.byref(p))


def epl_weight_cast_validate(p: WeightCast) -> int:
    return load().epl_weight_cast_validate(ctypes.byref(p))


def epl_product_fp8_validate(p: ProductFp8) -> int:
    return load().epl_product_fp8_validate(ctypes.byref(p))


def epl_product_fp8_workspace_bytes(p: ProductFp8) -> int:
    return int(load().epl_product_fp8_workspace_bytes(ctypes.byref(p)))


def _groups(cols: int) -> int:
    return (cols + 127) // 128


def _need_row_scales(t, name, fmt, rows, groups, cap, dev):
    """Scales of 8-bit rows in one of the EPL_SCALE_* formats."""
    torch = _torch()
    if fmt == EPL_SCALE_UE8M0:
        _need_same(t, name, torch.int32, ((groups + 3) // 4, rows), dev)
    elif fmt == EPL_SCALE_F32_RECT:
        _need_same(t, name, torch.float32, (rows // max(cap, 1), groups, cap), dev)
    else:
        _need_same(t, name, torch.float32, (rows, groups), dev)


def _need_weight_scales(t, fmt, E, rows, cols, dev):
    _need_same(t, "weight_scale",
               _torch().uint8 if fmt == EPL_SCALE_UE8M0 else _torch().float32,
               (E, _groups(rows), _groups(cols)), dev)


def _cast_args(p: Cast, values, value_cols, codes, scale, expert_start_loc,
               num_tokens_per_expert):
    """The checks that both directions of a cast share; the device."""
    torch = _torch()
    rows, C = p.num_rows, p.cols
    dev = getattr(values, "device", None)
    _need_same(values, "values", torch.bfloat16 if p.value_type == EPL_OUT_BF16 else torch.float32,
               (rows, value_cols), dev)
    _need_same(codes, "codes", torch.uint8, (rows, C), dev)
    _need_row_scales(scale, "scale", p.scale_format, rows, _groups(C), p.rows_per_expert, dev)
    if p.num_experts:
        _blocks(p, expert_start_loc, num_tokens_per_expert, dev)
    elif expert_start_loc is not None or num_tokens_per_expert is not None:
        raise ValueError("blocks given but the cast has num_experts == 0")
    return dev


def epl_quantize(p: Cast, x, expert_start_loc, num_tokens_per_expert, codes, scale, stream=None):
    dev = _cast_args(p, x, p.cols * (2 if p.activation == EPL_ACT_SWIGLU else 1), codes, scale,
                     expert_start_loc, num_tokens_per_expert)
    _launch("epl_quantize", dev, stream, ctypes.byref(p), _ptr(x), _ptr(expert_start_loc),
            _ptr(num_tokens_per_expert), _ptr(codes), _ptr(scale))


def epl_dequantize(p: Cast, codes, scale, expert_start_loc, num_tokens_per_expert, y, stream=None):
    dev = _cast_args(p, y, p.cols, codes, scale, expert_start_loc, num_tokens_per_expert)
    _launch("epl_dequantize", dev, stream, ctypes.byref(p), _ptr(codes), _ptr(scale),
            _ptr(expert_start_loc), _ptr(num_tokens_per_expert), _ptr(y))


def epl_quantize_weight(p: WeightCast, weight, codes, scale, stream=None):
    torch = _torch()
    E, N, K = p.num_experts, p.out_cols, p.in_cols
    dev = getattr(weight, "device", None)
    _need_same(weight, "weight", torch.bfloat16 if p.value_type == EPL_OUT_BF16 else torch.float32,
               (E, N, K), dev)
    _need_same(codes, "codes", torch.uint8, (E, N, K), dev)
    _need_weight_scales(scale, p.scale_format, E, N, K, dev)
    _launch("epl_quantize_weight", dev, stream, ctypes.byref(p), _ptr(weight), _ptr(codes),
            _ptr(scale))


def epl_expert_product_fp8(p: ProductFp8, x, x_scale, weight, weight_scale, bias, residual,
                           expert_start_loc, num_tokens_per_expert, pre, y, codes=None,
                           codes_scale=None, workspace=None, stream=None):
    torch = _torch()
    rows, E, K, N = p.num_rows, p.num_experts, p.in_cols, p.out_cols
    bf16, u8 = torch.bfloat16, torch.uint8
    dev = getattr(x, "device", None)
    _need_same(x, "x", u8, (rows, K), dev)
    _need_row_scales(x_scale, "x_scale", p.scale_format, rows, _groups(K), p.rows_per_expert, dev)
    shape = (E, K, N) if p.weight_layout == EPL_WEIGHT_IN_OUT else (E, N, K)
    _need_same(weight, "weight", u8, shape, dev)
    _need_weight_scales(weight_scale, p.weight_scale_format, *shape, dev)
    if bias is not None:
        _need_same(bias, "bias", torch.float32, (E, N), dev)
    grad = p.activation >= EPL_ACT_SILU_GRAD
    cols = N // 2 if p.activation == EPL_ACT_SWIGLU else \
        2 * N if p.activation == EPL_ACT_SWIGLU_GRAD else N
    if residual is not None:
        _need_same(residual, "residual", bf16, (rows, cols), dev)
    if pre is not None or grad:
        _need_same(pre, "pre", bf16, (rows, cols if grad else N), dev)
    if y is not None or p.codes_scale_format == EPL_SCALE_NONE:
        _need_same(y, "y", bf16 if p.out_type == EPL_OUT_BF16 else torch.float32, (rows, cols), dev)
    if p.codes_scale_format != EPL_SCALE_NONE:
        _need_same(codes, "codes", u8, (rows, cols), dev)
        _need_row_scales(codes_scale, "codes_scale", p.codes_scale_format, rows, _groups(cols), 0,
                         dev)
    elif codes is not None or codes_scale is not None:
        raise ValueError("codes given but the product has codes_scale_format == EPL_SCALE_NONE")
    _blocks(p, expert_start_loc, num_tokens_per_expert, dev)
    if workspace is not None:
        _need_split_ws(workspace, dev, epl_product_fp8_workspace_bytes(p),
                       "epl_expert_product_fp8")
    _launch("epl_expert_product_fp8", dev, stream, ctypes.byref(p), _ptr(x), _ptr(x_scale),
            _ptr(weight), _ptr(weight_scale), _ptr(bias), _ptr(residual), _ptr(expert_start_loc),
            _ptr(num_tokens_per_expert), _ptr(pre), _ptr(y), _ptr(codes), _ptr(codes_scale),
            _ptr(workspace))


def epl_combine_backward(p: Problem, grad_y, expert_out, expert_rows, output_index, topk_weights,
                         grad_rows, grad_weights, workspace=None, stream=None):
    torch = _torch()
    T, K, H = p.num_tokens, p.num_topk, p.hidden
    dev = getattr(output_index, "device", None)
    _need_same(output_index, "output_index", torch.int32, (T, K), dev)
    code = _type_code(getattr(grad_y, "dtype", None), "grad_y")
    _need_same(grad_y, "grad_y", grad_y.dtype, (T, H), dev)
    _need_same(expert_out, "expert_out", torch.bfloat16, (expert_rows, H), dev)
    _need_same(topk_weights, "topk_weights", torch.float32, (T, K), dev)
    _need_same(grad_rows, "grad_rows", torch.bfloat16, (expert_rows, H), dev)
    _need_same(grad_weights, "grad_weights", torch.float32, (T, K), dev)
    _need_ws_arg(workspace, dev, allow_none=True)
    if workspace is not None:
        _need_workspace(workspace, WS_HEADER_BYTES, "epl_combine_backward")
    _launch("epl_combine_backward", dev, stream, _prob(p), code, _ptr(grad_y), _ptr(expert_out),
            int(expert_rows), _ptr(output_index), _ptr(topk_weights), _ptr(grad_rows),
            _ptr(grad_weights), _ptr(workspace))


def epl_status(workspace, stream=None) -> int:
    _need_workspace(workspace, WS_HEADER_BYTES, "epl_status")
    return int(load().epl_status(_ptr(workspace), _stream(stream, workspace.device)))


def epl_total(workspace, stream=None) -> int:
    _need_workspace(workspace, WS_HEADER_BYTES, "epl_total")
    n = int(load().epl_total(_ptr(workspace), _stream(stream, workspace.device)))
    if n < 0:
        raise EplError(n, "epl_total")
    return n


def prepare(name: str, *args, stream=None):
    """A zero-overhead caller of C entry point `name` with fixed arguments:
    tensors become their device addresses, a Problem is passed by reference,
    and the stream (default: torch's current stream) is resolved once. The
    arguments are not checked here: call the checked ``epl_*`` wrapper with
    the same arguments first (e.g. in a warm-up). Raises EplError on a non-zero
    return code."""
    import torch
    fn = getattr(load(), name)
    cargs = []
    for a in args:
        if isinstance(a, Problem):
            cargs.append(ctypes.byref(a))
        elif isinstance(a, torch.Tensor):
            cargs.append(ctypes.c_void_p(a.data_ptr()))
        else:
            cargs.append(a)
    cargs.append(ctypes.c_void_p(_stream(stream)))

    def call():
        rc = fn(*cargs)
        if rc != EPL_OK:
            raise EplError(rc, name)
    return call


# ------------------------------------------------------- tensor helpers --

def _run_on(stream, device, call, *args):
    """call(*args) with `stream` as torch's current stream: what it allocates,
    fills and launches is in that stream's order (memory taken from another
    stream's pool may still be in use there, and a fill on another stream is
    ordered with nothing). Its outputs are kept for the caller's stream too:
    they may be used and dropped there once it has waited for `stream`."""
    torch = _torch()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        out = call(*args)
    if stream.cuda_stream != caller.cuda_stream:
        for t in out if isinstance(out, tuple) else (out,):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(caller)
    return out


class DispatchResult(NamedTuple):
    out: "torch.Tensor"                  # [capacity, H] bf16 (rows >= total unwritten)
    out_scale: Optional["torch.Tensor"]  # [capacity, S] f32 or None
    m_indices: "torch.Tensor"            # [capacity] i32
    output_index: "torch.Tensor"         # [T, K] i32
    expert_start_loc: "torch.Tensor"     # [E] i32
    num_tokens_per_expert: "torch.Tensor"
    num_tokens_per_rank: "torch.Tensor"
    num_tokens_per_rdma_rank: Optional["torch.Tensor"]   # [R / G] i32, None on one node
    is_token_in_rank: "torch.Tensor"     # [T, R] u8 (0/1)
    total_host: "torch.Tensor"           # pinned [1] i32, valid after the stream syncs
    workspace: "torch.Tensor"
    problem: Problem

    def total(self) -> int:
        """Routed row count N (synchronises the current stream)."""
        _torch().cuda.current_stream(self.out.device).synchronize()
        return int(self.total_host[0])


def workspace_for(p: Problem, device):
    torch = _torch()
    n = epl_workspace_bytes(p)
    if n == 0:
        raise EplError(EPL_EINVAL, "epl_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def dispatch(x, topk_idx, num_experts: int, num_ranks: int, x_scale=None,
             capacity: Optional[int] = None, mode: str = "capacity", workspace=None,
             stream=None, expert_alignment: int = 0, ranks_per_node: int = 0) -> DispatchResult:
    """Layout + scan + scatter.

    mode="capacity" (default): one epl_dispatch call; the output buffers have
    `capacity` rows (default epl_capacity_rows, which always suffices) and no
    host wait happens. mode="exact": epl_layout + epl_scan, then the host waits for the
    total N, allocates exactly N rows and calls epl_scatter.

    Receive side: pass the rank's local expert ids (-1 for other ranks'
    experts) with num_experts = the local expert count and num_ranks = 1.
    """
    torch = _torch()
    if stream is not None and x.is_cuda:
        return _run_on(stream, x.device, dispatch, x, topk_idx, num_experts, num_ranks, x_scale,
                       capacity, mode, workspace, None, expert_alignment, ranks_per_node)
    T, H = x.shape
    K = topk_idx.shape[1]
    S = 0 if x_scale is None else x_scale.shape[1]
    p = Problem.make(T, K, num_experts, num_ranks, H, S, expert_alignment, ranks_per_node)
    _check(epl_validate(p), "epl_validate")
    dev = x.device
    ws = workspace if workspace is not None else workspace_for(p, dev)
    i32 = torch.int32
    cnt = torch.empty(num_experts, dtype=i32, device=dev)
    per_rank = torch.empty(num_ranks, dtype=i32, device=dev)
    per_node = torch.empty(p.num_nodes, dtype=i32, device=dev) if p.num_nodes else None
    in_rank = torch.empty((T, num_ranks), dtype=torch.uint8, device=dev)
    start = torch.empty(num_experts, dtype=i32, device=dev)
    oi = torch.empty((T, K), dtype=i32, device=dev)
    total_host = torch.zeros(1, dtype=i32, pin_memory=True)
    if mode == "capacity":
        cap = epl_capacity_rows(p) if capacity is None else int(capacity)
        out = torch.empty((cap, H), dtype=torch.bfloat16, device=dev)
        out_scale = torch.empty((cap, S), dtype=torch.float32, device=dev) if S else None
        m_idx = torch.empty(cap, dtype=i32, device=dev)
        epl_dispatch(p, topk_idx, x, x_scale, cap, cnt, per_rank, per_node, in_rank, start,
                     total_host, out, out_scale, m_idx, oi, ws)
    elif mode == "exact":
        epl_layout(p, topk_idx, cnt, per_rank, per_node, in_rank, ws)
        epl_scan(p, cnt, start, total_host, ws)
        torch.cuda.current_stream(dev).synchronize()
        cap = int(total_host[0])
        out = torch.empty((cap, H), dtype=torch.bfloat16, device=dev)
        out_scale = torch.empty((cap, S), dtype=torch.float32, device=dev) if S else None
        m_idx = torch.empty(cap, dtype=i32, device=dev)
        epl_scatter(p, x, x_scale, topk_idx, start, ws, cap, out, out_scale, m_idx, oi)
    else:
        raise ValueError(f"unknown mode {mode!r}")
    return DispatchResult(out, out_scale, m_idx, oi, start, cnt, per_rank, per_node, in_rank,
                          total_host, ws, p)


def combine(expert_out, output_index, topk_weights, out_dtype=None, workspace=None,
            stream=None):
    """y[t] = sum_k w[t,k] * expert_out[output_index[t,k]] (fp32 accumulation)."""
    torch = _torch()
    if stream is not None and expert_out.is_cuda:
        return _run_on(stream, expert_out.device, combine, expert_out, output_index, topk_weights,
                       out_dtype, workspace)
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    T, K = output_index.shape
    rows, H = expert_out.shape
    p = Problem.make(T, K, 1, 1, H, 0)
    code = EPL_OUT_BF16 if out_dtype == torch.bfloat16 else EPL_OUT_F32
    y = torch.empty((T, H), dtype=out_dtype, device=expert_out.device)
    epl_combine(p, expert_out, rows, output_index, topk_weights, code, y, workspace)
    return y


def expert_scale(res: DispatchResult, rows_in=None, stream=None):
    """The large-batch workload's synthetic expert applied to a dispatch result."""
    torch = _torch()
    rows_in = res.out if rows_in is None else rows_in
    if stream is not None and rows_in.is_cuda:
        return _run_on(stream, rows_in.device, expert_scale, res, rows_in)
    out = torch.empty_like(rows_in)
    epl_expert_scale(res.problem, rows_in, res.m_indices, rows_in.shape[0], out, res.workspace)
    return out


@functools.lru_cache(maxsize=256)
def _router_for(*fields) -> Router:
    """A checked description; the same sizes come again and again."""
    p = Router(*fields, 0)
    _check(epl_router_validate(p), "epl_router_validate")
    return p


@functools.lru_cache(maxsize=256)
def _combine_problem(T: int, K: int, H: int) -> Problem:
    p = Problem.make(T, K, 1, 1, H, 0)
    _check(epl_validate(p), "epl_validate")
    return p


@functools.lru_cache(maxsize=256)
def _product_for(*fields):
    """A checked description and its workspace's bytes."""
    p = Product(*fields, 0)
    _check(epl_product_validate(p), "epl_product_validate")
    return p, epl_product_workspace_bytes(p)


def _split_ws(nbytes, device):
    """A product's workspace, from torch's allocator."""
    if nbytes == 0:
        return None
    torch = _torch()
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


_SCORES = {"softmax": EPL_SCORE_SOFTMAX, "sigmoid": EPL_SCORE_SIGMOID}
_ACTIVATIONS = {"none": EPL_ACT_NONE, "silu": EPL_ACT_SILU, "gelu": EPL_ACT_GELU,
                "swiglu": EPL_ACT_SWIGLU, "silu_grad": EPL_ACT_SILU_GRAD,
                "gelu_grad": EPL_ACT_GELU_GRAD, "swiglu_grad": EPL_ACT_SWIGLU_GRAD}


def _named(table, name, what):
    try:
        return table[name]
    except (KeyError, TypeError):
        raise ValueError(f"unknown {what} {name!r}; choose from {sorted(table)}") from None


def _matrix(t, name, dims):
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(t.shape)}")


def route(logits, num_topk: int, score: str = "softmax", bias=None, num_groups: int = 1,
          topk_groups: int = 1, group_top: int = 1, renormalize: bool = False, scale: float = 1.0,
          token_mask=None, stream=None):
    """Router: (topk_idx int64 [T, K], topk_weights fp32 [T, K]) from logits
    [T, E] (fp32 or bf16), as `dispatch` and `combine` take them; the rules
    are those of epl_route in include/epl.h. `token_mask` (uint8 [T], 0 =
    padding) gives a token no selection at all."""
    torch = _torch()
    _matrix(logits, "logits", 2)
    if stream is not None and logits.is_cuda:
        return _run_on(stream, logits.device, route, logits, num_topk, score, bias, num_groups,
                       topk_groups, group_top, renormalize, scale, token_mask)
    T, E = logits.shape
    K = int(num_topk)
    p = _router_for(T, K, E, _named(_SCORES, score, "score"), int(num_groups), int(topk_groups),
                    int(group_top), int(bool(renormalize)), _type_code(logits.dtype, "logits"),
                    float(scale))
    dev = logits.device
    idx = torch.empty(T, K, dtype=torch.int64, device=dev)       # (a tuple takes 0.7 us more)
    w = torch.empty(T, K, dtype=torch.float32, device=dev)
    _route(p, logits, bias, token_mask, idx, w, None)
    return idx, w


def route_backward(logits, topk_idx, grad_weights, score: str = "softmax",
                   renormalize: bool = False, scale: float = 1.0, stream=None):
    """Gradient of `route`'s logits (their dtype) from that of its weights,
    for the choice topk_idx it made."""
    torch = _torch()
    _matrix(logits, "logits", 2)
    _matrix(topk_idx, "topk_idx", 2)
    if stream is not None and logits.is_cuda:
        return _run_on(stream, logits.device, route_backward, logits, topk_idx, grad_weights, score,
                       renormalize, scale)
    T, E = logits.shape
    p = _router_for(T, topk_idx.shape[1], E, _named(_SCORES, score, "score"), 1, 1, 1,
                    int(bool(renormalize)), _type_code(logits.dtype, "logits"), float(scale))
    grad = torch.empty_like(logits)
    epl_route_backward(p, logits, topk_idx, grad_weights, grad)
    return grad


def expert_product(x, weight, expert_start_loc, num_tokens_per_expert, bias=None,
                   activation: str = "none", residual=None, pre=None, out=None, out_dtype=None,
                   transposed: bool = False, expected_rows: int = 0, workspace=None, stream=None):
    """act(x @ weight[e]^T + bias[e]) + residual for the rows of each expert
    (x [rows, K] bf16, e.g. DispatchResult.out; weight [E, N, K] bf16), as
    epl_expert_product in include/epl.h. transposed=True takes weight as
    [E, K, N] and multiplies by it as it is: with the forward pass's array
    that is the data gradient. `pre` (bf16 [rows, N]) receives the product
    before the activation, or feeds a "..._grad" activation. Rows outside the
    experts' blocks are not written: pass `out` to choose what they hold.
    A workspace is taken from torch's allocator where none is passed."""
    torch = _torch()
    _matrix(x, "x", 2)
    _matrix(weight, "weight", 3)
    if stream is not None and x.is_cuda:
        return _run_on(stream, x.device, expert_product, x, weight, expert_start_loc,
                       num_tokens_per_expert, bias, activation, residual, pre, out, out_dtype,
                       transposed, expected_rows, workspace)
    E = weight.shape[0]
    N = weight.shape[2] if transposed else weight.shape[1]
    act = _named(_ACTIVATIONS, activation, "activation")
    if out is not None:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = torch.bfloat16
    p, ws_bytes = _product_for(x.shape[0], int(expected_rows), E, x.shape[1], N,
                               EPL_WEIGHT_IN_OUT if transposed else EPL_WEIGHT_OUT_IN, act,
                               _type_code(out_dtype, "out"))
    if out is None:
        cols = N // 2 if act == EPL_ACT_SWIGLU else 2 * N if act == EPL_ACT_SWIGLU_GRAD else N
        out = torch.empty((x.shape[0], cols), dtype=out_dtype, device=x.device)
    if workspace is None and x.is_cuda:
        workspace = _split_ws(ws_bytes, x.device)
    epl_expert_product(p, x, weight, bias, residual, expert_start_loc, num_tokens_per_expert, pre,
                       out, workspace)
    return out


def expert_weight_grad(grad, x, expert_start_loc, num_tokens_per_expert, out=None, out_dtype=None,
                       bias_grad=None, accumulate: bool = False, workspace=None, stream=None,
                       expected_rows: int = 0):
    """Gradient of expert_product's weight, [E, N, K], from that of its
    product `grad` (bf16 [rows, N]) and its input x (bf16 [rows, K]).
    `bias_grad` (fp32 [E, N]) receives the bias's. accumulate=True adds to
    what `out` and `bias_grad` hold. `expected_rows` chooses the kernel, as
    for expert_product: give it where the buffers have many more rows than
    the experts."""
    torch = _torch()
    _matrix(grad, "grad", 2)
    _matrix(x, "x", 2)
    _matrix(expert_start_loc, "expert_start_loc", 1)
    if stream is not None and x.is_cuda:
        return _run_on(stream, x.device, expert_weight_grad, grad, x, expert_start_loc,
                       num_tokens_per_expert, out, out_dtype, bias_grad, accumulate, workspace,
                       None, expected_rows)
    E, N, K = expert_start_loc.shape[0], grad.shape[1], x.shape[1]
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((E, N, K), dtype=torch.bfloat16 if out_dtype is None else out_dtype,
                          device=x.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
    p, _ = _product_for(grad.shape[0], int(expected_rows), E, K, N, EPL_WEIGHT_OUT_IN, EPL_ACT_NONE,
                        _type_code(out.dtype, "out"))
    if workspace is None and x.is_cuda:
        workspace = _split_ws(epl_weight_grad_workspace_bytes(p), x.device)
    epl_expert_weight_grad(p, grad, x, expert_start_loc, num_tokens_per_expert, accumulate, out,
                           bias_grad, workspace)
    return out


@functools.lru_cache(maxsize=256)
def _cast_for(*fields) -> Cast:
    p = Cast(*fields, 0, 0)
    _check(epl_cast_validate(p), "epl_cast_validate")
    return p


@functools.lru_cache(maxsize=256)
def _weight_cast_for(*fields) -> WeightCast:
    p = WeightCast(*fields, 0)
    _check(epl_weight_cast_validate(p), "epl_weight_cast_validate")
    return p


@functools.lru_cache(maxsize=256)
def _product_fp8_for(*fields):
    """A checked description and its workspace's bytes."""
    p = ProductFp8(*fields, 0, 0)
    _check(epl_product_fp8_validate(p), "epl_product_fp8_validate")
    return p, epl_product_fp8_workspace_bytes(p)


_FORMATS = {"f32": EPL_SCALE_F32, "ue8m0": EPL_SCALE_UE8M0}
_CAST_ACTIVATIONS = {"none": EPL_ACT_NONE, "swiglu": EPL_ACT_SWIGLU}


def _scale_kind(scale, rows: int, name: str):
    """(format, rows per expert) of row scales, by their type and shape."""
    torch = _torch()
    if not isinstance(scale, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if scale.dtype == torch.int32:
        return EPL_SCALE_UE8M0, 0
    if scale.dtype != torch.float32:
        raise TypeError(f"{name} must be torch.float32 or torch.int32, got {scale.dtype}")
    if scale.dim() == 3:
        return EPL_SCALE_F32_RECT, scale.shape[2]
    return EPL_SCALE_F32, 0


def _row_scales(fmt: int, rows: int, cols: int, device):
    """A buffer for the scales of `rows` rows."""
    torch = _torch()
    S = _groups(cols)
    if fmt == EPL_SCALE_UE8M0:
        return torch.empty((S + 3) // 4, rows, dtype=torch.int32, device=device)
    return torch.empty(rows, S, dtype=torch.float32, device=device)


def _num_blocks(expert_start_loc, num_tokens_per_expert) -> int:
    if expert_start_loc is None and num_tokens_per_expert is None:
        return 0
    _matrix(expert_start_loc, "expert_start_loc", 1)
    if expert_start_loc.shape[0] == 0:
        raise ValueError("expert_start_loc is empty")
    return expert_start_loc.shape[0]


def quantize(x, activation: str = "none", scale_format: str = "f32", expert_start_loc=None,
             num_tokens_per_expert=None, out=None, out_scale=None, stream=None):
    """(codes uint8 [rows, C], scales) of rows x [rows, C] (bf16 or fp32), a
    scale for each 128 columns, as epl_quantize in include/epl.h: what
    epl_dispatch_fp8 and expert_product_fp8 take. activation="swiglu" casts
    silu(x[:, :C]) * x[:, C:] of x [rows, 2C]. scale_format "f32": fp32 [rows,
    C / 128]; "ue8m0": powers of two, int32 [C / 512, rows]; `out_scale` has its format
    by itself (also the low-latency rectangle's fp32 [E, C / 128, cap]). With the experts'
    blocks only their rows are cast: pass `out` and `out_scale` to choose what
    the others hold."""
    torch = _torch()
    _matrix(x, "x", 2)
    if stream is not None and x.is_cuda:
        return _run_on(stream, x.device, quantize, x, activation, scale_format, expert_start_loc,
                       num_tokens_per_expert, out, out_scale)
    act = _named(_CAST_ACTIVATIONS, activation, "activation")
    rows, C = x.shape
    if act == EPL_ACT_SWIGLU:
        if C % 2:
            raise ValueError(f"x must have an even number of columns, got {C}")
        C //= 2
    if out_scale is not None:
        fmt, cap = _scale_kind(out_scale, rows, "out_scale")
    else:
        fmt, cap = _named(_FORMATS, scale_format, "scale format"), 0
    p = _cast_for(rows, _num_blocks(expert_start_loc, num_tokens_per_expert), C,
                  _type_code(x.dtype, "x"), act, fmt, cap)
    if out is None:
        out = torch.empty(rows, C, dtype=torch.uint8, device=x.device)
    if out_scale is None:
        out_scale = _row_scales(fmt, rows, C, x.device)
    epl_quantize(p, x, expert_start_loc, num_tokens_per_expert, out, out_scale)
    return out, out_scale


def dequantize(codes, scale, expert_start_loc=None, num_tokens_per_expert=None, out=None,
               out_dtype=None, stream=None):
    """code * scale, bf16 or fp32 [rows, C], of 8-bit rows: codes uint8 [rows,
    C] with scales of any format of the dispatch (fp32 [rows, C / 128], int32
    [C / 512, rows], or the low-latency rectangle's fp32 [E, C / 128, cap] with
    rows = E cap). With the experts' blocks only their rows are written: pass
    `out` to choose what the others hold."""
    torch = _torch()
    _matrix(codes, "codes", 2)
    if stream is not None and codes.is_cuda:
        return _run_on(stream, codes.device, dequantize, codes, scale, expert_start_loc,
                       num_tokens_per_expert, out, out_dtype)
    rows, C = codes.shape
    if out is not None:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
    else:
        out = torch.empty(rows, C, dtype=torch.bfloat16 if out_dtype is None else out_dtype,
                          device=codes.device)
    fmt, cap = _scale_kind(scale, rows, "scale")
    p = _cast_for(rows, _num_blocks(expert_start_loc, num_tokens_per_expert), C,
                  _type_code(out.dtype, "out"), EPL_ACT_NONE, fmt, cap)
    epl_dequantize(p, codes, scale, expert_start_loc, num_tokens_per_expert, out)
    return out


def quantize_weight(weight, scale_format: str = "f32", out=None, out_scale=None, stream=None):
    """(codes uint8 [E, N, K], scales [E, N / 128, K / 128]) of weights [E, N,
    K] (bf16 or fp32), a scale for each 128 x 128 block: fp32, or with "ue8m0"
    (or a uint8 `out_scale`) powers of two as uint8 exponents."""
    torch = _torch()
    _matrix(weight, "weight", 3)
    if stream is not None and weight.is_cuda:
        return _run_on(stream, weight.device, quantize_weight, weight, scale_format, out, out_scale)
    E, N, K = weight.shape
    fmt = _named(_FORMATS, scale_format, "scale format")
    if out_scale is not None:
        fmt = EPL_SCALE_UE8M0 if out_scale.dtype == torch.uint8 else EPL_SCALE_F32
    p = _weight_cast_for(E, N, K, _type_code(weight.dtype, "weight"), fmt)
    if out is None:
        out = torch.empty(E, N, K, dtype=torch.uint8, device=weight.device)
    if out_scale is None:
        out_scale = torch.empty(E, _groups(N), _groups(K), device=weight.device,
                                dtype=torch.uint8 if fmt == EPL_SCALE_UE8M0 else torch.float32)
    epl_quantize_weight(p, weight, out, out_scale)
    return out, out_scale


def expert_product_fp8(x, x_scale, weight, weight_scale, expert_start_loc, num_tokens_per_expert,
                       bias=None, activation: str = "none", residual=None, pre=None, out=None,
                       out_dtype=None, quantized=None, transposed: bool = False,
                       expected_rows: int = 0, workspace=None, stream=None):
    """expert_product on 8-bit rows and weights, as epl_expert_product_fp8 in
    include/epl.h: x codes uint8 [rows, K] with x_scale of any format of the
    dispatch (see `dequantize`), weight codes uint8 [E, N, K] ([E, K, N] with
    transposed=True) with weight_scale as `quantize_weight` makes them.

    `quantized` asks for the result's cast: "f32" or "ue8m0", or the buffers
    (codes, scales) that receive it. Returns the result (bf16, or `out_dtype`);
    with `quantized` (codes, scales) alone, or (out, codes, scales) where `out`
    or `out_dtype` asks for both.

    `expected_rows`, about how many rows the experts hold together, chooses the
    kernel (0: all of x's rows). Give it where the buffers have many more, as
    the low-latency rectangle has."""
    torch = _torch()
    _matrix(x, "x", 2)
    _matrix(weight, "weight", 3)
    if stream is not None and x.is_cuda:
        return _run_on(stream, x.device, expert_product_fp8, x, x_scale, weight, weight_scale,
                       expert_start_loc, num_tokens_per_expert, bias, activation, residual, pre,
                       out, out_dtype, quantized, transposed, expected_rows, workspace)
    E, rows = weight.shape[0], x.shape[0]
    N = weight.shape[2] if transposed else weight.shape[1]
    act = _named(_ACTIVATIONS, activation, "activation")
    cols = N // 2 if act == EPL_ACT_SWIGLU else 2 * N if act == EPL_ACT_SWIGLU_GRAD else N
    if out is not None:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
        out_dtype = out.dtype
    elif out_dtype is None:
        if quantized is None:
            out_dtype = torch.bfloat16
    codes = codes_scale = None
    to = EPL_SCALE_NONE
    if isinstance(quantized, tuple):
        codes, codes_scale = quantized
        to, cap = _scale_kind(codes_scale, rows, "quantized scales")
        if to == EPL_SCALE_F32_RECT:
            raise ValueError("quantized scales must be fp32 [rows, groups] or int32")
    elif quantized is not None:
        to = _named(_FORMATS, quantized, "scale format")
    fmt, cap = _scale_kind(x_scale, rows, "x_scale")
    w_fmt = EPL_SCALE_UE8M0 if getattr(weight_scale, "dtype", None) == torch.uint8 else EPL_SCALE_F32
    p, ws_bytes = _product_fp8_for(
        rows, int(expected_rows), E, x.shape[1], N,
        EPL_WEIGHT_IN_OUT if transposed else EPL_WEIGHT_OUT_IN, act,
        EPL_OUT_BF16 if out_dtype is None else _type_code(out_dtype, "out"), fmt, cap, w_fmt, to)
    if out is None and out_dtype is not None:
        out = torch.empty(rows, cols, dtype=out_dtype, device=x.device)
    if to != EPL_SCALE_NONE and codes is None:
        codes = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
        codes_scale = _row_scales(to, rows, cols, x.device)
    if workspace is None and x.is_cuda:
        workspace = _split_ws(ws_bytes, x.device)
    epl_expert_product_fp8(p, x, x_scale, weight, weight_scale, bias, residual, expert_start_loc,
                           num_tokens_per_expert, pre, out, codes, codes_scale, workspace)
    if codes is None:
        return out
    return (codes, codes_scale) if out is None else (out, codes, codes_scale)


def gated_block_fp8(x, x_scale, w1, w1_scale, w2, w2_scale, expert_start_loc,
                    num_tokens_per_expert, pre=None, out=None, expected_rows: int = 0,
                    scale_format: str = "f32", stream=None):
    """The experts' gated feed-forward block on 8-bit rows: h = silu(x W1g^T)
    * (x W1u^T) and its cast in one product (w1 [E, 2F, H], gate rows first),
    then h W2^T (w2 [E, H, F]), bf16 [rows, H]. F is a multiple of 128. x,
    weights and their scales are as expert_product_fp8 takes them; h is cast
    with `scale_format` scales. `pre` (bf16 [rows, 2F]) receives x W1^T for
    gated_block_fp8_backward. Rows outside the experts' blocks are not
    written. `expected_rows` as for expert_product_fp8: 64 rows in a rectangle
    of 8 x 128 take 80 us with it and 115 without (H 7168, F 2048)."""
    _matrix(x, "x", 2)
    if stream is not None and x.is_cuda:
        return _run_on(stream, x.device, gated_block_fp8, x, x_scale, w1, w1_scale, w2, w2_scale,
                       expert_start_loc, num_tokens_per_expert, pre, out, expected_rows,
                       scale_format)
    h, h_scale = expert_product_fp8(x, x_scale, w1, w1_scale, expert_start_loc,
                                    num_tokens_per_expert, activation="swiglu", pre=pre,
                                    quantized=scale_format, expected_rows=expected_rows)
    return expert_product_fp8(h, h_scale, w2, w2_scale, expert_start_loc, num_tokens_per_expert,
                              out=out, expected_rows=expected_rows)


def gated_block_fp8_backward(grad_y, pre, w1, w1_scale, w2, w2_scale, expert_start_loc,
                             num_tokens_per_expert, grad_x=None, grad_pre=None,
                             expected_rows: int = 0, scale_format: str = "f32", stream=None):
    """Gradients of gated_block_fp8: (grad_x bf16 [rows, H], grad_pre bf16
    [rows, 2F]) from grad_y (bf16 or fp32 [rows, H], e.g. of combine_backward) and the
    `pre` it kept. grad_y is cast to 8 bits for the product with W2, and
    grad_pre, whose cast leaves that product's epilogue too, for the one with
    W1. Casts pass gradients through. Rows outside the experts' blocks are not
    written. The weights' gradients are expert_weight_grad(grad_pre, x) and
    expert_weight_grad(grad_y, h) on bf16 rows: grad_pre and (bf16) grad_y as
    they are, x by `dequantize`, and h, which the block does not keep, from
    `pre`: dequantize(*quantize(pre, activation="swiglu", ..), ..)."""
    torch = _torch()
    _matrix(grad_y, "grad_y", 2)
    _matrix(w2, "w2", 3)
    if stream is not None and grad_y.is_cuda:
        return _run_on(stream, grad_y.device, gated_block_fp8_backward, grad_y, pre, w1, w1_scale,
                       w2, w2_scale, expert_start_loc, num_tokens_per_expert, grad_x, grad_pre,
                       expected_rows, scale_format)
    dy, dy_scale = quantize(grad_y, scale_format=scale_format, expert_start_loc=expert_start_loc,
                            num_tokens_per_expert=num_tokens_per_expert)
    grad_pre, dz, dz_scale = expert_product_fp8(
        dy, dy_scale, w2, w2_scale, expert_start_loc, num_tokens_per_expert,
        activation="swiglu_grad", pre=pre, out=grad_pre, out_dtype=torch.bfloat16,
        quantized=scale_format, transposed=True, expected_rows=expected_rows)
    grad_x = expert_product_fp8(dz, dz_scale, w1, w1_scale, expert_start_loc,
                                num_tokens_per_expert, out=grad_x, transposed=True,
                                expected_rows=expected_rows)
    return grad_x, grad_pre


def combine_backward(grad_y, expert_out, output_index, topk_weights, grad_rows=None,
                     workspace=None, stream=None):
    """Gradients of `combine`: (grad_rows bf16 like expert_out, grad_weights
    fp32 [T, K]). Rows that no slot names are not written: pass `grad_rows` to
    choose what they hold."""
    torch = _torch()
    _matrix(output_index, "output_index", 2)
    _matrix(expert_out, "expert_out", 2)
    if stream is not None and expert_out.is_cuda:
        return _run_on(stream, expert_out.device, combine_backward, grad_y, expert_out,
                       output_index, topk_weights, grad_rows, workspace)
    T, K = output_index.shape
    rows, H = expert_out.shape
    p = _combine_problem(T, K, H)
    if grad_rows is None:
        grad_rows = torch.empty_like(expert_out)
    grad_weights = torch.empty(T, K, dtype=torch.float32, device=expert_out.device)
    epl_combine_backward(p, grad_y, expert_out, rows, output_index, topk_weights, grad_rows,
                         grad_weights, workspace)
    return grad_rows, grad_weights


def dispatch_backward(grad_rows, output_index, out_dtype=None, workspace=None, stream=None):
    """Gradient of `dispatch`'s x [T, H]: the sum of a token's rows of
    grad_rows, i.e. `combine` with unit weights."""
    torch = _torch()
    _matrix(output_index, "output_index", 2)
    if stream is not None and output_index.is_cuda:
        return _run_on(stream, output_index.device, dispatch_backward, grad_rows, output_index,
                       out_dtype, workspace)
    dev = output_index.device
    ones = torch.ones(output_index.shape, dtype=torch.float32, device=dev)
    if output_index.is_cuda and dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev.index):         # kernels go to the current GPU
            return combine(grad_rows, output_index, ones, out_dtype, workspace)
    return combine(grad_rows, output_index, ones, out_dtype, workspace)
