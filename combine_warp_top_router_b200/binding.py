"""Thin ctypes binding of libmoedispatch (include/moedispatch.h).

Argument marshalling only: every function checks tensor placement, dtype and
contiguity, allocates outputs with torch when the caller passes none, and calls
the C entry point of the same name on the current CUDA stream, or as in
`torch.cuda.stream(stream)` where `stream=` is given.  All arithmetic runs in
the library's kernels.  If libmoedispatch.so is missing the first call raises;
there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import threading
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoedispatch.so")

MD_OK, MD_ERR_ARG, MD_ERR_UNSUPPORTED, MD_ERR_CUDA = 0, 1, 2, 3
MD_ERR_WORKSPACE, MD_ERR_DATA, MD_ERR_TIMEOUT = 4, 5, 6
MD_CONV, MD_DEDUP = 0, 1
MD_GATE_TOPK_SOFTMAX, MD_GATE_FULL_SOFTMAX = 0, 1
MD_COMBINE_FUSED, MD_COMBINE_WIRE = 0, 1
MD_SEED_CONTIGUOUS, MD_SEED_GREEDY_PAIRS = 0, 1
MD_REFINE_NONE, MD_REFINE_SWAPS, MD_REFINE_KL = 0, 1, 2
MD_PERMUTE_AUTO, MD_PERMUTE_BULK, MD_PERMUTE_VECTOR = 0, 1, 2
MD_LAYOUT_AUTO, MD_LAYOUT_COOPERATIVE, MD_LAYOUT_SPLIT = 0, 1, 2
MD_W_NK, MD_W_KN = 0, 1
MD_F32, MD_BF16 = 0, 1
MD_EXPERT_AUTO, MD_EXPERT_FEW, MD_EXPERT_ONE, MD_EXPERT_TWO = 0, 1, 2, 3
MD_CHECKPOINT_BLOCK = 32  # columns that share a scale of the 8-bit checkpoint

_lock = threading.Lock()
_lib = None

_P, _I, _L, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_SIGNATURES = {
    "md_status_string": ([_I], ctypes.c_char_p),
    "md_version": ([], _I),
    "md_launch_count": ([], ctypes.c_uint64),
    "md_memset_count": ([], ctypes.c_uint64),
    "md_route_topk": ([_P, _L, _I, _I, _I, _P, _P, _P], _I),
    "md_dispatch_layout_workspace_size": ([_L, _I, _I, _I, _I], _S),
    "md_dispatch_layout": ([_P, _L, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                            _P, _S, _P, _P], _I),
    "md_dispatch_layout_noalloc_max_scratch": ([], _S),
    "md_dispatch_layout_noalloc": ([_P, _L, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P,
                                    _P, _P, _P], _I),
    "md_dispatch_permute": ([_P, _L, _I, _I, _P, _L, _P, _P, _P], _I),
    "md_set_permute_path": ([_I], _I),
    "md_set_layout_path": ([_I], _I),
    "md_exchange_plan": ([_P, _I, _I, _P, _P], _I),
    "md_dispatch_exchange": ([_P, _L, _I, _I, _P, _P, _P, _I, _I, _P, _P, _L, _P, _P, _P], _I),
    "md_combine_partials": ([_P, _L, _P, _P, _P, _L, _I, _I, _P, _P, _P], _I),
    "md_combine_exchange": ([_P, _L, _I, _I, _P, _P, _I, _I, _P, _P, _P, _P, _P], _I),
    "md_dedup_expand": ([_P, _L, _I, _P, _P, _L, _I, _L, _P, _P, _P], _I),
    "md_combine": ([_P, _L, _P, _P, _P, _L, _I, _I, _I, _P, _L, _P, _P, _P, _P], _I),
    "md_coselect_stats": ([_P, _P, _L, _I, _I, _P, _P, _I, _P, _P], _I),
    "md_place_correlated_workspace_size": ([_I, _I], _S),
    "md_place_correlated": ([_P, _I, _I, _I, _I, _P, _P, _S, _P, _P], _I),
    "md_token_shuffle_workspace_size": ([_L, _I, _I], _S),
    "md_token_shuffle": ([_P, _I, _P, _P, _L, _I, _I, _P, _P, _P, _P, _S, _P, _P], _I),
    "md_coselect_pair_stats": ([_P, _P, _P, _L, _I, _I, _P, _I, _P, _P], _I),
    "md_token_shuffle_rounds_workspace_size": ([_L, _I, _I], _S),
    "md_token_shuffle_rounds": ([_P, _I, _P, _P, _L, _I, _I, _P, _P, _P, _P, _P, _S, _P, _P], _I),
    "md_rank_stats": ([_P, _L, _I, _I, _I, _P, _P, _P, _P], _I),
    "md_set_test_hooks": ([ctypes.c_longlong, _I, ctypes.c_longlong], None),
    "md_place_two_level_workspace_size": ([_I, _I, _I], _S),
    "md_place_two_level": ([_P, _I, _I, _I, _I, _I, _P, _P, _S, _P, _P], _I),
    "md_successor_share": ([_P, _P, _I, _P, _P, _P], _I),
    "md_count_sums": ([_P, _P, _L, _P, _P], _I),
    "md_table1_row": ([_P, _I, _P], _I),
    "md_pearson_from_sums": ([_P, _L, _P], _I),
    "md_token_shuffle_pair_workspace_size": ([_L, _I, _I], _S),
    "md_token_shuffle_pair": ([_P, _P, _I, _P, _P, _P, _L, _I, _I, ctypes.c_uint32, _P, _P, _P, _P,
                               _P, _S, _P, _P], _I),
    "md_expert_gemm": ([_P, _L, _I, _P, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "md_expert_gated": ([_P, _L, _I, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P], _I),
    "md_expert_wgrad": ([_P, _P, _L, _I, _I, _I, _P, _P, _I, _I, _P, _P, _P], _I),
    "md_set_expert_path": ([_I], _I),
    "md_expert_gated_backward": ([_P, _P, _P, _L, _I, _P, _P, _P], _I),
    "md_combine_backward": ([_P, _P, _L, _P, _P, _L, _I, _I, _P, _P, _P, _P], _I),
    "md_gather_rows": ([_P, _L, _L, _P, _L, _P, _P, _P], _I),
}


class MoeDispatchError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)}")
        self.code = code


def lib():
    """The loaded libmoedispatch.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m combine_warp_top_router_b200.build` (there is no CPU fallback)")
            h = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in _SIGNATURES.items():
                fn = getattr(h, name)
                fn.argtypes = args
                fn.restype = res
            _lib = h
    return _lib


def status_string(code: int) -> str:
    return lib().md_status_string(int(code)).decode()


def launch_count() -> int:
    """Kernels the library has launched in this process."""
    return int(lib().md_launch_count())


def memset_count() -> int:
    """Device memsets and device-to-device copies the library has enqueued."""
    return int(lib().md_memset_count())


def _check(rc: int, what: str):
    if rc != MD_OK:
        raise MoeDispatchError(rc, what)


def _call(name: str, dev, *args) -> int:
    """Call entry point `name` with `dev` as the current CUDA device.

    The CUDA runtime launches on the calling thread's current device, and the
    library looks up per-device state (kernel attributes, the allocation-free
    scratch array) for that device, so tensors on another device are handled
    by making their device current for the call."""
    fn = getattr(lib(), name)
    if type(dev) is not torch.device:
        dev = torch.device(dev)
    if dev.index is None or torch.cuda.current_device() == dev.index:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


# the current stream's handle without the Stream object around it (2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on_its_stream(fn):
    """With `stream=` given the call runs as in `torch.cuda.stream(stream)`: what it allocates, outputs
    and scratch, then belongs to that stream.  Memory of the current stream may be freed there while
    kernels still use it, and the call on the other stream would write into it."""
    last = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None and len(args) == last + 1:  # given by position
            args, stream = args[:last], args[last]
        if stream is None:
            return fn(*args, **kw)
        if _raw_stream is not None and _raw_stream(stream.device_index) == stream.cuda_stream:
            return fn(*args, stream=stream, **kw)  # already the current one
        with torch.cuda.stream(stream):
            return fn(*args, stream=stream, **kw)
    return call


def _need(t, name, dtype, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _room(t, name, n):
    """The kernels write by computed offsets: a buffer must hold n elements."""
    if t is not None and t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {n}")
    return t


def new_status(device) -> torch.Tensor:
    """A device status word for the dev_status arguments."""
    return torch.zeros(1, dtype=torch.int32, device=device)


def check_status(dev_status: torch.Tensor, what: str = "device status"):
    """Synchronise on the status word and raise if a kernel reported an error."""
    code = int(dev_status.item())
    if code != MD_OK:
        raise MoeDispatchError(code, what)


# ------------------------------------------------------------------ router

@_on_its_stream
def md_route_topk(logits, k, gate_mode=MD_GATE_TOPK_SOFTMAX, topk_idx=None, topk_w=None,
                  stream=None):
    _need(logits, "logits", torch.float32)
    T, E = logits.shape
    dev = logits.device
    if topk_idx is None:
        topk_idx = torch.empty(T, k, dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty(T, k, dtype=torch.float32, device=dev)
    _need(topk_idx, "topk_idx", torch.int32, dev)
    _need(topk_w, "topk_w", torch.float32, dev)
    _room(topk_idx, "topk_idx", T * k)
    _room(topk_w, "topk_w", T * k)
    rc = _call("md_route_topk", dev, _ptr(logits), T, E, k, gate_mode, _ptr(topk_idx), _ptr(topk_w),
                             _stream(stream, dev))
    _check(rc, "md_route_topk")
    return topk_idx, topk_w


# ------------------------------------------------------------------ layout

@dataclass
class Layout:
    """Outputs of md_dispatch_layout (device tensors)."""
    mode: int
    row_of_slot: torch.Tensor   # int32 [T, k]
    assign_row: torch.Tensor    # int32 [T, k]
    row_token: torch.Tensor     # int32 [row capacity]
    row_mask: torch.Tensor      # int32 [row capacity] (uint32 bit patterns)
    send_counts: torch.Tensor   # int32 [R, R]
    expert_counts: torch.Tensor  # int32 [E]
    expert_offsets: torch.Tensor  # int32 [E+1]
    rank_offsets: torch.Tensor  # int32 [R+1]
    n_rows: torch.Tensor        # int32 [1]
    row_capacity: int


def _check_layout(L, T, E, k, R, mode, dev):
    """A caller's Layout must have the buffers md_dispatch_layout writes."""
    cap = T * k if mode == MD_CONV else T * min(k, R)
    for name, n in (("row_of_slot", T * k), ("assign_row", T * k), ("row_token", cap),
                    ("row_mask", cap), ("send_counts", R * R), ("expert_counts", E),
                    ("expert_offsets", E + 1), ("rank_offsets", R + 1), ("n_rows", 1)):
        t = getattr(L, name)
        _need(t, name, torch.int32, dev)
        _room(t, name, n)


def dispatch_layout_workspace_size(T, E, k, R, mode) -> int:
    return int(lib().md_dispatch_layout_workspace_size(T, E, k, R, mode))


def alloc_layout(T, E, k, R, mode, device) -> Layout:
    cap = T * k if mode == MD_CONV else T * min(k, R)
    i32 = dict(dtype=torch.int32, device=device)
    return Layout(mode=mode, row_of_slot=torch.empty(T, k, **i32),
                  assign_row=torch.empty(T, k, **i32), row_token=torch.empty(max(cap, 1), **i32),
                  row_mask=torch.empty(max(cap, 1), **i32), send_counts=torch.empty(R, R, **i32),
                  expert_counts=torch.empty(E, **i32), expert_offsets=torch.empty(E + 1, **i32),
                  rank_offsets=torch.empty(R + 1, **i32), n_rows=torch.empty(1, **i32),
                  row_capacity=cap)


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


@_on_its_stream
def md_dispatch_layout(topk_idx, E, R, expert_to_rank, mode, out: Layout | None = None,
                       workspace=None, dev_status=None, stream=None) -> Layout:
    _need(topk_idx, "topk_idx", torch.int32)
    dev = topk_idx.device
    _need(expert_to_rank, "expert_to_rank", torch.int32, dev)
    T, k = topk_idx.shape
    if out is None:
        out = alloc_layout(T, E, k, R, mode, dev)
    _check_layout(out, T, E, k, R, mode, dev)
    need = dispatch_layout_workspace_size(T, E, k, R, mode)
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    _need(workspace, "workspace", torch.uint8, dev)
    rc = _call("md_dispatch_layout", dev, 
        _ptr(topk_idx), T, E, k, R, _ptr(expert_to_rank), mode, _ptr(out.row_of_slot),
        _ptr(out.assign_row), _ptr(out.row_token), _ptr(out.row_mask), _ptr(out.send_counts),
        _ptr(out.expert_counts), _ptr(out.expert_offsets), _ptr(out.rank_offsets),
        _ptr(out.n_rows), _ptr(workspace), workspace.numel(), _ptr(dev_status),
        _stream(stream, dev))
    _check(rc, "md_dispatch_layout")
    return out


@_on_its_stream
def md_dispatch_layout_noalloc(topk_idx, E, R, expert_to_rank, mode, out: Layout | None = None,
                               dev_status=None, stream=None) -> Layout:
    """md_dispatch_layout without a workspace, for callers that cannot allocate
    device memory: the library uses its own fixed 4 MiB per-GPU scratch array.
    Calls that overlap on one GPU share that array and must be serialised."""
    _need(topk_idx, "topk_idx", torch.int32)
    dev = topk_idx.device
    _need(expert_to_rank, "expert_to_rank", torch.int32, dev)
    T, k = topk_idx.shape
    if out is None:
        out = alloc_layout(T, E, k, R, mode, dev)
    _check_layout(out, T, E, k, R, mode, dev)
    rc = _call("md_dispatch_layout_noalloc", dev, 
        _ptr(topk_idx), T, E, k, R, _ptr(expert_to_rank), mode, _ptr(out.row_of_slot),
        _ptr(out.assign_row), _ptr(out.row_token), _ptr(out.row_mask), _ptr(out.send_counts),
        _ptr(out.expert_counts), _ptr(out.expert_offsets), _ptr(out.rank_offsets),
        _ptr(out.n_rows), _ptr(dev_status), _stream(stream, dev))
    _check(rc, "md_dispatch_layout_noalloc")
    return out


# --------------------------------------------------------- permute/combine

@_on_its_stream
def md_dispatch_permute(x, row_of_slot, out_rows=None, out=None, dev_status=None, stream=None):
    _need(x, "x", torch.bfloat16)
    dev = x.device
    _need(row_of_slot, "row_of_slot", torch.int32, dev)
    T, H = x.shape
    k = row_of_slot.shape[1]
    if out is None:
        out = torch.empty(out_rows if out_rows is not None else T * k, H, dtype=torch.bfloat16,
                          device=dev)
    _need(out, "out", torch.bfloat16, dev)
    if out.dim() != 2 or out.shape[1] != H:
        raise ValueError(f"out must be [rows, {H}]")
    rc = _call("md_dispatch_permute", dev, _ptr(x), T, H, k, _ptr(row_of_slot), out.shape[0], _ptr(out),
                                   _ptr(dev_status), _stream(stream, dev))
    _check(rc, "md_dispatch_permute")
    return out


def md_set_permute_path(path=MD_PERMUTE_AUTO):
    """Choose md_dispatch_permute's kernel (tests and tuning; same bits either way)."""
    _check(lib().md_set_permute_path(int(path)), "md_set_permute_path")


def md_set_layout_path(path=MD_LAYOUT_AUTO):
    """Choose md_dispatch_layout's launch form (tests; same results either way)."""
    _check(lib().md_set_layout_path(int(path)), "md_set_layout_path")


@_on_its_stream
def md_dedup_expand(wire, row_of_slot, assign_row, out_rows=None, out=None, dev_status=None,
                    stream=None):
    """out[assign_row[t, j]] = wire[row_of_slot[t, j]]: dedup rows to expert-grouped rows."""
    _need(wire, "wire", torch.bfloat16)
    dev = wire.device
    _need(row_of_slot, "row_of_slot", torch.int32, dev)
    _need(assign_row, "assign_row", torch.int32, dev)
    T, k = row_of_slot.shape
    H = wire.shape[1]
    if assign_row.shape != row_of_slot.shape:
        raise ValueError("assign_row and row_of_slot differ in shape")
    if out is None:
        out = torch.empty(out_rows if out_rows is not None else T * k, H, dtype=torch.bfloat16,
                          device=dev)
    _need(out, "out", torch.bfloat16, dev)
    if out.dim() != 2 or out.shape[1] != H:
        raise ValueError(f"out must be [rows, {H}]")
    rc = _call("md_dedup_expand", dev, _ptr(wire), wire.shape[0], H, _ptr(row_of_slot), _ptr(assign_row), T,
                               k, out.shape[0], _ptr(out), _ptr(dev_status), _stream(stream, dev))
    _check(rc, "md_dedup_expand")
    return out


@_on_its_stream
def md_combine(y, assign_row, topk_idx, topk_w, mode=MD_COMBINE_FUSED, row_of_slot=None, z=None,
               out=None, dev_status=None, stream=None):
    _need(y, "y", torch.bfloat16)
    dev = y.device
    _need(assign_row, "assign_row", torch.int32, dev)
    _need(topk_idx, "topk_idx", torch.int32, dev)
    _need(topk_w, "topk_w", torch.float32, dev)
    T, k = topk_idx.shape
    H = y.shape[1]
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, dev)
    _room(out, "out", T * H)
    _room(assign_row, "assign_row", T * k)
    _room(topk_w, "topk_w", T * k)
    z_rows = 0
    if mode == MD_COMBINE_WIRE:
        _need(row_of_slot, "row_of_slot", torch.int32, dev)
        _need(z, "z", torch.bfloat16, dev)
        _room(row_of_slot, "row_of_slot", T * k)
        z_rows = z.shape[0]
    rc = _call("md_combine", dev, _ptr(y), y.shape[0], _ptr(assign_row), _ptr(topk_idx), _ptr(topk_w), T,
                          k, H, mode, _ptr(row_of_slot), z_rows, _ptr(z), _ptr(out),
                          _ptr(dev_status), _stream(stream, dev))
    _check(rc, "md_combine")
    return out


@_on_its_stream
def md_gather_rows(src, index, out=None, dev_status=None, stream=None):
    if not src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous CUDA tensor")
    dev = src.device
    _need(index, "index", torch.int32, dev)
    n = index.shape[0]
    if out is None:
        out = torch.empty((n,) + tuple(src.shape[1:]), dtype=src.dtype, device=dev)
    if out.dtype != src.dtype or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous CUDA tensor of src's dtype")
    _room(out, "out", n * (src[0].numel() if src.shape[0] else out[0].numel()))
    row_bytes = src[0].numel() * src.element_size() if src.shape[0] else \
        out[0].numel() * out.element_size()
    rc = _call("md_gather_rows", dev, _ptr(src), src.shape[0], row_bytes, _ptr(index), n, _ptr(out),
                              _ptr(dev_status), _stream(stream, dev))
    _check(rc, "md_gather_rows")
    return out


# --------------------------------------------------- statistics / planning

@_on_its_stream
def md_coselect_stats(idx_l, idx_next, E, T_fit=None, W=None, C=None, accumulate=False,
                      want_W=True, want_C=True, dev_status=None, stream=None):
    _need(idx_l, "idx_l", torch.int32)
    dev = idx_l.device
    T, k = idx_l.shape
    T_fit = T if T_fit is None else T_fit
    if idx_next is not None:
        _need(idx_next, "idx_next", torch.int32, dev)
    if W is None and want_W:
        W = torch.empty(E, E, dtype=torch.int32, device=dev)
    if C is None and want_C and idx_next is not None:
        C = torch.empty(E, E, dtype=torch.int32, device=dev)
    if C is not None and idx_next is None:
        raise ValueError("C needs idx_next (the layer-l+1 top-k)")
    if idx_next is not None and idx_next.shape[1] != k:
        raise ValueError("idx_l and idx_next differ in k")
    if idx_next is not None and idx_next.shape[0] < T_fit:
        raise ValueError("idx_next has fewer than T_fit rows")
    if T_fit > T:
        raise ValueError("T_fit exceeds the rows of idx_l")
    for t, n in ((W, "W"), (C, "C")):
        if t is not None:
            _need(t, n, torch.int32, dev)
            _room(t, n, E * E)
    rc = _call("md_coselect_stats", dev, _ptr(idx_l), _ptr(idx_next), T_fit, E, k, _ptr(W), _ptr(C),
                                 1 if accumulate else 0, _ptr(dev_status), _stream(stream, dev))
    _check(rc, "md_coselect_stats")
    return W, C


@_on_its_stream
def md_place_correlated(W, R, seed_mode=MD_SEED_CONTIGUOUS, refine=True, out=None,
                        workspace=None, dev_status=None, stream=None):
    _need(W, "W", torch.int32)
    dev = W.device
    E = W.shape[0]
    if W.dim() != 2 or W.shape[1] != E:
        raise ValueError("W must be [E, E]")
    if out is None:
        out = torch.empty(E, dtype=torch.int32, device=dev)
    _need(out, "out", torch.int32, dev)
    _room(out, "out", E)
    need = int(lib().md_place_correlated_workspace_size(E, R))
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    rc = _call("md_place_correlated", dev, _ptr(W), E, R, seed_mode, 1 if refine else 0, _ptr(out),
                                   _ptr(workspace), workspace.numel(), _ptr(dev_status),
                                   _stream(stream, dev))
    _check(rc, "md_place_correlated")
    return out


@_on_its_stream
def md_place_two_level(W, R, nodes=1, seed_mode=MD_SEED_CONTIGUOUS, refine_mode=MD_REFINE_SWAPS,
                       out=None, workspace=None, dev_status=None, stream=None):
    """Placement over `nodes` nodes of R/nodes ranks (nodes=1: one level), with no
    refinement, best single swaps, or Kernighan-Lin passes."""
    _need(W, "W", torch.int32)
    dev = W.device
    E = W.shape[0]
    if W.dim() != 2 or W.shape[1] != E:
        raise ValueError("W must be [E, E]")
    if out is None:
        out = torch.empty(E, dtype=torch.int32, device=dev)
    _need(out, "out", torch.int32, dev)
    _room(out, "out", E)
    need = int(lib().md_place_two_level_workspace_size(E, R, nodes))
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    rc = _call("md_place_two_level", dev, _ptr(W), E, R, nodes, seed_mode, refine_mode, _ptr(out),
                                  _ptr(workspace), workspace.numel(), _ptr(dev_status),
                                  _stream(stream, dev))
    _check(rc, "md_place_two_level")
    return out


def _shuffle_checks(C, E, p_next, T, dev, **outs):
    if C.dim() != 2 or C.shape[1] != E:
        raise ValueError("C must be [E, E]")
    _room(p_next, "expert_to_rank_next", E)
    for name, t in outs.items():
        _need(t, name, torch.int32, dev)
        _room(t, name, T)


@_on_its_stream
def md_token_shuffle(idx_l, C, expert_to_rank_next, R, pred_rank=None, perm=None, inv=None,
                     workspace=None, dev_status=None, stream=None):
    _need(idx_l, "idx_l", torch.int32)
    dev = idx_l.device
    _need(C, "C", torch.int32, dev)
    _need(expert_to_rank_next, "expert_to_rank_next", torch.int32, dev)
    T, k = idx_l.shape
    E = C.shape[0]
    i32 = dict(dtype=torch.int32, device=dev)
    pred_rank = torch.empty(T, **i32) if pred_rank is None else pred_rank
    perm = torch.empty(T, **i32) if perm is None else perm
    inv = torch.empty(T, **i32) if inv is None else inv
    _shuffle_checks(C, E, expert_to_rank_next, T, dev, pred_rank=pred_rank, perm=perm, inv=inv)
    need = int(lib().md_token_shuffle_workspace_size(T, E, R))
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    rc = _call("md_token_shuffle", dev, _ptr(idx_l), k, _ptr(C), _ptr(expert_to_rank_next), T, E, R,
                                _ptr(pred_rank), _ptr(perm), _ptr(inv), _ptr(workspace),
                                workspace.numel(), _ptr(dev_status), _stream(stream, dev))
    _check(rc, "md_token_shuffle")
    return pred_rank, perm, inv


@_on_its_stream
def md_token_shuffle_rounds(idx_l, C, expert_to_rank_next, R, pred_rank=None, perm=None,
                            inv=None, workspace=None, dev_status=None, stream=None):
    """Rounds-based capacity assignment -> (pred, perm, inv, rounds [1] device tensor)."""
    _need(idx_l, "idx_l", torch.int32)
    dev = idx_l.device
    _need(C, "C", torch.int32, dev)
    _need(expert_to_rank_next, "expert_to_rank_next", torch.int32, dev)
    T, k = idx_l.shape
    E = C.shape[0]
    i32 = dict(dtype=torch.int32, device=dev)
    pred_rank = torch.empty(T, **i32) if pred_rank is None else pred_rank
    perm = torch.empty(T, **i32) if perm is None else perm
    inv = torch.empty(T, **i32) if inv is None else inv
    _shuffle_checks(C, E, expert_to_rank_next, T, dev, pred_rank=pred_rank, perm=perm, inv=inv)
    rounds = torch.zeros(1, **i32)
    need = int(lib().md_token_shuffle_rounds_workspace_size(T, E, R))
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    rc = _call("md_token_shuffle_rounds", dev, _ptr(idx_l), k, _ptr(C), _ptr(expert_to_rank_next), T, E, R,
                                       _ptr(pred_rank), _ptr(perm), _ptr(inv), _ptr(rounds),
                                       _ptr(workspace), workspace.numel(), _ptr(dev_status),
                                       _stream(stream, dev))
    _check(rc, "md_token_shuffle_rounds")
    return pred_rank, perm, inv, rounds


@_on_its_stream
def md_coselect_pair_stats(idx_prev, idx_l, idx_next, E, T_fit=None, C2=None, accumulate=False,
                           dev_status=None, stream=None):
    """Pair counts C2[a, b, e'] (int32 view of uint32 [E, E, E])."""
    _need(idx_l, "idx_l", torch.int32)
    dev = idx_l.device
    _need(idx_prev, "idx_prev", torch.int32, dev)
    _need(idx_next, "idx_next", torch.int32, dev)
    T, k = idx_l.shape
    T_fit = T if T_fit is None else T_fit
    if C2 is None:
        C2 = torch.empty(E, E, E, dtype=torch.int32, device=dev)
    _need(C2, "C2", torch.int32, dev)
    _room(C2, "C2", E * E * E)
    if idx_prev.shape[1] != k or idx_next.shape[1] != k:
        raise ValueError("idx_prev, idx_l and idx_next differ in k")
    if min(idx_prev.shape[0], idx_next.shape[0], T) < T_fit:
        raise ValueError("fewer than T_fit rows")
    rc = _call("md_coselect_pair_stats", dev, _ptr(idx_prev), _ptr(idx_l), _ptr(idx_next), T_fit, E, k,
                                      _ptr(C2), 1 if accumulate else 0, _ptr(dev_status),
                                      _stream(stream, dev))
    _check(rc, "md_coselect_pair_stats")
    return C2


@_on_its_stream
def md_token_shuffle_pair(idx_prev, idx_l, C, C2, expert_to_rank_next, R, min_obs, pred_rank=None,
                          perm=None, inv=None, use_pair=None, workspace=None, dev_status=None,
                          stream=None):
    """Pair-based shuffle prediction with single-expert fallback -> (pred, perm, inv, use_pair)."""
    _need(idx_l, "idx_l", torch.int32)
    dev = idx_l.device
    _need(idx_prev, "idx_prev", torch.int32, dev)
    _need(C, "C", torch.int32, dev)
    _need(C2, "C2", torch.int32, dev)
    _need(expert_to_rank_next, "expert_to_rank_next", torch.int32, dev)
    T, k = idx_l.shape
    E = C.shape[0]
    i32 = dict(dtype=torch.int32, device=dev)
    pred_rank = torch.empty(T, **i32) if pred_rank is None else pred_rank
    perm = torch.empty(T, **i32) if perm is None else perm
    inv = torch.empty(T, **i32) if inv is None else inv
    use_pair = torch.empty(T, **i32) if use_pair is None else use_pair
    _shuffle_checks(C, E, expert_to_rank_next, T, dev, pred_rank=pred_rank, perm=perm, inv=inv,
                    use_pair=use_pair)
    if idx_prev.shape != idx_l.shape:
        raise ValueError("idx_prev and idx_l differ in shape")
    _room(C2, "C2", E * E * E)
    need = int(lib().md_token_shuffle_pair_workspace_size(T, E, R))
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    rc = _call("md_token_shuffle_pair", dev, _ptr(idx_prev), _ptr(idx_l), k, _ptr(C), _ptr(C2),
                                     _ptr(expert_to_rank_next), T, E, R, int(min_obs),
                                     _ptr(pred_rank), _ptr(perm), _ptr(inv), _ptr(use_pair),
                                     _ptr(workspace), workspace.numel(), _ptr(dev_status),
                                     _stream(stream, dev))
    _check(rc, "md_token_shuffle_pair")
    return pred_rank, perm, inv, use_pair


# ------------------------------------------------------- experts

# A call for a few rows takes about as long on the host as on the GPU, so the checks
# below look at everything at once and ask what is wrong only if something is.

def _first(t, name, dtype, dims):
    """A call's first tensor: it names the device."""
    _need(t, name, dtype)
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    return t.device


def _exact(t, name, dtype, dev, shape):
    """A contiguous tensor of this type, device and shape."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.shape == shape
            and t.is_contiguous()):
        _need(t, name, dtype, dev)
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _words(t, name, dev, n):
    """A contiguous int32 tensor of n elements or more."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.device == dev
            and t.numel() >= n and t.is_contiguous()):
        _need(t, name, torch.int32, dev)
        _room(t, name, n)


def _tail(dev_status, stream, dev):
    """The addresses of the last two arguments of every entry point."""
    if dev_status is not None:
        _words(dev_status, "dev_status", dev, 1)
        dev_status = dev_status.data_ptr()
    if stream is not None:
        return dev_status, stream.cuda_stream
    if _raw_stream is not None:
        return dev_status, _raw_stream(dev.index)
    return dev_status, torch.cuda.current_stream(dev).cuda_stream


def md_set_expert_path(path=MD_EXPERT_AUTO):
    """Choose the kernel form of the expert products (tests and tuning)."""
    _check(_call("md_set_expert_path", "cpu", int(path)), "md_set_expert_path")


@_on_its_stream
def md_expert_gemm(x, w, expert_offsets, expert_counts, w_layout=MD_W_NK, out=None,
                   dev_status=None, stream=None):
    """y[r] = x[r] times the matrix of row r's expert (MD_W_NK: w [E, N, K], MD_W_KN: w [E, K, N]).

    Rows are expert-grouped: expert_offsets and expert_counts come from md_dispatch_layout.
    Rows of no expert are left untouched in `out`."""
    dev = _first(x, "x", torch.bfloat16, 2)
    if w_layout != MD_W_NK and w_layout != MD_W_KN:
        raise ValueError("w_layout must be MD_W_NK or MD_W_KN")
    _need(w, "w", torch.bfloat16, dev)
    rows, K = x.shape
    if w.dim() != 3 or w.shape[2 if w_layout == MD_W_NK else 1] != K:
        raise ValueError(f"w has shape {tuple(w.shape)}, expected three dimensions and K = {K}")
    E, N = w.shape[0], w.shape[1 if w_layout == MD_W_NK else 2]
    _words(expert_offsets, "expert_offsets", dev, E)
    _words(expert_counts, "expert_counts", dev, E)
    if out is None:
        out = x.new_empty((rows, N))
    else:
        _exact(out, "out", torch.bfloat16, dev, (rows, N))
    status, stream = _tail(dev_status, stream, dev)
    rc = _call("md_expert_gemm", dev, x.data_ptr(), rows, K, w.data_ptr(), E, N, w_layout,
               expert_offsets.data_ptr(), expert_counts.data_ptr(), out.data_ptr(), status, stream)
    _check(rc, "md_expert_gemm")
    return out


@_on_its_stream
def md_expert_gated(x, w, expert_offsets, expert_counts, keep=False, out=None, codes=None,
                    scales=None, dev_status=None, stream=None):
    """Gated up-projection act = silu(g) * u with g, u = x w[e]^T; w [E, 2F, K] holds g's rows, then u's.

    keep=True (or codes or scales given) also writes the 8-bit checkpoint of g and u that
    md_expert_gated_backward reads, and returns (act, codes, scales)."""
    dev = _first(x, "x", torch.bfloat16, 2)
    _need(w, "w", torch.bfloat16, dev)
    rows, K = x.shape
    if w.dim() != 3 or w.shape[2] != K or w.shape[1] % 2:
        raise ValueError(f"w has shape {tuple(w.shape)}, expected [E, 2F, {K}]")
    E, N = w.shape[0], w.shape[1]
    F = N // 2
    _words(expert_offsets, "expert_offsets", dev, E)
    _words(expert_counts, "expert_counts", dev, E)
    if out is None:
        out = x.new_empty((rows, F))
    else:
        _exact(out, "out", torch.bfloat16, dev, (rows, F))
    keep = keep or codes is not None or scales is not None
    if keep:
        blocks = 2 * -(-F // MD_CHECKPOINT_BLOCK)
        if codes is None:
            codes = torch.empty((rows, N), dtype=torch.float8_e4m3fn, device=dev)
        else:
            _exact(codes, "codes", torch.float8_e4m3fn, dev, (rows, N))
        if scales is None:
            scales = torch.empty((rows, blocks), dtype=torch.uint8, device=dev)
        else:
            _exact(scales, "scales", torch.uint8, dev, (rows, blocks))
    status, stream = _tail(dev_status, stream, dev)
    rc = _call("md_expert_gated", dev, x.data_ptr(), rows, K, w.data_ptr(), E, F,
               expert_offsets.data_ptr(), expert_counts.data_ptr(), out.data_ptr(),
               codes.data_ptr() if keep else None, scales.data_ptr() if keep else None, status, stream)
    _check(rc, "md_expert_gated")
    return (out, codes, scales) if keep else out


@_on_its_stream
def md_expert_wgrad(dy, x, expert_offsets, expert_counts, out_dtype=torch.float32, dw=None,
                    accumulate=False, dev_status=None, stream=None):
    """dw[e] = sum over expert e's rows of dy[r]^T x[r], [E, N, K]; accumulate adds into a float32 dw.

    E is the length of expert_counts (or dw's first extent)."""
    dev = _first(dy, "dy", torch.bfloat16, 2)
    _need(x, "x", torch.bfloat16, dev)
    rows, N = dy.shape
    if x.dim() != 2 or x.shape[0] != rows:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [{rows}, K]")
    K = x.shape[1]
    if dw is not None:
        out_dtype = dw.dtype
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dw must be float32 or bfloat16")
    if accumulate and (dw is None or out_dtype != torch.float32):
        raise ValueError("accumulate needs a float32 dw to add to")
    E = expert_counts.numel() if dw is None else dw.shape[0]
    _words(expert_offsets, "expert_offsets", dev, E)
    _words(expert_counts, "expert_counts", dev, E)
    if dw is None:
        dw = torch.empty((E, N, K), dtype=out_dtype, device=dev)
    else:
        _exact(dw, "dw", out_dtype, dev, (E, N, K))
    status, stream = _tail(dev_status, stream, dev)
    rc = _call("md_expert_wgrad", dev, dy.data_ptr(), x.data_ptr(), rows, E, N, K,
               expert_offsets.data_ptr(), expert_counts.data_ptr(),
               MD_F32 if out_dtype == torch.float32 else MD_BF16, 1 if accumulate else 0,
               dw.data_ptr(), status, stream)
    _check(rc, "md_expert_wgrad")
    return dw


@_on_its_stream
def md_expert_gated_backward(da, codes, scales, dh=None, act=None, want_act=True, stream=None):
    """(dh, act) from the gradient of the activation and the checkpoint of md_expert_gated.

    dh [rows, 2F] is the gradient of g, then of u; act is the activation computed again from
    the checkpoint (None with want_act=False)."""
    dev = _first(da, "da", torch.bfloat16, 2)
    rows, F = da.shape
    _exact(codes, "codes", torch.float8_e4m3fn, dev, (rows, 2 * F))
    _exact(scales, "scales", torch.uint8, dev, (rows, 2 * -(-F // MD_CHECKPOINT_BLOCK)))
    if dh is None:
        dh = da.new_empty((rows, 2 * F))
    else:
        _exact(dh, "dh", torch.bfloat16, dev, (rows, 2 * F))
    if act is not None:
        _exact(act, "act", torch.bfloat16, dev, (rows, F))
    elif want_act:
        act = torch.empty_like(da)
    _, stream = _tail(None, stream, dev)
    rc = _call("md_expert_gated_backward", dev, da.data_ptr(), codes.data_ptr(), scales.data_ptr(), rows,
               F, dh.data_ptr(), None if act is None else act.data_ptr(), stream)
    _check(rc, "md_expert_gated_backward")
    return dh, act


@_on_its_stream
def md_combine_backward(dout, assign_row, topk_w, y=None, y_rows=None, dy=None, dw=None,
                        dev_status=None, stream=None):
    """Gradient of md_combine: (dy, dw), dy[assign_row[t, j]] = topk_w[t, j] dout[t].

    dw [T, k] is the gates' gradient; it needs the expert outputs y (without y it is None).
    dy has y_rows rows: y's, or without y dy's or T * k by default."""
    dev = _first(dout, "dout", torch.bfloat16, 2)
    T, H = dout.shape
    _need(topk_w, "topk_w", torch.float32, dev)
    if topk_w.dim() != 2 or topk_w.shape[0] != T:
        raise ValueError(f"topk_w has shape {tuple(topk_w.shape)}, expected [{T}, k]")
    k = topk_w.shape[1]
    _exact(assign_row, "assign_row", torch.int32, dev, (T, k))
    if y is not None:
        if y_rows is None and isinstance(y, torch.Tensor) and y.dim() == 2:
            y_rows = y.shape[0]
        _exact(y, "y", torch.bfloat16, dev, (y_rows, H))
        if dw is None:
            dw = torch.empty_like(topk_w)
        else:
            _exact(dw, "dw", torch.float32, dev, (T, k))
    elif dw is not None:
        raise ValueError("dw needs y (the expert outputs)")
    if dy is None and y is not None:
        dy = torch.empty_like(y)
    elif dy is None:
        dy = dout.new_empty((T * k if y_rows is None else y_rows, H))
    else:
        _exact(dy, "dy", torch.bfloat16, dev, (dy.shape[0] if y_rows is None else y_rows, H))
    status, stream = _tail(dev_status, stream, dev)
    rc = _call("md_combine_backward", dev, dout.data_ptr(), None if y is None else y.data_ptr(),
               dy.shape[0], assign_row.data_ptr(), topk_w.data_ptr(), T, k, H, dy.data_ptr(),
               None if dw is None else dw.data_ptr(), status, stream)
    _check(rc, "md_combine_backward")
    return dy, dw


# ------------------------------------------------------- EP exchange

class md_peer_rows(ctypes.Structure):
    """One rank's exchange buffers as this rank addresses them (include/moedispatch.h)."""
    _fields_ = [("rows", ctypes.c_void_p), ("token", ctypes.c_void_p),
                ("slot_idx", ctypes.c_void_p), ("slot_w", ctypes.c_void_p),
                ("row_base", ctypes.c_int64), ("rows_cap", ctypes.c_int64)]


@dataclass
class PeerRows:
    """Buffers of one destination rank: tensors on this device, or raw device
    addresses (ints) of another GPU's memory mapped into this process."""
    rows: object
    row_base: int
    rows_cap: int
    token: object = None
    slot_idx: object = None
    slot_w: object = None


def _addr(v):
    if v is None:
        return None
    if isinstance(v, torch.Tensor):
        return v.data_ptr()
    return int(v)


def _peer_table(peers):
    arr = (md_peer_rows * len(peers))()
    for i, q in enumerate(peers):
        arr[i] = md_peer_rows(_addr(q.rows), _addr(q.token), _addr(q.slot_idx), _addr(q.slot_w),
                              int(q.row_base), int(q.rows_cap))
    return arr


def md_exchange_plan(src_rank_offsets, me):
    """(dst_row_base [R], recv_offsets [R+1]) of rank `me` from every source's
    layout rank_offsets, gathered ([R, R+1], row s = source s), on the host."""
    rows = [[int(v) for v in r] for r in src_rank_offsets.tolist()] \
        if hasattr(src_rank_offsets, "tolist") else [[int(v) for v in r] for r in src_rank_offsets]
    R = len(rows)
    if any(len(r) != R + 1 for r in rows):
        raise ValueError("src_rank_offsets must be [R, R+1]")
    flat = (ctypes.c_int64 * (R * (R + 1)))(*[v for r in rows for v in r])
    base = (ctypes.c_int64 * R)()
    recv = (ctypes.c_int64 * (R + 1))()
    _check(lib().md_exchange_plan(ctypes.cast(flat, _P), R, int(me), ctypes.cast(base, _P),
                                  ctypes.cast(recv, _P)), "md_exchange_plan")
    return list(base), list(recv)


@_on_its_stream
def md_dispatch_exchange(x, topk_idx, topk_w, expert_to_rank, E, row_of_slot, rank_offsets,
                         token_base, peers, dev_status=None, stream=None):
    """Write this rank's dispatch rows (and their metadata) into the R
    destination ranks' buffers `peers` (a list of PeerRows)."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    _need(topk_idx, "topk_idx", torch.int32, dev)
    if topk_w is not None:
        _need(topk_w, "topk_w", torch.float32, dev)
    _need(expert_to_rank, "expert_to_rank", torch.int32, dev)
    _need(row_of_slot, "row_of_slot", torch.int32, dev)
    _need(rank_offsets, "rank_offsets", torch.int32, dev)
    T, H = x.shape
    k = topk_idx.shape[1]
    R = len(peers)
    _room(rank_offsets, "rank_offsets", R + 1)
    _room(row_of_slot, "row_of_slot", T * k)
    tab = _peer_table(peers)
    rc = _call("md_dispatch_exchange", dev, _ptr(x), T, H, k, _ptr(topk_idx), _ptr(topk_w),
               _ptr(expert_to_rank), E, R, _ptr(row_of_slot), _ptr(rank_offsets), int(token_base),
               ctypes.cast(tab, _P), _ptr(dev_status), _stream(stream, dev))
    _check(rc, "md_dispatch_exchange")


@_on_its_stream
def md_combine_partials(y, y_row, slot_idx, slot_w, out=None, dev_status=None, stream=None):
    """Return rows of a receiving rank: z[i] = bf16(sum over carried slots, by
    ascending expert, of slot_w * y[y_row])."""
    _need(y, "y", torch.bfloat16)
    dev = y.device
    _need(y_row, "y_row", torch.int32, dev)
    _need(slot_idx, "slot_idx", torch.int32, dev)
    _need(slot_w, "slot_w", torch.float32, dev)
    n, k = y_row.shape
    H = y.shape[1]
    if slot_idx.shape != (n, k) or slot_w.shape != (n, k):
        raise ValueError("y_row, slot_idx and slot_w differ in shape")
    if out is None:
        out = torch.empty(n, H, dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, dev)
    _room(out, "out", n * H)
    rc = _call("md_combine_partials", dev, _ptr(y), y.shape[0], _ptr(y_row), _ptr(slot_idx),
               _ptr(slot_w), n, k, H, _ptr(out), _ptr(dev_status), _stream(stream, dev))
    _check(rc, "md_combine_partials")
    return out


@_on_its_stream
def md_combine_exchange(peers, topk_idx, expert_to_rank, E, row_of_slot, rank_offsets, H,
                        out=None, dev_status=None, stream=None):
    """out[t] = bf16(fp32 sum, by ascending rank, of the return rows of t read
    from the R ranks' buffers `peers`)."""
    _need(topk_idx, "topk_idx", torch.int32)
    dev = topk_idx.device
    _need(expert_to_rank, "expert_to_rank", torch.int32, dev)
    _need(row_of_slot, "row_of_slot", torch.int32, dev)
    _need(rank_offsets, "rank_offsets", torch.int32, dev)
    T, k = topk_idx.shape
    R = len(peers)
    _room(rank_offsets, "rank_offsets", R + 1)
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, dev)
    _room(out, "out", T * H)
    tab = _peer_table(peers)
    rc = _call("md_combine_exchange", dev, ctypes.cast(tab, _P), T, H, k, _ptr(topk_idx),
               _ptr(expert_to_rank), E, R, _ptr(row_of_slot), _ptr(rank_offsets), _ptr(out),
               _ptr(dev_status), _stream(stream, dev))
    _check(rc, "md_combine_exchange")
    return out


# ------------------------------------------------------------ statistics

@_on_its_stream
def md_rank_stats(topk_idx, E, R, expert_to_rank, hist=None, dev_status=None, stream=None):
    """hist int64 [k+1]: tokens whose experts sit on exactly D distinct ranks."""
    _need(topk_idx, "topk_idx", torch.int32)
    dev = topk_idx.device
    _need(expert_to_rank, "expert_to_rank", torch.int32, dev)
    T, k = topk_idx.shape
    hist = torch.empty(k + 1, dtype=torch.int64, device=dev) if hist is None else hist
    _need(hist, "hist", torch.int64, dev)
    _room(hist, "hist", k + 1)
    _room(expert_to_rank, "expert_to_rank", E)
    rc = _call("md_rank_stats", dev, _ptr(topk_idx), T, E, k, R, _ptr(expert_to_rank), _ptr(hist),
                             _ptr(dev_status), _stream(stream, dev))
    _check(rc, "md_rank_stats")
    return hist


def table1_row(hist):
    """Table I columns from a rank histogram: (same-rank %, ranks per token, dedup %)
    (md_table1_row on the host)."""
    h = (ctypes.c_int64 * len(hist))(*[int(v) for v in hist.tolist()])
    out = (ctypes.c_double * 3)()
    _check(lib().md_table1_row(ctypes.cast(h, _P), len(hist) - 1, ctypes.cast(out, _P)),
           "md_table1_row")
    return out[0], out[1], out[2]


@_on_its_stream
def md_successor_share(C, W, stream=None):
    """(num, den) int32 views of uint32 [E]: max_e' C[e, e'] and W[e, e]."""
    _need(C, "C", torch.int32)
    dev = C.device
    _need(W, "W", torch.int32, dev)
    E = C.shape[0]
    if C.shape != (E, E) or W.shape != (E, E):
        raise ValueError("C and W must be [E, E]")
    num = torch.empty(E, dtype=torch.int32, device=dev)
    den = torch.empty(E, dtype=torch.int32, device=dev)
    rc = _call("md_successor_share", dev, _ptr(C), _ptr(W), E, _ptr(num), _ptr(den), _stream(stream, dev))
    _check(rc, "md_successor_share")
    return num, den


@_on_its_stream
def md_count_sums(x, y, stream=None):
    """Exact (sx, sy, sxx, syy, sxy) of two count tables (int32 views of uint32)."""
    _need(x, "x", torch.int32)
    dev = x.device
    _need(y, "y", torch.int32, dev)
    if x.numel() != y.numel():
        raise MoeDispatchError("md_count_sums: tables differ in size")
    out = torch.empty(10, dtype=torch.int64, device=dev)
    rc = _call("md_count_sums", dev, _ptr(x), _ptr(y), x.numel(), _ptr(out), _stream(stream, dev))
    _check(rc, "md_count_sums")
    w = [v & (2 ** 64 - 1) for v in out.cpu().tolist()]
    return tuple(w[2 * i] | (w[2 * i + 1] << 64) for i in range(5))


def pearson_from_sums(n, sums):
    """Pearson correlation from the exact sums of md_count_sums (md_pearson_from_sums
    on the host); NaN when a table has zero variance."""
    words = []
    for v in sums:
        v = int(v)
        words += [v & (2 ** 64 - 1), (v >> 64) & (2 ** 64 - 1)]
    c = (ctypes.c_uint64 * 10)(*words)
    r = ctypes.c_double()
    rc = lib().md_pearson_from_sums(ctypes.cast(c, _P), int(n), ctypes.byref(r))
    if rc == MD_ERR_DATA:
        return float("nan")
    _check(rc, "md_pearson_from_sums")
    return r.value


def md_set_test_hooks(poll_limit=0, layout_skip_tile=-1, expand_skip_unit=-1):
    """Fault injection for tests: make a bounded device-side wait run out."""
    lib().md_set_test_hooks(int(poll_limit), int(layout_skip_tile), int(expand_skip_unit))
