"""Python binding of libmoe_route_sort.so: argument marshalling only.

Every step of the route-sort path (FP32 conversion, bias, grouped top-k,
histogram, prefix, scatter) runs in the HIP kernels behind the C ABI declared
in include/moe_route_sort.h.  This module checks tensors, allocates outputs
when the caller gives none, and forwards raw device pointers and the current
HIP stream.  It fails loudly when the library is not built; there is no
fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import NamedTuple, Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_route_sort.so")

MRS_OK = 0
MRS_ERR_INVALID_ARG = -1
MRS_ERR_NULL_POINTER = -2
MRS_ERR_MISALIGNED = -3
MRS_ERR_WORKSPACE = -4
MRS_ERR_OVERFLOW = -5
MRS_ERR_LAUNCH = -6
MRS_ERR_SCRATCH = -7
MRS_DTYPE_F32 = 0
MRS_DTYPE_BF16 = 1
MRS_DTYPE_F16 = 2
MRS_X_TOKENS = 0
MRS_X_SORTED = 1
MRS_INT4_PLAIN = 0
MRS_INT4_GATED = 1
MRS_INT4_SUM = 2
MRS_TILE_NARROW = 1 << 16
FLAG_FORCE_SINGLE_WG = 1
FLAG_FORCE_MULTI_WG = 2
FLAG_FORCE_EXACT = 4
PRODUCT_BY_RULE, PRODUCT_ROWS_16, PRODUCT_ROWS_32 = 0, 1, 2
PRODUCT_TILE_16, PRODUCT_TILE_32, PRODUCT_TILE_64, PRODUCT_TILE_128 = 3, 4, 5, 6

EXPORTED = [
    "moe_route_sort",
    "moe_route_sort_ex",
    "moe_route_sort_profiled",
    "moe_route_sort_local",
    "moe_route_sort_static",
    "moe_sort_from_ids",
    "moe_sort_from_ids_counters",
    "moe_route_sort_max_rows",
    "moe_route_sort_max_blocks",
    "moe_route_sort_workspace_bytes",
    "moe_route_sort_strerror",
    "moe_route_sort_sigmoid_probe",
    "moe_route_sort_sigmoid_table_probe",
    "moe_grouped_gemm1",
    "moe_grouped_gemm1_profiled",
    "moe_gate_route_sort",
    "moe_mxfp4_quantize",
    "moe_grouped_gemm_mxfp4",
    "moe_grouped_gemm_mxfp4_ex",
    "moe_balance_workspace_bytes",
    "moe_balance_loss",
    "moe_route_far_weights",
    "moe_router_backward",
    "moe_grouped_gemm",
    "moe_grouped_gemm_ex",
    "moe_grouped_gemm_dx",
    "moe_grouped_gemm_dx_ex",
    "moe_grouped_gemm_dw",
    "moe_swiglu",
    "moe_swiglu_backward",
    "moe_slot_rows",
    "moe_combine",
    "moe_combine_backward",
    "moe_int4_quantize",
    "moe_int4_matvec",
]

_lib = None


class RouteSortError(RuntimeError):
    def __init__(self, code: int):
        super().__init__(f"moe_route_sort failed ({code}): {strerror(code)}")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "or python align_moe_route_amd/build.py")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    common = [vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    L.moe_route_sort.argtypes = common
    L.moe_route_sort.restype = i32
    L.moe_route_sort_ex.argtypes = common + [ctypes.c_uint, vp]
    L.moe_route_sort_ex.restype = i32
    L.moe_route_sort_profiled.argtypes = common + [ctypes.c_uint, vp, vp, vp]
    L.moe_route_sort_profiled.restype = i32
    L.moe_route_sort_local.argtypes = common[:8] + [i32, i32] + common[8:]
    L.moe_route_sort_local.restype = i32
    L.moe_route_sort_static.argtypes = common[:14] + [vp]
    L.moe_route_sort_static.restype = i32
    L.moe_sort_from_ids.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.moe_sort_from_ids.restype = i32
    L.moe_sort_from_ids_counters.argtypes = [vp, i32, i32, i32, i32, vp, ctypes.c_int64, vp, vp, vp, vp, sz, vp]
    L.moe_sort_from_ids_counters.restype = i32
    for name in ("moe_route_sort_max_rows", "moe_route_sort_max_blocks"):
        getattr(L, name).argtypes = [i32, i32, i32, i32]
        getattr(L, name).restype = ctypes.c_int64
    L.moe_route_sort_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.moe_route_sort_workspace_bytes.restype = sz
    L.moe_route_sort_strerror.argtypes = [i32]
    L.moe_route_sort_strerror.restype = ctypes.c_char_p
    L.moe_route_sort_sigmoid_probe.argtypes = [vp, i32, vp, vp, vp]
    L.moe_route_sort_sigmoid_probe.restype = i32
    L.moe_route_sort_sigmoid_table_probe.argtypes = [vp, i32, vp, vp, vp]
    L.moe_route_sort_sigmoid_table_probe.restype = i32
    L.moe_grouped_gemm1.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp]
    L.moe_grouped_gemm1.restype = i32
    L.moe_grouped_gemm1_profiled.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp]
    L.moe_grouped_gemm1_profiled.restype = i32
    L.moe_gate_route_sort.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    L.moe_gate_route_sort.restype = i32
    i64, f32 = ctypes.c_int64, ctypes.c_float
    L.moe_mxfp4_quantize.argtypes = [vp, i32, i64, i32, i64, vp, vp, vp, vp]
    L.moe_mxfp4_quantize.restype = i32
    L.moe_grouped_gemm_mxfp4.argtypes = [vp] * 7 + [i32] * 8 + [vp, vp]
    L.moe_grouped_gemm_mxfp4.restype = i32
    L.moe_grouped_gemm_mxfp4_ex.argtypes = L.moe_grouped_gemm_mxfp4.argtypes + [i32]
    L.moe_grouped_gemm_mxfp4_ex.restype = i32
    L.moe_balance_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.moe_balance_workspace_bytes.restype = sz
    L.moe_balance_loss.argtypes = [vp, i32, vp, vp, vp, i32, i32, i32, i32, f32, vp, vp, vp, vp, vp, sz, vp]
    L.moe_balance_loss.restype = i32
    L.moe_route_far_weights.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp]
    L.moe_route_far_weights.restype = i32
    L.moe_router_backward.argtypes = [vp, i32] + [vp] * 7 + [i32] * 4 + [f32, vp, vp]
    L.moe_router_backward.restype = i32
    L.moe_grouped_gemm.argtypes = [vp, vp, i32, vp, vp, vp] + [i32] * 8 + [vp, vp]
    L.moe_grouped_gemm.restype = i32
    L.moe_grouped_gemm_dx.argtypes = [vp, vp, i32, vp, vp, vp] + [i32] * 7 + [vp, vp]
    L.moe_grouped_gemm_dx.restype = i32
    L.moe_grouped_gemm_dw.argtypes = L.moe_grouped_gemm.argtypes
    L.moe_grouped_gemm_ex.argtypes = L.moe_grouped_gemm.argtypes + [i32]
    L.moe_grouped_gemm_ex.restype = i32
    L.moe_grouped_gemm_dx_ex.argtypes = L.moe_grouped_gemm_dx.argtypes + [i32]
    L.moe_grouped_gemm_dx_ex.restype = i32
    L.moe_grouped_gemm_dw.restype = i32
    L.moe_swiglu.argtypes = [vp, i32, vp, i64, i32, vp, vp]
    L.moe_swiglu.restype = i32
    L.moe_swiglu_backward.argtypes = [vp, vp, i32, vp, i64, i32, vp, vp]
    L.moe_swiglu_backward.restype = i32
    L.moe_slot_rows.argtypes = [vp, vp, i64, i32, i32, vp, vp]
    L.moe_slot_rows.restype = i32
    L.moe_combine.argtypes = [vp, i32, vp, vp, i64, i32, i32, i32, i32, vp, vp]
    L.moe_combine.restype = i32
    L.moe_combine_backward.argtypes = [vp, vp, i32, vp, vp, vp, vp, i64, i32, i32, i32, vp, vp, vp]
    L.moe_combine_backward.restype = i32
    L.moe_int4_quantize.argtypes = [vp, i32, i64, i32, i64, i32, i32, vp, vp, vp]
    L.moe_int4_quantize.restype = i32
    L.moe_int4_matvec.argtypes = [vp, i32, vp, vp, vp, vp] + [i32] * 8 + [vp, vp]
    L.moe_int4_matvec.restype = i32
    _lib = L
    return L


def strerror(code: int) -> str:
    return lib().moe_route_sort_strerror(int(code)).decode()


def max_rows(M: int, E: int, k: int, block: int) -> int:
    return int(lib().moe_route_sort_max_rows(M, E, k, block))


def max_blocks(M: int, E: int, k: int, block: int) -> int:
    return int(lib().moe_route_sort_max_blocks(M, E, k, block))


def workspace_bytes(M: int, E: int, k: int, block: int) -> int:
    v = int(lib().moe_route_sort_workspace_bytes(M, E, k, block))
    if v == ctypes.c_size_t(-1).value:
        raise ValueError("invalid sizes")
    return v


def raw_call(logits_ptr, bias_ptr, M, E, k, n_group, topk_group, block, out_ids_ptr, out_w_ptr,
             sorted_ids_ptr, eob_ptr, npp_ptr, dtype, ws_ptr, ws_bytes, stream_ptr,
             flags: int = 0, stats_ptr=None) -> int:
    """Direct C-ABI call with integer device pointers; returns the MRS code."""
    return int(lib().moe_route_sort_ex(logits_ptr, bias_ptr, M, E, k, n_group, topk_group, block,
                                       out_ids_ptr, out_w_ptr, sorted_ids_ptr, eob_ptr, npp_ptr,
                                       dtype, ws_ptr, ws_bytes, stream_ptr, flags, stats_ptr))


class _Route(NamedTuple):
    ids: "torch.Tensor"              # [M, k] int32, ascending expert ids per token
    weights: "torch.Tensor"          # [M, k] float32
    sorted_ids: "torch.Tensor"       # [max_rows] int32; [0, num_post_pad) defined
    expert_of_block: "torch.Tensor"  # [max_blocks] int32; [0, num_post_pad/block) defined
    num_post_pad: "torch.Tensor"     # [1] int32 (device)


class RouteSortOutput(_Route):
    """A call's ids, weights and metadata.  One that a call of this package returned also
    says how many experts the metadata numbers and the block that it was made for, for
    checks by what reads it; made by hand, or of another's parts, it does not know."""
    experts: Optional[int] = None
    block: Optional[int] = None

    def _replace(self, **kwargs):
        same = kwargs.keys() <= {"ids", "weights"}  # the metadata, which is what the two are about
        return _routed(super()._replace(**kwargs), self.experts if same else None, self.block if same else None)


def _overwritten(*tensors):
    """The caller's tensors, which a call is about to write: autograd is told, so that a
    backward pass whose saved tensors they are is refused, and not wrong."""
    import torch
    torch._C._increment_version(tensors)


def _routed(out, experts: Optional[int], block: Optional[int]):
    """`out`, which now holds metadata of so many experts and this block."""
    if isinstance(out, RouteSortOutput):
        out.experts, out.block = experts, block
    return out


# (device, stream handle) -> the workspaces made for that stream, the last the
# largest.  No call reads workspace words that an earlier call left, so one
# buffer serves every shape that fits in it.
_ws_cache = {}


def _workspace(device, stream_handle: int, nbytes: int):
    """A zeroed workspace of at least nbytes for calls on one stream.

    Calls on one stream run in order and share a buffer; calls on different
    streams may overlap in time and each stream gets buffers of its own.  An
    outgrown buffer is kept, not freed, since a captured graph may still hold
    its address; sizes are powers of two, so a stream's buffers add up to less
    than twice the largest.  A buffer is allocated and filled on its own stream:
    on another one the fill could run beside the kernels that use the buffer."""
    import torch
    bufs = _ws_cache.setdefault((str(device), int(stream_handle)), [])
    if bufs and bufs[-1].numel() >= nbytes:
        return bufs[-1]
    size = 256
    while size < nbytes:
        size *= 2
    own = contextlib.nullcontext()
    if torch.device(device).type == "cuda":
        own = torch.cuda.stream(torch.cuda.ExternalStream(stream_handle, device=device) if stream_handle else
                                torch.cuda.default_stream(device))
    with own:
        bufs.append(torch.zeros(size, dtype=torch.uint8, device=device))
    return bufs[-1]


def _check_tensor(t, dev, dtype, n: int, name: str):
    """t is a contiguous tensor of dtype (any dtype when None) with at least n
    elements on dev; every pointer handed to the library comes through here or
    through a check of the same kind, so no host address reaches a kernel."""
    import torch
    if not (isinstance(t, torch.Tensor) and t.device == dev and (dtype is None or t.dtype == dtype)
            and t.is_contiguous() and t.numel() >= n):
        what = "a" if dtype is None else f"a {dtype}"
        raise ValueError(f"{name} must be {what} contiguous tensor of at least {n} elements on {dev}")


def _check_metadata(sorted_ids, expert_of_block, num_post_pad, rows: int, blocks: int, dev):
    import torch
    for t, n, name in ((sorted_ids, rows, "sorted_ids"), (expert_of_block, blocks, "expert_of_block"),
                       (num_post_pad, 1, "num_post_pad")):
        _check_tensor(t, dev, torch.int32, n, name)


def _check_route_output(out, M: int, k: int, rows: int, blocks: int, dev):
    """A caller's RouteSortOutput: ids and weights exactly [M, k], the metadata
    buffers at least their capacities, all contiguous on dev."""
    import torch
    for t, dtype, name in ((out.ids, torch.int32, "out.ids"), (out.weights, torch.float32, "out.weights")):
        _check_tensor(t, dev, dtype, M * k, name)
        if tuple(t.shape) != (M, k):
            raise ValueError(f"{name} must have shape ({M}, {k})")
    _check_metadata(out.sorted_ids, out.expert_of_block, out.num_post_pad, rows, blocks, dev)


def route_sort(logits, bias, k: int, n_group: int, topk_group: int, block: int, *,
               out: Optional[RouteSortOutput] = None, workspace=None, flags: int = 0,
               stats=None, stream=None, events=None, local=None) -> RouteSortOutput:
    """Run the route-sort path on the GPU.

    logits: [M, E] float32 or bfloat16 CUDA/HIP tensor, contiguous.
    bias:   [E] float32 tensor on the same device.
    out:    optional preallocated RouteSortOutput (reused, nothing else written; a
            backward pass that still needs what it held is refused by autograd).
    workspace: optional uint8 tensor of at least workspace_bytes() bytes that
            was zeroed once; by default a cached buffer of the call's stream
            (calls on different streams may then overlap in time).  Make the
            first call on a stream before capturing a graph on it, or the
            allocation and zero fill of that buffer join the graph.
    stats:  optional int32 [3] device tensor (tokens decided by the workgroup-wide
            exact selection / by one wave / with group scores made exact by one wave).
    events: optional list of 6 torch.cuda.Event(enable_timing=True); events
            2i and 2i+1 take the start and end of the call's kernel i (pairs
            past the last kernel are recorded after it); returns
            (output, launches) then.
    local:  optional (begin, count): metadata only for experts
            [begin, begin + count), numbered from 0 (moe_route_sort_local);
            ids and weights stay global.  Not combined with flags, stats or
            events.
    """
    import torch
    if not (isinstance(logits, torch.Tensor) and logits.is_cuda):
        raise ValueError("logits must be a GPU tensor")
    if logits.dim() != 2 or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous [M, E] tensor")
    if logits.dtype == torch.float32:
        dt = MRS_DTYPE_F32
    elif logits.dtype == torch.bfloat16:
        dt = MRS_DTYPE_BF16
    else:
        raise NotImplementedError(f"logits dtype {logits.dtype} (float32 or bfloat16 only)")
    M, E = logits.shape
    if not (isinstance(bias, torch.Tensor) and bias.device == logits.device and
            bias.dtype == torch.float32 and bias.shape == (E,) and bias.is_contiguous()):
        raise ValueError("bias must be a contiguous float32 [E] tensor on the logits' device")
    dev = logits.device
    if local is not None:
        lb, lc = (int(v) for v in local)
        if not (0 <= lb and 1 <= lc and lb + lc <= E):
            raise ValueError("local range must lie inside [0, E) and hold at least one expert")
        if flags or stats is not None or events is not None:
            raise ValueError("a local range is not combined with flags, stats or events")
    EL = E if local is None else lc
    rows, blocks = _capacity(M, EL, k, block)
    if rows < 0:
        raise ValueError("invalid sizes or row capacity overflow")
    if out is None:
        out = RouteSortOutput(
            torch.empty((M, k), dtype=torch.int32, device=dev),
            torch.empty((M, k), dtype=torch.float32, device=dev),
            torch.empty((max(rows, 1),), dtype=torch.int32, device=dev),
            torch.empty((max(blocks, 1),), dtype=torch.int32, device=dev),
            torch.empty((1,), dtype=torch.int32, device=dev),
        )
    else:
        _check_route_output(out, M, k, rows, blocks, dev)
        _overwritten(out.ids, out.weights, out.sorted_ids, out.expert_of_block, out.num_post_pad)
    if stats is not None:
        _check_tensor(stats, dev, torch.int32, 3, "stats")
    nbytes = workspace_bytes(M, E, k, block)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    if workspace is None:
        workspace = _workspace(dev, stream.cuda_stream, nbytes) if nbytes else None
    else:
        _check_tensor(workspace, dev, None, 0, "workspace")
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if local is not None:
        rc = int(lib().moe_route_sort_local(
            logits.data_ptr(), bias.data_ptr(), M, E, k, n_group, topk_group, block, lb, lc,
            out.ids.data_ptr(), out.weights.data_ptr(), out.sorted_ids.data_ptr(),
            out.expert_of_block.data_ptr(), out.num_post_pad.data_ptr(), dt, ws_ptr, ws_len, stream.cuda_stream))
        if rc != MRS_OK:
            raise RouteSortError(rc)
        return _routed(out, EL, block)
    args = (logits.data_ptr(), bias.data_ptr(), M, E, k, n_group, topk_group, block,
            out.ids.data_ptr(), out.weights.data_ptr(), out.sorted_ids.data_ptr(),
            out.expert_of_block.data_ptr(), out.num_post_pad.data_ptr(), dt, ws_ptr, ws_len,
            stream.cuda_stream, flags, stats.data_ptr() if stats is not None else None)
    if events is not None:
        if len(events) != 6:
            raise ValueError("events must hold 6 torch.cuda.Event objects")
        for ev in events:
            if not ev.cuda_event:
                ev.record(stream)  # torch creates the HIP event on its first record
        handles = (ctypes.c_void_p * 6)(*[ev.cuda_event for ev in events])
        n = ctypes.c_int(0)
        rc = int(lib().moe_route_sort_profiled(*args, handles, ctypes.byref(n)))
        if rc != MRS_OK:
            raise RouteSortError(rc)
        return _routed(out, E, block), n.value
    rc = int(lib().moe_route_sort_ex(*args))
    if rc != MRS_OK:
        raise RouteSortError(rc)
    return _routed(out, E, block)


def route_sort_static(logits, bias, k: int, n_group: int, topk_group: int, block: int, *,
                      out: Optional[RouteSortOutput] = None, stream=None) -> RouteSortOutput:
    """moe_route_sort_static: the route-sort path with the library's own
    static scratch instead of a workspace (for callers that cannot allocate;
    concurrent calls on one GPU race).  Arguments as for route_sort."""
    import torch
    if not (isinstance(logits, torch.Tensor) and logits.is_cuda and logits.dim() == 2 and logits.is_contiguous()):
        raise ValueError("logits must be a contiguous [M, E] GPU tensor")
    if logits.dtype == torch.float32:
        dt = MRS_DTYPE_F32
    elif logits.dtype == torch.bfloat16:
        dt = MRS_DTYPE_BF16
    else:
        raise NotImplementedError(f"logits dtype {logits.dtype} (float32 or bfloat16 only)")
    M, E = logits.shape
    dev = logits.device
    _check_tensor(bias, dev, torch.float32, E, "bias")
    if bias.shape != (E,):
        raise ValueError("bias must be a float32 [E] tensor")
    rows, blocks = max_rows(M, E, k, block), max_blocks(M, E, k, block)
    if rows < 0:
        raise ValueError("invalid sizes or row capacity overflow")
    if out is None:
        out = RouteSortOutput(torch.empty((M, k), dtype=torch.int32, device=dev),
                              torch.empty((M, k), dtype=torch.float32, device=dev),
                              torch.empty((max(rows, 1),), dtype=torch.int32, device=dev),
                              torch.empty((max(blocks, 1),), dtype=torch.int32, device=dev),
                              torch.empty((1,), dtype=torch.int32, device=dev))
    else:
        _check_route_output(out, M, k, rows, blocks, dev)
        _overwritten(out.ids, out.weights, out.sorted_ids, out.expert_of_block, out.num_post_pad)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    rc = int(lib().moe_route_sort_static(logits.data_ptr(), bias.data_ptr(), M, E, k, n_group, topk_group, block,
                                         out.ids.data_ptr(), out.weights.data_ptr(), out.sorted_ids.data_ptr(),
                                         out.expert_of_block.data_ptr(), out.num_post_pad.data_ptr(), dt,
                                         stream.cuda_stream))
    if rc != MRS_OK:
        raise RouteSortError(rc)
    return _routed(out, E, block)


def sigmoid_probe(x):
    """Both sigmoid forms of the kernels on a float32 GPU tensor (diagnostics)."""
    import torch
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype == torch.float32):
        raise ValueError("x must be a float32 GPU tensor")
    x = x.contiguous()
    f = torch.empty_like(x)
    e = torch.empty_like(x)
    rc = lib().moe_route_sort_sigmoid_probe(x.data_ptr(), x.numel(), f.data_ptr(), e.data_ptr(),
                                            torch.cuda.current_stream(x.device).cuda_stream)
    if rc != MRS_OK:
        raise RouteSortError(rc)
    return f, e


def sigmoid_table_probe(bits):
    """Sigmoid of BF16 bit patterns (an int16/uint16-valued GPU tensor) through
    the kernels' LDS table: (single-value form, packed-pair form)."""
    import torch
    if not (isinstance(bits, torch.Tensor) and bits.is_cuda):
        raise ValueError("bits must be a GPU tensor")
    h = bits.contiguous().to(torch.int16)
    o1 = torch.empty(h.shape, dtype=torch.float32, device=h.device)
    o2 = torch.empty_like(o1)
    rc = lib().moe_route_sort_sigmoid_table_probe(h.data_ptr(), h.numel(), o1.data_ptr(), o2.data_ptr(),
                                                  torch.cuda.current_stream(h.device).cuda_stream)
    if rc != MRS_OK:
        raise RouteSortError(rc)
    return o1, o2


class SortOutput(NamedTuple):
    sorted_ids: "torch.Tensor"       # [max_rows] int32; [0, num_post_pad) defined
    expert_of_block: "torch.Tensor"  # [max_blocks] int32
    num_post_pad: "torch.Tensor"     # [1] int32 (device)


def sort_from_ids(ids, E: int, block: int, *, out: Optional[SortOutput] = None, workspace=None,
                  stream=None, counters=None, rows_capacity: Optional[int] = None) -> SortOutput:
    """The two sort phases from caller-given expert ids ([M, k] int32 GPU
    tensor); ids outside [0, E) are dropped routes.

    counters: optional int32 [E] GPU tensor of initial per-expert counters
    (moe_sort_from_ids_counters): counters[e] rows at the head of expert e's
    segment belong to the caller and are not written; the counters advance by
    this call's routes.  rows_capacity (with counters): the sorted_ids entries
    the call may use; by default the length of out.sorted_ids, required when
    no out is given.  If a counter is negative or the rows do not fit,
    num_post_pad reads -1 and nothing else is written."""
    import torch
    if not (isinstance(ids, torch.Tensor) and ids.is_cuda and ids.dtype == torch.int32 and ids.dim() == 2
            and ids.is_contiguous()):
        raise ValueError("ids must be a contiguous int32 [M, k] GPU tensor")
    M, k = ids.shape
    dev = ids.device
    if counters is not None:
        _check_tensor(counters, dev, torch.int32, E, "counters")
        if out is None:
            if rows_capacity is None:
                raise ValueError("rows_capacity is required with counters when no out is given")
            rows, blocks = int(rows_capacity), int(rows_capacity) // block
        else:
            rows = int(out.sorted_ids.numel()) if rows_capacity is None else int(rows_capacity)
            blocks = rows // block
    else:
        rows, blocks = _capacity(M, E, k, block)
        if rows < 0:
            raise ValueError("invalid sizes or row capacity overflow")
    if out is None:
        out = SortOutput(torch.empty((max(rows, 1),), dtype=torch.int32, device=dev),
                         torch.empty((max(blocks, 1),), dtype=torch.int32, device=dev),
                         torch.empty((1,), dtype=torch.int32, device=dev))
    else:
        _check_metadata(out.sorted_ids, out.expert_of_block, out.num_post_pad, rows, blocks, dev)
        _overwritten(out.sorted_ids, out.expert_of_block, out.num_post_pad)
    nbytes = workspace_bytes(M, E, k, block)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    if workspace is None:
        workspace = _workspace(dev, stream.cuda_stream, nbytes) if nbytes else None
    else:
        _check_tensor(workspace, dev, None, 0, "workspace")
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if counters is not None:
        rc = int(lib().moe_sort_from_ids_counters(ids.data_ptr() if M else None, M, E, k, block,
                                                  counters.data_ptr(), rows, out.sorted_ids.data_ptr(),
                                                  out.expert_of_block.data_ptr(), out.num_post_pad.data_ptr(),
                                                  ws_ptr, ws_len, stream.cuda_stream))
    else:
        rc = int(lib().moe_sort_from_ids(ids.data_ptr(), M, E, k, block, out.sorted_ids.data_ptr(),
                                         out.expert_of_block.data_ptr(), out.num_post_pad.data_ptr(), ws_ptr,
                                         ws_len, stream.cuda_stream))
    if rc != MRS_OK:
        raise RouteSortError(rc)
    return out


def grouped_gemm1(x, w, sorted_ids, expert_of_block, num_post_pad, k: int, block: int, *,
                  out=None, stream=None, events=None):
    """First grouped GEMM of the MoE over the route-sort metadata
    (include/moe_gemm1.h): y[r] = x[sorted_ids[r] // k] . W[expert_of_block[r // block]]^T
    for sorted rows below num_post_pad, zeros for padding rows.

    x: [M, K] bfloat16, w: [E, N, K] bfloat16, metadata as returned by
    route_sort / sort_from_ids.  Returns y, [max_rows, N] bfloat16 (rows at
    or past num_post_pad are left as they were).  `events` = (start, stop)
    torch.cuda.Event pair stamped by the kernel's own launch."""
    import torch
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 2
            and x.is_contiguous()):
        raise ValueError("x must be a contiguous bfloat16 [M, K] GPU tensor")
    if not (isinstance(w, torch.Tensor) and w.device == x.device and w.dtype == torch.bfloat16 and w.dim() == 3
            and w.is_contiguous()):
        raise ValueError("w must be a contiguous bfloat16 [E, N, K] tensor on x's device")
    M, K = x.shape
    E, N, K2 = w.shape
    if K2 != K:
        raise ValueError("x and w disagree on K")
    rows = max_rows(M, E, k, block)
    blocks = max_blocks(M, E, k, block)
    if rows < 0:
        raise ValueError("invalid sizes or row capacity overflow")
    _check_metadata(sorted_ids, expert_of_block, num_post_pad, rows, blocks, x.device)
    if out is None:
        out = torch.empty((max(rows, 1), N), dtype=torch.bfloat16, device=x.device)
    elif not (out.device == x.device and out.dtype == torch.bfloat16 and out.is_contiguous()
              and out.dim() == 2 and out.shape[1] == N and out.shape[0] >= rows):
        raise ValueError("out must be a contiguous bfloat16 [max_rows, N] tensor on x's device")
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    args = (x.data_ptr(), w.data_ptr(), sorted_ids.data_ptr(), expert_of_block.data_ptr(),
            num_post_pad.data_ptr(), M, k, E, K, N, block, out.data_ptr(), stream.cuda_stream)
    if events is not None:
        ev0, ev1 = events
        for ev in (ev0, ev1):
            if not ev.cuda_event:
                ev.record(stream)  # torch creates the HIP event on its first record
        rc = int(lib().moe_grouped_gemm1_profiled(*args, ev0.cuda_event, ev1.cuda_event))
    else:
        rc = int(lib().moe_grouped_gemm1(*args))
    if rc != MRS_OK:
        raise RouteSortError(rc)
    return out


def gate_route_sort(hidden, w_gate, bias, k: int, n_group: int, topk_group: int, block: int, *,
                    out: Optional[RouteSortOutput] = None, logits=None, stream=None):
    """Router gate projection then the route-sort path (include/moe_gate.h).

    hidden: [M, H] bfloat16 (M <= 64), w_gate: [E, H] bfloat16, bias: [E]
    float32, all on one GPU.  Returns (logits [M, E] float32, RouteSortOutput)."""
    import torch
    if not (isinstance(hidden, torch.Tensor) and hidden.is_cuda and hidden.dtype == torch.bfloat16 and
            hidden.dim() == 2 and hidden.is_contiguous()):
        raise ValueError("hidden must be a contiguous bfloat16 [M, H] GPU tensor")
    if not (isinstance(w_gate, torch.Tensor) and w_gate.device == hidden.device and
            w_gate.dtype == torch.bfloat16 and w_gate.dim() == 2 and w_gate.is_contiguous()):
        raise ValueError("w_gate must be a contiguous bfloat16 [E, H] tensor on hidden's device")
    M, H = hidden.shape
    E = w_gate.shape[0]
    if w_gate.shape[1] != H:
        raise ValueError("hidden and w_gate disagree on H")
    if not (isinstance(bias, torch.Tensor) and bias.device == hidden.device and bias.dtype == torch.float32 and
            bias.shape == (E,) and bias.is_contiguous()):
        raise ValueError("bias must be a contiguous float32 [E] tensor on hidden's device")
    dev = hidden.device
    rows, blocks = max_rows(M, E, k, block), max_blocks(M, E, k, block)
    if rows < 0:
        raise ValueError("invalid sizes or row capacity overflow")
    if logits is None:
        logits = torch.empty((M, E), dtype=torch.float32, device=dev)
    elif not (logits.dtype == torch.float32 and tuple(logits.shape) == (M, E) and logits.is_contiguous() and
              logits.device == dev):
        raise ValueError("logits must be a contiguous float32 [M, E] tensor on hidden's device")
    else:
        _overwritten(logits)
    if out is None:
        out = RouteSortOutput(torch.empty((M, k), dtype=torch.int32, device=dev),
                              torch.empty((M, k), dtype=torch.float32, device=dev),
                              torch.empty((max(rows, 1),), dtype=torch.int32, device=dev),
                              torch.empty((max(blocks, 1),), dtype=torch.int32, device=dev),
                              torch.empty((1,), dtype=torch.int32, device=dev))
    else:
        _check_route_output(out, M, k, rows, blocks, dev)
        _overwritten(out.ids, out.weights, out.sorted_ids, out.expert_of_block, out.num_post_pad)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    rc = int(lib().moe_gate_route_sort(hidden.data_ptr(), w_gate.data_ptr(), bias.data_ptr(), M, E, H, k, n_group,
                                       topk_group, block, logits.data_ptr(), out.ids.data_ptr(),
                                       out.weights.data_ptr(), out.sorted_ids.data_ptr(),
                                       out.expert_of_block.data_ptr(), out.num_post_pad.data_ptr(),
                                       stream.cuda_stream))
    if rc != MRS_OK:
        raise RouteSortError(rc)
    return logits, _routed(out, E, block)


class MXFP4(NamedTuple):
    """4-bit rows (include/moe_mxfp4.h): K columns padded with zeros to Kp, a
    multiple of 128, in blocks of 32 that share a scale byte."""
    codes: "torch.Tensor"   # uint8 [..., Kp / 2], two codes a byte, the even column in the low half
    scales: "torch.Tensor"  # uint8 [..., Kp / 32], 2^(byte - 127), 255 = NaN


def _handle(stream, dev) -> int:
    """The HIP stream handle of `stream`, by default of dev's current stream."""
    import torch
    return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream


def _foreign(stream, dev):
    """`stream` where it is not dev's current stream, else None."""
    return None if stream.cuda_stream == _handle(None, dev) else stream


def _allocate(foreign, dev, make, *args):
    """make(*args), the tensors that a call on the stream `foreign` writes: out of
    that stream's memory (a block that the current stream's work still reads is not
    written), and not given back before the current stream, where they go, is
    through with them."""
    import torch
    with torch.cuda.stream(foreign):
        made = make(*args)
    current = torch.cuda.current_stream(dev)
    for t in made if isinstance(made, tuple) else (made,):
        t.record_stream(current)
    return made


def _hold(foreign, *tensors):
    """The memory of what a call on the stream `foreign` reads or writes is not
    given back before that stream has passed the call."""
    for t in tensors:
        if t is not None:
            t.record_stream(foreign)


def _empty(shape, dtype, dev):
    """A contiguous tensor.  With the strides given, torch takes 1.3 us in place of
    1.7, which shows in calls of a token or two."""
    import torch
    if len(shape) == 1:
        return torch.empty_strided(shape, (1,), dtype=dtype, device=dev)
    if len(shape) == 2:
        return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=dev)
    if len(shape) == 3:
        return torch.empty_strided(shape, (shape[1] * shape[2], shape[2], 1), dtype=dtype, device=dev)
    return torch.empty(shape, dtype=dtype, device=dev)


@functools.lru_cache(maxsize=4096)
def _capacity(M: int, E: int, k: int, block: int):
    return max_rows(M, E, k, block), max_blocks(M, E, k, block)


def _check_mxfp4(q, dev, dims: int, name: str) -> int:
    """q holds contiguous 4-bit rows with `dims` dimensions on dev; returns Kp."""
    import torch
    codes, scales = q if isinstance(q, MXFP4) else (None, None)
    u8 = torch.uint8
    if not (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor) and codes.device == dev
            and scales.device == dev and codes.dtype == u8 and scales.dtype == u8 and codes.dim() == dims
            and scales.dim() == dims and codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name} must be an MXFP4 of contiguous uint8 tensors with {dims} dimensions on {dev}")
    *lead, n = codes.shape
    Kp = n * 2
    if Kp == 0 or Kp % 128 or scales.shape != (*lead, Kp // 32):
        raise ValueError(f"{name}: codes [..., Kp / 2] and scales [..., Kp / 32] of the same rows, Kp a multiple of 128")
    return Kp


def _new_mxfp4(lead, Kp: int, u8, dev) -> MXFP4:
    return MXFP4(_empty((*lead, Kp // 2), u8, dev), _empty((*lead, Kp // 32), u8, dev))


def _row_stride(x, K: int) -> int:
    """The stride of x's rows of K consecutive values, leading dimensions collapsed."""
    if x.numel() == 0 or x.is_contiguous():
        return K
    if K > 1 and x.stride(-1) != 1:
        raise ValueError("x's last dimension must be consecutive")
    step = None  # stride of the rows, from the innermost leading dimension outwards
    span = 1
    for n, st in zip(x.shape[-2::-1], x.stride()[-2::-1]):
        if n == 1:
            continue
        if step is None:
            step = st
        elif st != step * span:
            raise ValueError("x's leading dimensions must collapse to rows of one stride")
        span *= n
    row_stride = K if step is None else step
    if row_stride < K:
        raise ValueError("x's rows must not overlap")
    return row_stride


def mxfp4_quantize(x, *, values=None, out: Optional[MXFP4] = None, stream=None) -> MXFP4:
    """Rows of x to 4-bit rows (moe_mxfp4_quantize).

    x: float32, bfloat16 or float16 GPU tensor [..., K], 1 <= K <= 262144; the
    last dimension is consecutive and the leading ones collapse to rows of one
    stride (a slice of a wider buffer's columns is fine).
    values: optional contiguous tensor of x's shape and type that takes the
    values the 4-bit rows stand for, for training with rounded values.  It is a
    plain buffer: rounding has no slope, and x whose gradient it would drop is
    refused in grad mode.  The gradient that passes the rounding by is
        amr.mxfp4_quantize(x.detach(), values=v);  y = x + (v - x.detach())
    out: optional MXFP4 to write into, codes [..., Kp / 2], scales [..., Kp / 32].
    stream: the stream to run on, by default the current one; on another the
    caller orders it after what made the inputs and before what reads the results."""
    import torch
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dim() >= 1):
        raise ValueError("x must be a GPU tensor of at least one dimension")
    dts = {torch.float32: MRS_DTYPE_F32, torch.bfloat16: MRS_DTYPE_BF16, torch.float16: MRS_DTYPE_F16}
    if x.dtype not in dts:
        raise NotImplementedError(f"x dtype {x.dtype} (float32, bfloat16 or float16 only)")
    *lead, K = x.shape
    if not 1 <= K <= 262144:
        raise ValueError("the last dimension must hold 1 to 262144 values")
    rows, row_stride = x.numel() // K, _row_stride(x, K)
    dev = x.device
    Kp = (K + 127) // 128 * 128
    foreign = None if stream is None else _foreign(stream, dev)
    if out is None:
        out = (_new_mxfp4(lead, Kp, torch.uint8, dev) if foreign is None else
               _allocate(foreign, dev, _new_mxfp4, lead, Kp, torch.uint8, dev))
    else:
        _check_mxfp4(out, dev, x.dim(), "out")
        if out.codes.shape != (*lead, Kp // 2):
            raise ValueError(f"out.codes must have shape {(*lead, Kp // 2)}")
    if values is not None:
        _check_tensor(values, dev, x.dtype, x.numel(), "values")
        if values.shape != x.shape:
            raise ValueError("values must have x's shape")
        if (x.requires_grad or values.requires_grad) and torch.is_grad_enabled():
            raise ValueError("values carries no gradient: quantise x.detach(), and use x + (values - x.detach())")
    handle = _handle(stream, dev)
    rc = int(lib().moe_mxfp4_quantize(x.data_ptr(), dts[x.dtype], rows, K, row_stride, out.codes.data_ptr(),
                                      out.scales.data_ptr(), values.data_ptr() if values is not None else None,
                                      handle))
    if foreign is not None:
        _hold(foreign, x, *out, values)
    if rc != MRS_OK:
        raise RouteSortError(rc)
    return out


def grouped_gemm_mxfp4(x: MXFP4, w: MXFP4, sorted_ids, expert_of_block, num_post_pad, k: int, block: int, *,
                       tokens: Optional[int] = None, out_dtype=None, out=None, stream=None,
                       kernel: int = PRODUCT_BY_RULE):
    """Grouped product of 4-bit rows over the route-sort metadata
    (moe_grouped_gemm_mxfp4): y[r] = x[row(r)] . W[expert_of_block[r // block]]^T
    for sorted rows below num_post_pad, zeros for padding rows.

    x: 4-bit rows of the M tokens, row(r) = sorted_ids[r] // k; with `tokens` = M
    given, x holds max_rows rows in sorted order and row(r) = r (a later product
    on the rows an earlier one wrote).  w: 4-bit rows [E, N].  block: a multiple
    of 16.  out_dtype: bfloat16 (default) or float32.  Returns y [max_rows, N];
    rows at or past num_post_pad are left as they were.  stream: as for
    mxfp4_quantize.  kernel: a PRODUCT_* constant in place of the choice by sizes
    (moe_grouped_gemm_mxfp4_ex; for tests and tuning)."""
    import torch
    if not (isinstance(x, MXFP4) and isinstance(x.codes, torch.Tensor) and x.codes.is_cuda):
        raise ValueError("x must be an MXFP4 of GPU tensors")
    dev = x.codes.device
    Kp = _check_mxfp4(x, dev, 2, "x")
    if _check_mxfp4(w, dev, 3, "w") != Kp:
        raise ValueError("x and w disagree on K")
    E, N = w.codes.shape[:2]
    M = x.codes.shape[0] if tokens is None else int(tokens)
    rows, blocks = _capacity(M, E, k, block)
    if rows < 0:
        raise ValueError("invalid sizes or row capacity overflow")
    if tokens is not None and x.codes.shape[0] < rows:
        raise ValueError(f"x must hold at least {rows} rows in sorted order")
    _check_metadata(sorted_ids, expert_of_block, num_post_pad, rows, blocks, dev)
    foreign = None if stream is None else _foreign(stream, dev)
    if out is None:
        new = (max(rows, 1), N), out_dtype or torch.bfloat16, dev
        out = _empty(*new) if foreign is None else _allocate(foreign, dev, _empty, *new)
    elif not (isinstance(out, torch.Tensor) and out.device == dev and out.is_contiguous() and out.dim() == 2
              and out.shape[1] == N and out.shape[0] >= rows and (out_dtype is None or out.dtype == out_dtype)):
        raise ValueError("out must be a contiguous [max_rows, N] tensor of out_dtype on x's device")
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise NotImplementedError(f"y dtype {out.dtype} (bfloat16 or float32 only)")
    handle = _handle(stream, dev)
    rc = int(lib().moe_grouped_gemm_mxfp4_ex(
        x.codes.data_ptr(), x.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(), sorted_ids.data_ptr(),
        expert_of_block.data_ptr(), num_post_pad.data_ptr(), M, k, E, Kp, N, block,
        MRS_X_TOKENS if tokens is None else MRS_X_SORTED,
        MRS_DTYPE_BF16 if out.dtype == torch.bfloat16 else MRS_DTYPE_F32, out.data_ptr(), handle, kernel))
    if foreign is not None:
        _hold(foreign, *x, *w, sorted_ids, expert_of_block, num_post_pad, out)
    if rc != MRS_OK:
        raise RouteSortError(rc)
    return out


class BalanceOutput(NamedTuple):
    loss: "torch.Tensor"    # [1] float32
    counts: "torch.Tensor"  # [B, E] int32, routes per sequence and expert
    tokens: "torch.Tensor"  # [B + 1] int32, unmasked tokens per sequence, then the sequences that have any
    shares: "torch.Tensor"  # [B, E] float32, mean normalised score


def _check_router(logits, ids, seq_offsets, mask):
    """Common checks of balance_loss and router_backward: (dtype code, M, E, k, B)."""
    import torch
    if not (isinstance(logits, torch.Tensor) and logits.is_cuda and logits.dim() == 2 and logits.is_contiguous()):
        raise ValueError("logits must be a contiguous [M, E] GPU tensor")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise NotImplementedError(f"logits dtype {logits.dtype} (float32 or bfloat16 only)")
    M, E = logits.shape
    dev = logits.device
    _check_tensor(ids, dev, torch.int32, 0, "ids")
    if ids.dim() != 2 or ids.shape[0] != M:
        raise ValueError(f"ids must have shape ({M}, k)")
    B = 1
    if seq_offsets is not None:
        _check_tensor(seq_offsets, dev, torch.int32, 2, "seq_offsets")
        if seq_offsets.dim() != 1:
            raise ValueError("seq_offsets must have one dimension")
        B = seq_offsets.numel() - 1
    if mask is not None:
        if not (isinstance(mask, torch.Tensor) and mask.dtype in (torch.bool, torch.uint8)):
            raise ValueError("mask must be a bool or uint8 tensor")
        _check_tensor(mask, dev, None, M, "mask")
        if tuple(mask.shape) != (M,):
            raise ValueError(f"mask must have shape ({M},)")
    return (MRS_DTYPE_F32 if logits.dtype == torch.float32 else MRS_DTYPE_BF16), M, E, ids.shape[1], B


def _ptr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=4096)
def balance_workspace_bytes(M: int, E: int, k: int, B: int = 1) -> int:
    v = int(lib().moe_balance_workspace_bytes(M, E, k, B))
    if v == ctypes.c_size_t(-1).value:
        raise ValueError("invalid sizes")
    return v


def _new_balance(B: int, E: int, f32, i32, dev) -> BalanceOutput:
    return BalanceOutput(_empty((1,), f32, dev), _empty((B, E), i32, dev), _empty((B + 1,), i32, dev),
                         _empty((B, E), f32, dev))


def _clones(*tensors):
    return tuple(t.clone() for t in tensors)


def balance_loss(logits, ids, coef: float = 1.0, *, seq_offsets=None, mask=None, out: Optional[BalanceOutput] = None,
                 workspace=None, stream=None) -> BalanceOutput:
    """Balance loss, per-expert counts and mean scores of a routing
    (moe_balance_loss, include/moe_balance.h).

    logits: [M, E] float32 or bfloat16, ids: [M, k] int32 as route_sort returns
    them (ids outside [0, E) are dropped routes).  seq_offsets: int32 [B + 1],
    the loss is the mean over the sequences; mask: bool or uint8 [M], zero for
    padding tokens.  workspace: as for route_sort (balance_workspace_bytes);
    stream: as for mxfp4_quantize.

    Where logits require a gradient (and grad mode is on) the returned loss carries
    it (router_backward; counts and ids are constants).  With `out` the returned
    loss is another tensor on out.loss's memory, and only the returned one does.
    A captured training step calls router_backward itself (as for route_sort_train)."""
    import torch
    dt, M, E, k, B = _check_router(logits, ids, seq_offsets, mask)
    dev = logits.device
    nbytes = balance_workspace_bytes(M, E, k, B)
    foreign = None if stream is None else _foreign(stream, dev)
    given = out is not None
    if not given:
        new = B, E, torch.float32, torch.int32, dev
        out = _new_balance(*new) if foreign is None else _allocate(foreign, dev, _new_balance, *new)
    else:
        for t, dtype, shape, name in ((out.loss, torch.float32, (1,), "out.loss"),
                                      (out.counts, torch.int32, (B, E), "out.counts"),
                                      (out.tokens, torch.int32, (B + 1,), "out.tokens"),
                                      (out.shares, torch.float32, (B, E), "out.shares")):
            _check_tensor(t, dev, dtype, 1, name)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must have shape {shape}")
    handle = _handle(stream, dev)
    if workspace is None:
        workspace = _workspace(dev, handle, nbytes)
    else:
        _check_tensor(workspace, dev, None, 0, "workspace")
    rc = int(lib().moe_balance_loss(logits.data_ptr(), dt, ids.data_ptr(), _ptr(seq_offsets), _ptr(mask), M, E, k, B,
                                    float(coef), out.loss.data_ptr(), out.counts.data_ptr(), out.tokens.data_ptr(),
                                    out.shares.data_ptr(), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), handle))
    if foreign is not None:
        _hold(foreign, logits, ids, seq_offsets, mask, *out, workspace)
    if rc != MRS_OK:
        raise RouteSortError(rc)
    if logits.requires_grad and torch.is_grad_enabled():
        loss, counts, tokens, _ = out
        if given:  # the caller may write its buffers again before the backward pass
            loss = loss.detach()
            counts, tokens = (_clones(counts, tokens) if foreign is None else
                              _allocate(foreign, dev, _clones, counts, tokens))
        out = out._replace(loss=_balance_function().apply(logits, (loss,), ids, counts, tokens, float(coef), seq_offsets,
                                                          mask))
    return out


@functools.lru_cache(maxsize=1)
def _balance_function():
    import torch
    from torch.autograd.function import once_differentiable

    class Balance(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, box, ids, counts, tokens, coef, seq_offsets, mask):
            ctx.save_for_backward(logits, ids, counts, tokens, seq_offsets, mask)
            ctx.coef = coef
            return box[0]  # in a tuple: as an argument of its own torch would return a view of it

        @staticmethod
        @once_differentiable
        def backward(ctx, grad_loss):
            logits, ids, counts, tokens, seq_offsets, mask = ctx.saved_tensors
            return (router_backward(logits, ids, balance=BalanceOutput(None, counts, tokens, None), coef=ctx.coef,
                                    grad_loss=grad_loss.float().contiguous(), seq_offsets=seq_offsets, mask=mask),
                    ) + (None,) * 7

    return Balance


def router_backward(logits, ids, *, grad_weights=None, balance: Optional[BalanceOutput] = None, coef: float = 1.0,
                    grad_loss=None, seq_offsets=None, mask=None, out=None, stream=None):
    """Gradient of the logits (moe_router_backward): of the balance loss when
    `balance` (what balance_loss returned for the same logits, ids, seq_offsets
    and mask) is given, times grad_loss (float32 [1], default 1), plus that of
    the routing weights when grad_weights ([M, k] float32) is given.  Returns
    [M, E] of the logits' type.  stream: as for mxfp4_quantize."""
    import torch
    dt, M, E, k, B = _check_router(logits, ids, seq_offsets, mask)
    dev = logits.device
    if grad_weights is not None:
        _check_tensor(grad_weights, dev, torch.float32, M * k, "grad_weights")
        if tuple(grad_weights.shape) != (M, k):
            raise ValueError(f"grad_weights must have shape ({M}, {k})")
    if balance is not None:
        for t, shape, name in ((balance.counts, (B, E), "balance.counts"), (balance.tokens, (B + 1,), "balance.tokens")):
            _check_tensor(t, dev, torch.int32, 1, name)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must have shape {shape}")
    if grad_loss is not None:
        _check_tensor(grad_loss, dev, torch.float32, 1, "grad_loss")
    foreign = None if stream is None else _foreign(stream, dev)
    if out is None:
        out = torch.empty_like(logits) if foreign is None else _allocate(foreign, dev, torch.empty_like, logits)
    else:
        _check_tensor(out, dev, logits.dtype, M * E, "out")
        if out.shape != logits.shape:
            raise ValueError("out must have the logits' shape")
    handle = _handle(stream, dev)
    rc = int(lib().moe_router_backward(logits.data_ptr(), dt, ids.data_ptr(), _ptr(grad_weights),
                                       _ptr(balance.counts) if balance is not None else None,
                                       _ptr(balance.tokens) if balance is not None else None, _ptr(grad_loss),
                                       _ptr(seq_offsets), _ptr(mask), M, E, k, B, float(coef), out.data_ptr(),
                                       handle))
    if foreign is not None:
        _hold(foreign, logits, ids, grad_weights, grad_loss, seq_offsets, mask, out,
              *(() if balance is None else (balance.counts, balance.tokens)))
    if rc != MRS_OK:
        raise RouteSortError(rc)
    return out


@functools.lru_cache(maxsize=1)
def _route_train_function():
    import torch
    from torch.autograd.function import once_differentiable

    class RouteTrain(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, bias, sizes, coef, seq_offsets, mask):
            out = route_sort(logits, bias, *sizes)
            rc = int(lib().moe_route_far_weights(logits.data_ptr(),
                                                 MRS_DTYPE_F32 if logits.dtype == torch.float32 else MRS_DTYPE_BF16,
                                                 out.ids.data_ptr(), *logits.shape, sizes[0], out.weights.data_ptr(),
                                                 _handle(None, logits.device)))
            if rc != MRS_OK:
                raise RouteSortError(rc)
            bal = balance_loss(logits, out.ids, coef, seq_offsets=seq_offsets, mask=mask)
            ctx.save_for_backward(logits, out.ids, bal.counts, bal.tokens, seq_offsets, mask)
            ctx.coef = coef
            ctx.set_materialize_grads(False)
            rest = (out.ids, out.sorted_ids, out.expert_of_block, out.num_post_pad, bal.counts, bal.tokens, bal.shares)
            ctx.mark_non_differentiable(*rest)
            return (out.weights, bal.loss) + rest

        @staticmethod
        @once_differentiable
        def backward(ctx, grad_weights, grad_loss, *_):
            logits, ids, counts, tokens, seq_offsets, mask = ctx.saved_tensors
            if grad_weights is None and grad_loss is None:
                return (None,) * 6
            balance = None if grad_loss is None else BalanceOutput(None, counts, tokens, None)
            grad = router_backward(logits, ids, balance=balance, coef=ctx.coef, seq_offsets=seq_offsets, mask=mask,
                                   grad_weights=None if grad_weights is None else grad_weights.float().contiguous(),
                                   grad_loss=None if grad_loss is None else grad_loss.float().contiguous())
            return (grad,) + (None,) * 5

    return RouteTrain


def route_sort_train(logits, bias, k: int, n_group: int, topk_group: int, block: int, *, balance_coef: float = 0.0,
                     seq_offsets=None, mask=None):
    """route_sort and balance_loss under autograd: (RouteSortOutput, BalanceOutput)
    whose `weights` and `loss` carry gradients to logits (router_backward; the
    selection and the counts are constants, the bias gets no gradient).

    logits, bias and sizes as for route_sort, coefficient, seq_offsets and mask as
    for balance_loss; padding tokens (mask) are routed as any other but take part
    in neither the loss nor the gradients.  Tokens whose picked logits all lie below
    -87 (rows of the type's lowest value, say) get the weights that the gradient is
    the gradient of, in place of the route's infinite or NaN quotients of vanished
    scores (moe_route_far_weights).  To capture a training step in a graph
    call balance_loss and router_backward themselves."""
    w, loss, ids, sid, eob, npp, counts, tokens, shares = _route_train_function().apply(
        logits, bias, (k, n_group, topk_group, block), float(balance_coef), seq_offsets, mask)
    route = _routed(RouteSortOutput(ids, w, sid, eob, npp), logits.shape[1], block)
    return route, BalanceOutput(loss, counts, tokens, shares)


_EXPERTS = ("Int4", "combine", "combine_backward", "experts_train", "grouped_gemm", "grouped_gemm_dw", "grouped_gemm_dx",
            "int4_matvec", "int4_quantize", "slot_rows", "swiglu", "swiglu_backward")


def __getattr__(name):
    """The experts' operators (experts.py), which import torch with their module: loaded
    when the first is asked for."""
    if name not in _EXPERTS:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    from . import experts
    globals().update({n: getattr(experts, n) for n in _EXPERTS})
    return globals()[name]


def __dir__():
    return sorted({*globals(), *_EXPERTS})
