"""Python binding of the experts' operators: 16-bit products grouped by expert with
their gradients, the gated activation, the mix of the outputs (include/moe_experts.h)
and matrix-vector products with 4-bit weights (include/moe_int4.h).

Checks of arguments, allocation and streams as in the package's other calls: every
call runs on the current stream, or on `stream`, which the caller then orders after
what made the inputs and before what reads the results.  The calls that have an
explicit backward entry point take no part in autograd and refuse, in grad mode,
inputs whose gradient they would drop; experts_train joins them under autograd.  Nor
does autograd hear of what they write into `out`: that must be no tensor which a
backward pass still reads.
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import (MRS_DTYPE_BF16, MRS_DTYPE_F16, MRS_DTYPE_F32, MRS_INT4_GATED, MRS_INT4_PLAIN, MRS_INT4_SUM, MRS_OK,
               MRS_X_SORTED, MRS_X_TOKENS, RouteSortError, _allocate, _capacity, _check_metadata, _check_tensor, _empty,
               _foreign, _handle, _hold, _ptr, _row_stride, lib)


_CODES = {torch.bfloat16: MRS_DTYPE_BF16, torch.float16: MRS_DTYPE_F16}
_CODES_F32 = {**_CODES, torch.float32: MRS_DTYPE_F32}


def _code(dtype, name: str, f32: bool = False) -> int:
    code = (_CODES_F32 if f32 else _CODES).get(dtype)
    if code is None:
        raise NotImplementedError(f"{name} dtype {dtype} (bfloat16{', float16 or float32' if f32 else ' or float16'} only)")
    return code


def _is(t, index: int, dtype) -> bool:
    """t is a contiguous tensor of dtype on GPU `index` (short: a call of a token or two
    takes as long as its checks)."""
    return isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype == dtype and t.is_contiguous()


def _first(t, dims: int, name: str):
    """(type code, device, its index) of a call's first matrix."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == dims and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous GPU tensor of {dims} dimensions")
    return _code(t.dtype, name), t.device, t.get_device()


def _matrix(t, dims: int, name: str, index: int, dtype):
    """t is a contiguous tensor of `dims` dimensions and dtype on GPU `index`."""
    if not (_is(t, index, dtype) and t.dim() == dims):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {dims} dimensions on GPU {index}")


def _metadata(sorted_ids, expert_of_block, num_post_pad, rows: int, blocks: int, dev, index: int):
    i32 = torch.int32
    if not (_is(sorted_ids, index, i32) and sorted_ids.numel() >= rows and _is(expert_of_block, index, i32)
            and expert_of_block.numel() >= blocks and _is(num_post_pad, index, i32) and num_post_pad.numel() >= 1):
        _check_metadata(sorted_ids, expert_of_block, num_post_pad, rows, blocks, dev)


def _no_grad(what: str, *tensors):
    for t in tensors:
        if t is None or not t.requires_grad or not torch.is_grad_enabled():
            continue
        raise ValueError(f"{what} takes no part in autograd: call it under no_grad with its backward entry point, "
                         "or use experts_train")


def _output(out, shape, dtype, dev, foreign, rows: Optional[int] = None):
    """`out` checked (its first dimension may be larger than `rows`), or a new tensor."""
    if out is None:
        return _empty(shape, dtype, dev) if foreign is None else _allocate(foreign, dev, _empty, shape, dtype, dev)
    if not (isinstance(out, torch.Tensor) and out.device == dev and out.dtype == dtype and out.is_contiguous()
            and out.dim() == len(shape) and out.shape[1:] == tuple(shape[1:])
            and (out.shape[0] == shape[0] if rows is None else out.shape[0] >= rows)):
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}")
    return out


def _call(dev, entry, *args):
    """An entry point of the library with dev as the current device, whichever that is:
    the default stream's handle does not name its device."""
    if torch._C._cuda_getDevice() == dev.index:
        rc = entry(*args)
    else:
        with torch.cuda.device(dev):
            rc = entry(*args)
    return int(rc)


def _raise(rc: int):
    if rc != MRS_OK:
        raise RouteSortError(rc)


def _sizes(M: int, E: int, k: int, block: int):
    rows, blocks = _capacity(M, E, k, block)
    if rows < 0:
        raise ValueError("invalid sizes or row capacity overflow")
    return rows, blocks


def grouped_gemm(x, w, sorted_ids, expert_of_block, num_post_pad, k: int, block: int, *, tokens: Optional[int] = None,
                 out_dtype=None, out=None, stream=None, tile: int = 0):
    """16-bit product grouped by expert over the route-sort metadata
    (moe_grouped_gemm): y[r] = x[row(r)] . w[expert_of_block[r // block]]^T for sorted
    rows below num_post_pad, zeros for padding rows.

    x: [M, K] bfloat16 or float16, row(r) = sorted_ids[r] // k; with `tokens` = M given
    x holds max_rows rows in sorted order and row(r) = r.  w: [E, N, K] of x's type.
    Any K and N; block: a multiple of 16.  out_dtype: x's type (default) or float32.
    Returns y [max_rows, N]; rows at or past num_post_pad, and those of a block whose
    expert w does not hold, are left as they were.  tile: rows of a tile (16, 32, 64 or
    128, dividing block; MRS_TILE_NARROW | 16, 32 or 64) in place of the choice by sizes,
    for tests and tuning."""
    dt, dev, index = _first(x, 2, "x")
    _matrix(w, 3, "w", index, x.dtype)
    E, N, K = w.shape
    given, width = x.shape
    if width != K:
        raise ValueError("x and w disagree on K")
    _no_grad("grouped_gemm", x, w)
    M = given if tokens is None else int(tokens)
    rows, blocks = _sizes(M, E, k, block)
    if tokens is not None and given < rows:
        raise ValueError(f"x must hold at least {rows} rows in sorted order")
    _metadata(sorted_ids, expert_of_block, num_post_pad, rows, blocks, dev, index)
    foreign = None if stream is None else _foreign(stream, dev)
    out_dtype = out_dtype or (x.dtype if out is None else out.dtype)
    odt = dt if out_dtype == x.dtype else _code(out_dtype, "out", True)
    out = _output(out, (max(rows, 1), N), out_dtype, dev, foreign, rows)
    rc = _call(dev, lib().moe_grouped_gemm_ex, x.data_ptr(), w.data_ptr(), dt, sorted_ids.data_ptr(),
               expert_of_block.data_ptr(), num_post_pad.data_ptr(), M, k, E, K, N, block,
               MRS_X_TOKENS if tokens is None else MRS_X_SORTED, odt, out.data_ptr(),
               _handle(stream, dev), tile)
    if foreign is not None:
        _hold(foreign, x, w, sorted_ids, expert_of_block, num_post_pad, out)
    _raise(rc)
    return out


def grouped_gemm_dx(dy, w, sorted_ids, expert_of_block, num_post_pad, tokens: int, k: int, block: int, *,
                    out_dtype=None, out=None, stream=None, tile: int = 0):
    """Gradient of grouped_gemm's x in sorted rows (moe_grouped_gemm_dx): dx[r] = dy[r] .
    w[expert_of_block[r // block]], zeros for padding rows.

    dy: [max_rows, N], w: [E, N, K] of dy's type (bfloat16 or float16), tokens: M.
    Returns dx [max_rows, K] of dy's type (default) or float32; rows at or past
    num_post_pad, and those of a block whose expert w does not hold, are left as they
    were.  Of an x that holds the tokens' rows the gradient is combine(dx,
    slot_rows(...)).  tile: as for grouped_gemm."""
    dt, dev, index = _first(dy, 2, "dy")
    _matrix(w, 3, "w", index, dy.dtype)
    E, N, K = w.shape
    if dy.shape[1] != N:
        raise ValueError("dy and w disagree on N")
    _no_grad("grouped_gemm_dx", dy, w)
    M = int(tokens)
    rows, blocks = _sizes(M, E, k, block)
    if dy.shape[0] < rows:
        raise ValueError(f"dy must hold at least {rows} rows in sorted order")
    _metadata(sorted_ids, expert_of_block, num_post_pad, rows, blocks, dev, index)
    foreign = None if stream is None else _foreign(stream, dev)
    out_dtype = out_dtype or (dy.dtype if out is None else out.dtype)
    odt = dt if out_dtype == dy.dtype else _code(out_dtype, "out", True)
    out = _output(out, (max(rows, 1), K), out_dtype, dev, foreign, rows)
    rc = _call(dev, lib().moe_grouped_gemm_dx_ex, dy.data_ptr(), w.data_ptr(), dt, sorted_ids.data_ptr(),
               expert_of_block.data_ptr(), num_post_pad.data_ptr(), M, k, E, K, N, block, odt,
               out.data_ptr(), _handle(stream, dev), tile)
    if foreign is not None:
        _hold(foreign, dy, w, sorted_ids, expert_of_block, num_post_pad, out)
    _raise(rc)
    return out


def grouped_gemm_dw(dy, x, E: int, sorted_ids, expert_of_block, num_post_pad, k: int, block: int, *,
                    tokens: Optional[int] = None, out_dtype=None, out=None, stream=None):
    """Gradient of grouped_gemm's w (moe_grouped_gemm_dw): dw[e] = dy[rows of e]^T .
    x[row(r)], zeros for an expert without a route.

    dy: [max_rows, N]; x and `tokens` as for grouped_gemm; E: the experts.  Returns dw
    [E, N, K] of dy's type (default) or float32; equal inputs give equal bits."""
    dt, dev, index = _first(dy, 2, "dy")
    _matrix(x, 2, "x", index, dy.dtype)
    N, K, E = dy.shape[1], x.shape[1], int(E)
    _no_grad("grouped_gemm_dw", dy, x)
    M = x.shape[0] if tokens is None else int(tokens)
    rows, blocks = _sizes(M, E, k, block)
    if dy.shape[0] < rows or (tokens is not None and x.shape[0] < rows):
        raise ValueError(f"rows in sorted order must be at least {rows}")
    _metadata(sorted_ids, expert_of_block, num_post_pad, rows, blocks, dev, index)
    foreign = None if stream is None else _foreign(stream, dev)
    out_dtype = out_dtype or (dy.dtype if out is None else out.dtype)
    odt = dt if out_dtype == dy.dtype else _code(out_dtype, "out", True)
    out = _output(out, (E, N, K), out_dtype, dev, foreign)
    rc = _call(dev, lib().moe_grouped_gemm_dw, dy.data_ptr(), x.data_ptr(), dt, sorted_ids.data_ptr(),
               expert_of_block.data_ptr(), num_post_pad.data_ptr(), M, k, E, K, N, block,
               MRS_X_TOKENS if tokens is None else MRS_X_SORTED, odt, out.data_ptr(),
               _handle(stream, dev))
    if foreign is not None:
        _hold(foreign, dy, x, sorted_ids, expert_of_block, num_post_pad, out)
    _raise(rc)
    return out


def _vector(t, index: int, dtype, n: int, name: str, dev):
    """t is a contiguous tensor of dtype with at least n values on GPU `index`."""
    if not (_is(t, index, dtype) and t.numel() >= n):
        _check_tensor(t, dev, dtype, n, name)


def swiglu(a, num_post_pad=None, *, out=None, stream=None):
    """Gated activation (moe_swiglu): h[r, i] = silu(a[r, i]) * a[r, I + i].

    a: [rows, 2 I] bfloat16 or float16.  num_post_pad: int32 [1] on the device, the
    rows to take (the others of h are left as they were); by default all."""
    dt, dev, index = _first(a, 2, "a")
    rows, I2 = a.shape
    if I2 % 2 or I2 == 0:
        raise ValueError("a must have an even number of columns")
    _no_grad("swiglu", a)
    if num_post_pad is not None:
        _vector(num_post_pad, index, torch.int32, 1, "num_post_pad", dev)
    foreign = None if stream is None else _foreign(stream, dev)
    out = _output(out, (rows, I2 // 2), a.dtype, dev, foreign)
    rc = _call(dev, lib().moe_swiglu, a.data_ptr(), dt, _ptr(num_post_pad), rows, I2 // 2, out.data_ptr(),
               _handle(stream, dev))
    if foreign is not None:
        _hold(foreign, a, num_post_pad, out)
    _raise(rc)
    return out


def swiglu_backward(a, dh, num_post_pad=None, *, out=None, stream=None):
    """Gradient of swiglu's a (moe_swiglu_backward) from dh [rows, I]; `out` may be a."""
    dt, dev, index = _first(a, 2, "a")
    rows, I2 = a.shape
    if I2 % 2 or I2 == 0:
        raise ValueError("a must have an even number of columns")
    _matrix(dh, 2, "dh", index, a.dtype)
    if dh.shape != (rows, I2 // 2):
        raise ValueError(f"dh must have shape {(rows, I2 // 2)}")
    _no_grad("swiglu_backward", a, dh)
    if num_post_pad is not None:
        _vector(num_post_pad, index, torch.int32, 1, "num_post_pad", dev)
    foreign = None if stream is None else _foreign(stream, dev)
    out = _output(out, (rows, I2), a.dtype, dev, foreign)
    rc = _call(dev, lib().moe_swiglu_backward, a.data_ptr(), dh.data_ptr(), dt, _ptr(num_post_pad), rows, I2 // 2,
               out.data_ptr(), _handle(stream, dev))
    if foreign is not None:
        _hold(foreign, a, dh, num_post_pad, out)
    _raise(rc)
    return out


def slot_rows(sorted_ids, num_post_pad, tokens: int, k: int, *, out=None, stream=None):
    """Sorted row of every slot (moe_slot_rows): int32 [M, k], -1 for a dropped route."""
    if not isinstance(sorted_ids, torch.Tensor) or not sorted_ids.is_cuda:
        raise ValueError("sorted_ids must be a GPU tensor")
    dev, index, M = sorted_ids.device, sorted_ids.get_device(), int(tokens)
    _vector(sorted_ids, index, torch.int32, 0, "sorted_ids", dev)
    _vector(num_post_pad, index, torch.int32, 1, "num_post_pad", dev)
    if M < 0 or k < 1:
        raise ValueError("tokens must not be negative and k at least 1")
    foreign = None if stream is None else _foreign(stream, dev)
    out = _output(out, (M, k), torch.int32, dev, foreign)
    rc = _call(dev, lib().moe_slot_rows, sorted_ids.data_ptr(), num_post_pad.data_ptr(), sorted_ids.numel(), M, k,
               out.data_ptr(), _handle(stream, dev))
    if foreign is not None:
        _hold(foreign, sorted_ids, num_post_pad, out)
    _raise(rc)
    return out


def _check_weights(weights, M: int, k: int, dev, index: int):
    if weights is not None:
        _vector(weights, index, torch.float32, M * k, "weights", dev)
        if weights.shape != (M, k):
            raise ValueError(f"weights must have shape ({M}, {k})")


def combine(y, rows, weights=None, *, out_dtype=None, out=None, stream=None):
    """Mix of the picks' rows (moe_combine): out[t] = sum_j weights[t, j] * y[rows[t, j]].

    y: [R, N] bfloat16 or float16.  rows: int32 [M, k] (slot_rows; a row outside [0, R)
    adds nothing), or an integer k for y in slot order.  weights: float32 [M, k], by
    default ones.  Returns [M, N] of y's type (default) or float32."""
    dt, dev, index = _first(y, 2, "y")
    R, N = y.shape
    if isinstance(rows, int):
        k, rows = rows, None
        if k < 1 or R % k:
            raise ValueError("y must hold k rows for every token")
        M = R // k
    else:
        _matrix(rows, 2, "rows", index, torch.int32)
        M, k = rows.shape
    _check_weights(weights, M, k, dev, index)
    _no_grad("combine", y, weights)
    foreign = None if stream is None else _foreign(stream, dev)
    out_dtype = out_dtype or (y.dtype if out is None else out.dtype)
    odt = dt if out_dtype == y.dtype else _code(out_dtype, "out", True)
    out = _output(out, (M, N), out_dtype, dev, foreign)
    rc = _call(dev, lib().moe_combine, y.data_ptr(), dt, _ptr(rows), _ptr(weights), R, M, k, N, odt, out.data_ptr(),
               _handle(stream, dev))
    if foreign is not None:
        _hold(foreign, y, rows, weights, out)
    _raise(rc)
    return out


def combine_backward(dout, rows, sorted_ids, num_post_pad, *, weights=None, y=None, out=None, stream=None):
    """Gradients of combine (moe_combine_backward): dy[r] = weights[s] * dout[s // k] of
    the slot s = sorted_ids[r], zeros in padding rows, and, when y (what combine was
    given) is, the weights' gradient [M, k] float32.

    dout: [M, N] bfloat16 or float16; rows: slot_rows of this metadata.  Returns dy
    [rows of y, or of sorted_ids; N], or (dy, dweights); rows of dy at or past
    num_post_pad are left as they were."""
    dt, dev, index = _first(dout, 2, "dout")
    M, N = dout.shape
    _matrix(rows, 2, "rows", index, torch.int32)
    if rows.shape[0] != M:
        raise ValueError(f"rows must have shape ({M}, k)")
    k = rows.shape[1]
    _check_weights(weights, M, k, dev, index)
    R = sorted_ids.numel() if y is None else y.shape[0]
    if y is not None:
        _matrix(y, 2, "y", index, dout.dtype)
        if y.shape[1] != N:
            raise ValueError("y and dout disagree on N")
    _vector(sorted_ids, index, torch.int32, R, "sorted_ids", dev)
    _vector(num_post_pad, index, torch.int32, 1, "num_post_pad", dev)
    _no_grad("combine_backward", dout, weights, y)
    foreign = None if stream is None else _foreign(stream, dev)
    out = _output(out, (R, N), dout.dtype, dev, foreign)
    dv = None if y is None else _output(None, (M, k), torch.float32, dev, foreign)
    rc = _call(dev, lib().moe_combine_backward, dout.data_ptr(), _ptr(y), dt, rows.data_ptr(), sorted_ids.data_ptr(),
               num_post_pad.data_ptr(), _ptr(weights), R, M, k, N, out.data_ptr(), _ptr(dv),
               _handle(stream, dev))
    if foreign is not None:
        _hold(foreign, dout, y, rows, sorted_ids, num_post_pad, weights, out, dv)
    _raise(rc)
    return out if dv is None else (out, dv)


def _holds_experts(route, E: int, block: int) -> bool:
    """Whether the weights of E experts are known to hold every expert of the route; one
    that is known to be of more experts or of another block is refused."""
    experts, made_for = getattr(route, "experts", None), getattr(route, "block", None)
    if experts is not None and experts > E:
        raise ValueError(f"the route is of {experts} experts, w_up and w_down hold {E}")
    if made_for is not None and made_for != block:
        raise ValueError(f"the route was made for blocks of {made_for}, not {block}")
    if experts is not None:
        return True
    M, k = route.weights.shape
    rows, blocks = _sizes(M, E, k, block)  # they grow with the experts up to M k
    return M * k > E and (route.sorted_ids.numel(), route.expert_of_block.numel()) == (rows, blocks)


def _rows_of_nan(rows: int, columns: int, like):
    """Rows for a product that may leave some out, where any are asked for."""
    return torch.full((rows, columns), float("nan"), dtype=like.dtype, device=like.device) if rows else None


@functools.lru_cache(maxsize=1)
def _experts_function():
    class Experts(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w_up, w_down, weights, sorted_ids, expert_of_block, num_post_pad, block, whole):
            meta = (sorted_ids, expert_of_block, num_post_pad)
            M, k = weights.shape
            # as many as M k routes to any number of experts may take
            fill = 0 if whole else max(min(sorted_ids.numel(), M * k * block), 1)
            a = grouped_gemm(x, w_up, *meta, k, block, out=_rows_of_nan(fill, w_up.shape[1], x))
            h = swiglu(a, num_post_pad)
            y = grouped_gemm(h, w_down, *meta, k, block, tokens=M, out=_rows_of_nan(fill, w_down.shape[1], x))
            rows = slot_rows(sorted_ids, num_post_pad, M, k)
            ctx.save_for_backward(x, w_up, w_down, weights, a, h, y, rows, *meta)
            ctx.block, ctx.fill = block, fill
            return combine(y, rows, weights)

        @staticmethod
        @once_differentiable
        def backward(ctx, dout):
            x, w_up, w_down, weights, a, h, y, rows, *meta = ctx.saved_tensors
            sorted_ids, _, num_post_pad = meta
            (M, k), block, E = weights.shape, ctx.block, w_up.shape[0]
            need_x, need_up, need_down, need_v = ctx.needs_input_grad[:4]
            dy = combine_backward(dout.contiguous(), rows, sorted_ids, num_post_pad, weights=weights,
                                  y=y if need_v else None)
            dy, dv = dy if need_v else (dy, None)
            dx = d_up = d_down = None
            if need_down:
                d_down = grouped_gemm_dw(dy, h, E, *meta, k, block, tokens=M)
            if need_x or need_up:
                dh = grouped_gemm_dx(dy, w_down, *meta, M, k, block, out=_rows_of_nan(ctx.fill, w_down.shape[2], x))
                da = swiglu_backward(a, dh, num_post_pad)
                if need_up:
                    d_up = grouped_gemm_dw(da, x, E, *meta, k, block)
                if need_x:  # of 16-bit rows, which combine takes: each pick's is rounded before their FP32 sum
                    dx = grouped_gemm_dx(da, w_up, *meta, M, k, block, out=_rows_of_nan(ctx.fill, w_up.shape[2], x))
                    dx = combine(dx, rows)
            return dx, d_up, d_down, dv, None, None, None, None, None

    return Experts


def experts_train(x, w_up, w_down, route, block: int):
    """The experts of a routed layer under autograd: out[t] = sum over t's picks of
    weight * w_down[e] . (silu(gate) * up) with (gate, up) = w_up[e] . x[t].

    x: [M, H] bfloat16 or float16; w_up: [E, 2 I, H] (the gates' rows first) and w_down:
    [E, H, I] of x's type; route: what route_sort, or route_sort_train (whose weights
    pass the gradient on to the logits), returned for `block`.  Returns [M, H] with
    gradients to x, both weights and route.weights.  A route of more experts than the
    weights hold, or of another block, is refused; of one made by hand, whose sizes do
    not tell, tokens with a pick of an expert past the last get NaN, and so do their
    gradients.  To capture a training step in a graph call the entry points themselves,
    as for route_sort_train."""
    _, _, index = _first(x, 2, "x")
    _matrix(w_up, 3, "w_up", index, x.dtype)
    _matrix(w_down, 3, "w_down", index, x.dtype)
    _matrix(route.weights, 2, "route.weights", index, torch.float32)
    E, two, H = w_up.shape
    if x.shape[1] != H or two % 2 or tuple(w_down.shape) != (E, H, two // 2) or route.weights.shape[0] != x.shape[0]:
        raise ValueError("w_up must be [E, 2 I, H], w_down [E, H, I] and route.weights [M, k] for x [M, H]")
    meta = (route.sorted_ids, route.expert_of_block, route.num_post_pad)
    _metadata(*meta, *_sizes(x.shape[0], E, route.weights.shape[1], block), x.device, index)
    whole = _holds_experts(route, E, block)
    return _experts_function().apply(x, w_up, w_down, route.weights, *meta, block, whole)


class Int4(NamedTuple):
    """int4 rows (include/moe_int4.h): K columns padded with zeros to Kp, a multiple of
    128, in groups that share a scale; weight = scale * (code - 8)."""
    codes: "torch.Tensor"   # uint8 [..., Kp / 2], two codes a byte, the even column in the low half
    scales: "torch.Tensor"  # bfloat16 or float16 [..., Kp / group]


def _group_of(q, index: int, dims: int, name: str):
    """q holds contiguous int4 rows with `dims` dimensions on GPU `index`; returns the group
    and the codes' shape."""
    codes, scales = q if isinstance(q, Int4) else (None, None)
    if not (_is(codes, index, torch.uint8) and isinstance(scales, torch.Tensor) and scales.get_device() == index
            and scales.is_contiguous()):
        raise ValueError(f"{name} must be an Int4 of contiguous tensors, uint8 codes and scales, on GPU {index}")
    shape, (*same, n) = codes.shape, scales.shape
    Kp = shape[-1] * 2
    if len(shape) != dims or [*shape[:-1]] != same or Kp == 0 or Kp % 128 or n == 0 or Kp % n or \
            Kp // n not in (32, 64, 128):
        raise ValueError(f"{name}: codes [..., Kp / 2] and scales [..., Kp / group] of the same rows with {dims} "
                         "dimensions, Kp a multiple of 128, group 32, 64 or 128")
    return Kp // n, shape


def _new_int4(lead, Kp: int, group: int, u8, dtype, dev) -> Int4:
    return Int4(_empty((*lead, Kp // 2), u8, dev), _empty((*lead, Kp // group), dtype, dev))


def int4_quantize(w, group: int = 128, *, scale_dtype=None, out: Optional[Int4] = None, stream=None) -> Int4:
    """Rows of w to int4 rows (moe_int4_quantize).

    w: float32, bfloat16 or float16 GPU tensor [..., K], 1 <= K <= 262144, rows of one
    stride as for mxfp4_quantize.  group: 32, 64 or 128 columns to a scale.  scale_dtype:
    bfloat16 or float16, the type of the x that the weights will meet (default: w's, or
    bfloat16 for float32 weights)."""
    if not (isinstance(w, torch.Tensor) and w.is_cuda and w.dim() >= 1):
        raise ValueError("w must be a GPU tensor of at least one dimension")
    dt, dev = _code(w.dtype, "w", True), w.device
    *lead, K = w.shape
    if not 1 <= K <= 262144:
        raise ValueError("the last dimension must hold 1 to 262144 values")
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    rows, row_stride = w.numel() // K, _row_stride(w, K)
    if scale_dtype is None:
        scale_dtype = (torch.bfloat16 if w.dtype == torch.float32 else w.dtype) if out is None else out.scales.dtype
    sdt = _code(scale_dtype, "scale")
    Kp = (K + 127) // 128 * 128
    foreign = None if stream is None else _foreign(stream, dev)
    if out is None:
        new = lead, Kp, group, torch.uint8, scale_dtype, dev
        out = _new_int4(*new) if foreign is None else _allocate(foreign, dev, _new_int4, *new)
    elif _group_of(out, w.get_device(), w.dim(), "out")[0] != group or out.codes.shape != (*lead, Kp // 2) or \
            out.scales.dtype != scale_dtype:
        raise ValueError(f"out must hold codes {(*lead, Kp // 2)} and {scale_dtype} scales {(*lead, Kp // group)}")
    rc = _call(dev, lib().moe_int4_quantize, w.data_ptr(), dt, rows, K, row_stride, group, sdt, out.codes.data_ptr(),
               out.scales.data_ptr(), _handle(stream, dev))
    if foreign is not None:
        _hold(foreign, w, *out)
    _raise(rc)
    return out


def int4_matvec(x, w: Int4, ids, *, gated: bool = False, weights=None, out=None, stream=None):
    """Matrix-vector products of routed tokens with 4-bit weights (moe_int4_matvec),
    for few tokens: p[t, j] = w[ids[t, j]] . x[t] (or x[t, j]).

    x: [M, K], or [M, k, K] with a row for every pick, bfloat16 or float16.  w: int4 rows
    [E, N] of K columns, scales of x's type.  ids: int32 [M, k]; a pick outside [0, E)
    gives zeros.  Returns p [M, k, N]; with `gated` [M, k, N / 2], silu(p[..., :N / 2]) *
    p[..., N / 2:]; with weights (float32 [M, k]) their sum over the picks [M, N]."""
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.is_contiguous()):
        raise ValueError("x must be a contiguous [M, K] or [M, k, K] GPU tensor")
    xdt, dev, index, xshape = x.dtype, x.device, x.get_device(), x.shape
    dt = _code(xdt, "x")
    _matrix(ids, 2, "ids", index, torch.int32)
    M, k = ids.shape
    group, (E, N, half) = _group_of(w, index, 3, "w")
    if w.scales.dtype != xdt:
        raise ValueError("w's scales must have x's type")
    K, slots = xshape[-1], len(xshape) == 3
    if xshape[:-1] != ((M, k) if slots else (M,)) or (K + 127) // 128 * 64 != half:
        raise ValueError(f"x must have shape ({M}, K) or ({M}, {k}, K), K columns of w")
    if gated and (weights is not None or N % 2):
        raise ValueError("gated results need an even N and take no weights")
    if weights is not None:
        _check_weights(weights, M, k, dev, index)
    if x.requires_grad or w.scales.requires_grad or (weights is not None and weights.requires_grad):
        _no_grad("int4_matvec", x, w.scales, weights)
    foreign = None if stream is None else _foreign(stream, dev)
    out = _output(out, (M, N) if weights is not None else (M, k, N // 2 if gated else N), xdt, dev, foreign)
    mode = MRS_INT4_GATED if gated else MRS_INT4_PLAIN if weights is None else MRS_INT4_SUM
    rc = _call(dev, lib().moe_int4_matvec, x.data_ptr(), dt, w.codes.data_ptr(), w.scales.data_ptr(), ids.data_ptr(),
               _ptr(weights), M, k, E, K, N, group, int(slots), mode, out.data_ptr(),
               _handle(stream, dev))
    if foreign is not None:
        _hold(foreign, x, *w, ids, weights, out)
    _raise(rc)
    return out
