"""Gated delta rule: binding of the vscan_delta_* entry points.

Per value head, with log decay g = A softplus(a + bias) and write strength
beta = beta_scale sigmoid(b),

    S_t = e^g S_{t-1} + beta k_t (v_t - e^g S_{t-1}^T k_t)^T        [dim_k, dim_v]
    y_t = scale S_t^T q_t

    q, k    : [batch, tokens, heads_k, dim_k]   each head shared by heads_v / heads_k value heads
    v, y    : [batch, tokens, heads_v, dim_v]
    a, b    : [batch, tokens, heads_v]          raw decay step and raw write strength
    A, bias : [heads_v] float32
    states  : [batch, heads_v, dim_k, dim_v] float32

q, k, v, a, b and y share one dtype: torch.float32 or torch.bfloat16. Token and image strides
are free (slices of a wider projection output) but not 0 (an expanded axis is refused); the
heads of one token are contiguous. As in
the rest of the package, the binding only marshals tensors; the arithmetic runs in libvscan.so.

A call runs on `stream`, or on the current one: its kernels, what it allocates and the rows that it
clears. It waits for no other stream: with `stream` given, the caller orders it behind the work that
makes its inputs, and what reads its results behind it.
"""
import contextlib
import ctypes

import torch

from . import _abi
from ._abi import BF16, F32, ROUTES, VscanDeltaGrads, check

CODES = {torch.float32: F32, torch.bfloat16: BF16}
_f32 = torch.float32
_here = contextlib.nullcontext()
_dense = (0,) * 12  # strides of six dense tensors
_pack = _abi.delta_forward.pack


def launching(stream, index):
    """Context of a call on the tensors' device and on `stream`, the current one if None. What a call
    allocates and clears belongs to the stream that its kernels run on: memory of the current one may
    still be read there, and a fill there comes at any time."""
    if stream is None:
        return _here if torch._C._cuda_getDevice() == index else torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{index}")
    return torch.cuda.stream(stream)


def hand_over(stream, index, *tensors):
    """A call's tensors are used on its stream and on the caller's: their memory is not handed out
    again before both have passed the point where the last reference is dropped."""
    here = torch.cuda.current_stream(index)
    if here.cuda_stream != stream.cuda_stream:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
                t.record_stream(here)


def check_tensor(name, t, shape, dtype, index):
    """Raise for a tensor that is not what a call takes."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")


def check_dense(name, t, shape, dtype, index):
    check_tensor(name, t, shape, dtype, index)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fits(dtype, index, *pairs):
    """Whether every (tensor, shape) has the dtype, device and shape asked for: one look at what
    check_tensor would refuse one by one. The smallest calls take less time on the device
    than their checks do here."""
    for t, shape in pairs:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
            return False
    return True


def device_index(q):
    """Index of the tensors' device, and the dtype's code."""
    code = CODES.get(q.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {q.dtype} (float32 or bfloat16)")
    index = q.get_device()
    if index < 0:
        raise ValueError("the tensors must be on a CUDA device")
    return index, code


def _spaced(name, t):
    """Refuse a broadcast axis: the ABI reads a stride of 0 as dense."""
    for size, stride in zip(t.shape[:2], t.stride()):
        if stride == 0 and size > 1:
            raise ValueError(f"{name} repeats one row (a stride of 0): make it contiguous")


def head_strides(name, t, dense):
    """(token, image) strides of a [batch, tokens, heads, dim] tensor with contiguous heads;
    a size-1 axis has no meaningful stride and takes the dense value (0)."""
    if dense:
        return 0, 0
    b, n, h, d = t.shape
    sb, sn, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"the heads of one token of {name} must be contiguous")
    _spaced(name, t)
    tok = sn if n > 1 else h * d
    return tok, (sb if b > 1 else n * tok)


def _row_strides(name, t, dense):
    """(token, image) strides of a [batch, tokens, heads] tensor with contiguous heads."""
    if dense:
        return 0, 0
    b, n, h = t.shape
    if t.stride(2) != 1 and h > 1:
        raise ValueError(f"the heads of one token of {name} must be contiguous")
    _spaced(name, t)
    tok = t.stride(1) if n > 1 else h
    return tok, (t.stride(0) if b > 1 else n * tok)


def _rows(q, v, seq_offsets):
    """Images, or packed sequences."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and k are [batch, tokens, heads_k, dim_k], v is [batch, tokens, heads_v, dim_v]")
    if seq_offsets is None:
        return q.shape[0]
    if q.shape[0] != 1:
        raise ValueError("packed sequences have one row of tokens: batch must be 1")
    if seq_offsets.dim() != 1 or seq_offsets.numel() < 1:
        raise ValueError("seq_offsets must hold one more element than there are sequences")
    return seq_offsets.numel() - 1


def _fields(index, code, rows, q, k, v, a, b, A, bias, y, direction, seq_offsets, scale, beta_scale, initial_state,
            final_state):
    """Fields of vscan_delta_args up to the strides."""
    dtype, shape = q.dtype, q.shape
    batch, tokens, hk, dk = shape
    hv, dv = v.shape[2:]
    heads = (batch, tokens, hv)
    check_tensor("k", k, shape, dtype, index)
    check_tensor("v", v, (batch, tokens, hv, dv), dtype, index)
    check_tensor("a", a, heads, dtype, index)
    check_tensor("b", b, heads, dtype, index)
    check_tensor("y (dy)", y, v.shape, dtype, index)
    check_dense("A", A, (hv,), torch.float32, index)
    if bias is not None:
        check_dense("bias", bias, (hv,), torch.float32, index)
    if seq_offsets is not None:
        check_dense("seq_offsets", seq_offsets, seq_offsets.shape, torch.int32, index)
    if initial_state is not None:
        check_dense("initial_state", initial_state, (rows, hv, dk, dv), torch.float32, index)
    if final_state is not None:
        check_dense("final_state", final_state, (rows, hv, dk, dv), torch.float32, index)
    return (
        rows, tokens, hk, hv, dk, dv, code, direction,
        q.data_ptr(), k.data_ptr(), v.data_ptr(), a.data_ptr(), b.data_ptr(), y.data_ptr(), A.data_ptr(),
        0 if bias is None else bias.data_ptr(), 0 if initial_state is None else initial_state.data_ptr(),
        0 if final_state is None else final_state.data_ptr(), 0 if seq_offsets is None else seq_offsets.data_ptr(),
        (dk and dk ** -0.5) if scale is None else scale, beta_scale,  # a width of 0 is refused by the library
        *head_strides("q", q, q.is_contiguous()), *head_strides("k", k, k.is_contiguous()),
        *head_strides("v", v, v.is_contiguous()), *_row_strides("a", a, a.is_contiguous()),
        *_row_strides("b", b, b.is_contiguous()), *head_strides("y", y, y.is_contiguous()))


def fresh(t):
    """An uninitialised dense tensor like t."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _status(status, index):
    if status is None:
        return 0
    if status.dtype is not torch.int32 or status.numel() < 1 or status.get_device() != index:
        raise TypeError(f"status must be an int32 tensor on cuda:{index}")
    return status.data_ptr()


def _route_handle(route):
    return None if route is None else route.handle


def _partial(route, seq_offsets):
    """Whether a call may leave rows of its outputs unwritten."""
    return seq_offsets is not None or (route is not None and route.kind == ROUTES["atrous2"])


def _state_shape(rows, q, v):
    return rows, v.shape[2], q.shape[3], v.shape[3]


def _scratch(given, query, handle, fields, q, index):
    """(workspace, its address, its bytes)."""
    if given is None:
        need = ctypes.c_uint64()
        check(query.fn(handle, _pack(*fields, 0, 0, 0), ctypes.byref(need)))
        given = q.new_empty(need.value, dtype=torch.uint8)
    elif given.get_device() != index or not given.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{index}")
    return given, given.data_ptr(), given.numel() * given.element_size()


def delta_forward(q, k, v, a, b, A, bias=None, *, route=None, direction=0, seq_offsets=None, scale=None,
                  beta_scale=1.0, initial_state=None, final_state=False, out=None, workspace=None, stream=None,
                  status=None):
    """Gated delta rule over every token (vscan_delta_forward). Returns y, or (y, final state).

    route, direction: visit the tokens in the order of one direction of a BIDIR, CROSS4 or
    ATROUS2 Route (an ATROUS2 direction writes its own group's tokens only); without a route,
    first to last. seq_offsets: int32 [n + 1] on the device for n packed sequences in one row
    of tokens (batch 1); rows outside every sequence are left as they are. Rows that a call
    leaves are 0 in an output made here; one given as `out` must not overlap the inputs. scale:
    dim_k ** -0.5 if None. final_state: True, or a tensor to write the state after the last token
    to (initial_state itself is allowed). status: an int32 device word, zeroed by the caller, that
    tells of an internal wait that gave up; decode it with status_from_device_word. Without one
    nothing tells such a call's invalid outputs from good ones.
    """
    index, code = device_index(q)
    rows = _rows(q, v, seq_offsets)
    with launching(stream, index):
        if out is None:
            out = v.new_zeros(v.shape) if _partial(route, seq_offsets) else fresh(v)
        if final_state is True:
            final_state = q.new_empty(_state_shape(rows, q, v), dtype=torch.float32)
        elif final_state is False:
            final_state = None
        fields = _fields(index, code, rows, q, k, v, a, b, A, bias, out, direction, seq_offsets, scale, beta_scale,
                         initial_state, final_state)
        handle = _route_handle(route)
        scratch, *where = _scratch(workspace, _abi.delta_workspace_size, handle, fields, q, index)
        args = _pack(*fields, *where, _status(status, index))
        check(_abi.delta_forward.fn(handle, args, torch._C._cuda_getCurrentRawStream(index)))
    if stream is not None:
        hand_over(stream, index, out, final_state, workspace)
    return out if final_state is None else (out, final_state)


GRADIENTS = ("dq", "dk", "dv", "da", "db", "dA", "dbias", "d_initial_state")


def delta_backward(q, k, v, a, b, A, bias=None, *, dy, route=None, direction=0, seq_offsets=None, scale=None,
                   beta_scale=1.0, initial_state=None, d_final_state=None, want=None, workspace=None, stream=None,
                   status=None):
    """Gradients of delta_forward (vscan_delta_backward) in a dict, from its arguments, dy = dL/dy
    and d_final_state = dL/d(final state).

    Keys: dq, dk, dv, da, db (dense, in the dtype of q), dA, dbias and, with initial_state,
    d_initial_state (float32). `want` limits the keys computed. Tokens that no step visits get
    zeros. Equal calls give equal bits. status: as in delta_forward.
    """
    if want is not None and not set(want) <= set(GRADIENTS):
        raise ValueError(f"want holds unknown gradients {sorted(set(want) - set(GRADIENTS))}")
    index, code = device_index(q)
    rows = _rows(q, v, seq_offsets)
    with launching(stream, index):
        fields = _fields(index, code, rows, q, k, v, a, b, A, bias, dy, direction, seq_offsets, scale, beta_scale,
                         initial_state, None)
        grads, out = VscanDeltaGrads(), {}
        like = {"dq": q, "dk": k, "dv": v, "da": a, "db": b, "dA": A, "dbias": A, "d_initial_state": initial_state}
        for name in GRADIENTS if want is None else want:
            t = like[name]
            if t is not None:
                out[name] = fresh(t)
                setattr(grads, name, out[name].data_ptr())
        if d_final_state is not None:
            check_dense("d_final_state", d_final_state, _state_shape(rows, q, v), torch.float32, index)
            grads.d_final_state = d_final_state.data_ptr()
        handle = _route_handle(route)
        scratch, grads.workspace, grads.workspace_bytes = _scratch(workspace, _abi.delta_backward_workspace_size, handle,
                                                                   fields, q, index)
        args = _pack(*fields, 0, 0, _status(status, index))
        check(_abi.delta_backward.fn(handle, args, dy.data_ptr(), ctypes.byref(grads),
                                     torch._C._cuda_getCurrentRawStream(index)))
    if stream is not None:
        hand_over(stream, index, workspace, *out.values())
    return out


def delta_step(q, k, v, a, b, A, bias=None, *, state, state_out=None, scale=None, beta_scale=1.0, out=None,
               stream=None):
    """One token of each of a batch of sequences (vscan_delta_step). Returns (y, new state).

    q, k: [batch, heads_k, dim_k]; v, y: [batch, heads_v, dim_v]; a, b: [batch, heads_v].
    The new state goes to state_out, or in place to state. `out` must not overlap the inputs.
    """
    index, code = device_index(q)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and k are [batch, heads_k, dim_k], v is [batch, heads_v, dim_v]")
    dtype, shape, wide = q.dtype, q.shape, v.shape
    batch, hk, dk = shape
    hv, dv = wide[1:]
    heads, table = (batch, hv), (batch, hv, dk, dv)
    if not fits(dtype, index, (k, shape), (v, (batch, hv, dv)), (a, heads), (b, heads)):
        check_tensor("k", k, shape, dtype, index)
        check_tensor("v", v, (batch, hv, dv), dtype, index)
        check_tensor("a", a, heads, dtype, index)
        check_tensor("b", b, heads, dtype, index)
    if out is not None:
        check_tensor("y", out, wide, dtype, index)
    if state_out is None:
        state_out = state
    shift = A if bias is None else bias
    if not (fits(_f32, index, (A, (hv,)), (shift, (hv,)), (state, table), (state_out, table)) and A.is_contiguous()
            and shift.is_contiguous() and state.is_contiguous() and state_out.is_contiguous()):
        check_dense("A", A, (hv,), _f32, index)
        check_dense("bias", shift, (hv,), _f32, index)
        check_dense("state", state, table, _f32, index)
        check_dense("state_out", state_out, table, _f32, index)
    with launching(stream, index):
        if out is None:
            out = fresh(v)
        if (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and a.is_contiguous() and b.is_contiguous()
                and out.is_contiguous()):
            strides = _dense
        else:
            strides = []
            for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b), ("y", out)):
                if t.is_contiguous():
                    strides += (0, 0)
                elif t.dim() == 3:
                    strides += (0, head_strides(name, t.unsqueeze(1), False)[1])
                else:
                    strides += (0, _row_strides(name, t.unsqueeze(1), False)[1])
        args = _pack(batch, 1, hk, hv, dk, dv, code, 0, q.data_ptr(), k.data_ptr(), v.data_ptr(), a.data_ptr(), b.data_ptr(),
                     out.data_ptr(), A.data_ptr(), 0 if bias is None else bias.data_ptr(), state.data_ptr(),
                     state_out.data_ptr(), 0, (dk and dk ** -0.5) if scale is None else scale, beta_scale, *strides, 0, 0, 0)
        check(_abi.delta_step.fn(args, torch._C._cuda_getCurrentRawStream(index)))
    if stream is not None:
        hand_over(stream, index, out, state_out)
    return out, state_out
