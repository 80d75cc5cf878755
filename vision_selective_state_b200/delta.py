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
are free (slices of a wider projection output); the heads of one token are contiguous. As in
the rest of the package, the binding only marshals tensors; the arithmetic runs in libvscan.so.
"""
import contextlib
import ctypes

import torch

from ._abi import BF16, F32, ROUTES, VscanDeltaArgs, VscanDeltaGrads, check, lib

_CODES = {torch.float32: F32, torch.bfloat16: BF16}


def on_device(device):
    """Context in which the runtime's current device is the tensors' own."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def stream_handle(stream, device, *scratch):
    """The launch stream's handle. Tensors made here for a call on a stream other than the
    current one are marked as used there, so that their memory is not handed out again early."""
    current = torch.cuda.current_stream(device)
    if stream is None:
        return current.cuda_stream
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    if stream != current:
        for t in scratch:
            if t is not None:
                t.record_stream(stream)
    return stream.cuda_stream


def check_tensor(name, t, shape, dtype, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")


def check_dense(name, t, shape, dtype, device):
    check_tensor(name, t, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def head_strides(name, t):
    """(token, image) strides of a [batch, tokens, heads, dim] tensor with contiguous heads."""
    b, n, h, d = t.shape
    sb, sn, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"the heads of one token of {name} must be contiguous")
    # a size-1 axis has no meaningful stride: take the dense value
    tok = sn if n > 1 else h * d
    return tok, (sb if b > 1 else n * tok)


def _row_strides(name, t):
    """(token, image) strides of a [batch, tokens, heads] tensor with contiguous heads."""
    b, n, h = t.shape
    if t.stride(2) != 1 and h > 1:
        raise ValueError(f"the heads of one token of {name} must be contiguous")
    tok = t.stride(1) if n > 1 else h
    return tok, (t.stride(0) if b > 1 else n * tok)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _marshal(q, k, v, a, b, A, bias, y, *, route, direction, seq_offsets, scale, beta_scale, initial_state,
             final_state):
    if q.dtype not in _CODES:
        raise TypeError(f"unsupported dtype {q.dtype} (float32 or bfloat16)")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and k are [batch, tokens, heads_k, dim_k], v is [batch, tokens, heads_v, dim_v]")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device")
    batch, tokens, hk, dk = q.shape
    hv, dv = v.shape[2:]
    check_tensor("k", k, q.shape, q.dtype, dev)
    check_tensor("v", v, (batch, tokens, hv, dv), q.dtype, dev)
    check_tensor("a", a, (batch, tokens, hv), q.dtype, dev)
    check_tensor("b", b, (batch, tokens, hv), q.dtype, dev)
    check_tensor("y", y, v.shape, q.dtype, dev)
    check_dense("A", A, (hv,), torch.float32, dev)
    if bias is not None:
        check_dense("bias", bias, (hv,), torch.float32, dev)
    rows = batch
    if seq_offsets is not None:
        if batch != 1:
            raise ValueError("packed sequences have one row of tokens: batch must be 1")
        if seq_offsets.dim() != 1 or seq_offsets.numel() < 1:
            raise ValueError("seq_offsets must hold one more element than there are sequences")
        check_dense("seq_offsets", seq_offsets, seq_offsets.shape, torch.int32, dev)
        rows = seq_offsets.numel() - 1
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is not None:
            check_dense(name, t, (rows, hv, dk, dv), torch.float32, dev)
    return VscanDeltaArgs(
        rows, tokens, hk, hv, dk, dv, _CODES[q.dtype], int(direction),
        q.data_ptr(), k.data_ptr(), v.data_ptr(), a.data_ptr(), b.data_ptr(), y.data_ptr(), A.data_ptr(), _ptr(bias),
        _ptr(initial_state), _ptr(final_state), _ptr(seq_offsets),
        dk ** -0.5 if scale is None else float(scale), float(beta_scale),
        *head_strides("q", q), *head_strides("k", k), *head_strides("v", v), *_row_strides("a", a),
        *_row_strides("b", b), *head_strides("y", y))


def _route_handle(route):
    return None if route is None else route.handle


def _partial(route, seq_offsets):
    """Whether a call may leave rows of its outputs unwritten."""
    return seq_offsets is not None or (route is not None and route.kind == ROUTES["atrous2"])


def _state_rows(q, seq_offsets):
    return q.shape[0] if seq_offsets is None else seq_offsets.numel() - 1


def delta_forward(q, k, v, a, b, A, bias=None, *, route=None, direction=0, seq_offsets=None, scale=None,
                  beta_scale=1.0, initial_state=None, final_state=False, out=None, workspace=None, stream=None):
    """Gated delta rule over every token (vscan_delta_forward). Returns y, or (y, final state).

    route, direction: visit the tokens in the order of one direction of a BIDIR, CROSS4 or
    ATROUS2 Route (an ATROUS2 direction writes its own group's tokens only); without a route,
    first to last. seq_offsets: int32 [n + 1] on the device for n packed sequences in one row
    of tokens (batch 1); rows outside every sequence are left as they are. Rows that a call
    leaves are 0 in an output made here. scale: dim_k ** -0.5 if None. final_state: True, or a tensor to write
    the state after the last token to (initial_state itself is allowed).
    """
    if out is None:
        out = (torch.zeros if _partial(route, seq_offsets) else torch.empty)(v.shape, dtype=v.dtype, device=v.device)
    if final_state is True:
        final_state = torch.empty((_state_rows(q, seq_offsets), v.shape[2], q.shape[3], v.shape[3]),
                                  dtype=torch.float32, device=q.device)
    elif final_state is False:
        final_state = None
    args = _marshal(q, k, v, a, b, A, bias, out, route=route, direction=direction, seq_offsets=seq_offsets, scale=scale,
                    beta_scale=beta_scale, initial_state=initial_state, final_state=final_state)
    handle, ref = _route_handle(route), ctypes.byref(args)
    if workspace is None:
        need = ctypes.c_uint64()
        check(lib.vscan_delta_workspace_size(handle, ref, ctypes.byref(need)))
        workspace = torch.empty(need.value, dtype=torch.uint8, device=q.device)
    args.workspace, args.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    with on_device(q.device):
        check(lib.vscan_delta_forward(handle, ref, stream_handle(stream, q.device, out, final_state, workspace)))
    return out if final_state is None else (out, final_state)


GRADIENTS = ("dq", "dk", "dv", "da", "db", "dA", "dbias", "d_initial_state")


def delta_backward(q, k, v, a, b, A, bias=None, *, dy, route=None, direction=0, seq_offsets=None, scale=None,
                   beta_scale=1.0, initial_state=None, d_final_state=None, want=None, workspace=None, stream=None):
    """Gradients of delta_forward (vscan_delta_backward) in a dict, from its arguments, dy = dL/dy
    and d_final_state = dL/d(final state).

    Keys: dq, dk, dv, da, db (dense, in the dtype of q), dA, dbias and, with initial_state,
    d_initial_state (float32). `want` limits the keys computed. Tokens that no step visits get
    zeros. Equal calls give equal bits.
    """
    args = _marshal(q, k, v, a, b, A, bias, dy, route=route, direction=direction, seq_offsets=seq_offsets, scale=scale,
                    beta_scale=beta_scale, initial_state=initial_state, final_state=None)
    dev, grads, out = q.device, VscanDeltaGrads(), {}
    like = {"dq": q, "dk": k, "dv": v, "da": a, "db": b, "dA": A, "dbias": A, "d_initial_state": initial_state}
    if want is not None and not set(want) <= set(GRADIENTS):
        raise ValueError(f"want holds unknown gradients {sorted(set(want) - set(GRADIENTS))}")
    for name in GRADIENTS if want is None else want:
        t = like[name]
        if t is not None:
            out[name] = torch.empty(t.shape, dtype=t.dtype, device=dev)
            setattr(grads, name, out[name].data_ptr())
    if d_final_state is not None:
        check_dense("d_final_state", d_final_state, (_state_rows(q, seq_offsets), *v.shape[2:3], q.shape[3], v.shape[3]),
                    torch.float32, dev)
        grads.d_final_state = d_final_state.data_ptr()
    handle, ref = _route_handle(route), ctypes.byref(args)
    if workspace is None:
        need = ctypes.c_uint64()
        check(lib.vscan_delta_backward_workspace_size(handle, ref, ctypes.byref(need)))
        workspace = torch.empty(need.value, dtype=torch.uint8, device=dev)
    grads.workspace, grads.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    with on_device(dev):
        check(lib.vscan_delta_backward(handle, ref, dy.data_ptr(), ctypes.byref(grads),
                                       stream_handle(stream, dev, workspace, *out.values())))
    return out


def delta_step(q, k, v, a, b, A, bias=None, *, state, state_out=None, scale=None, beta_scale=1.0, out=None,
               stream=None):
    """One token of each of a batch of sequences (vscan_delta_step). Returns (y, new state).

    q, k: [batch, heads_k, dim_k]; v, y: [batch, heads_v, dim_v]; a, b: [batch, heads_v].
    The new state goes to state_out, or in place to state.
    """
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    if state_out is None:
        state_out = state
    args = _marshal(q.unsqueeze(1), k.unsqueeze(1), v.unsqueeze(1), a.unsqueeze(1), b.unsqueeze(1), A, bias,
                    out.unsqueeze(1), route=None, direction=0, seq_offsets=None, scale=scale, beta_scale=beta_scale,
                    initial_state=state, final_state=state_out)
    with on_device(q.device):
        check(lib.vscan_delta_step(ctypes.byref(args), stream_handle(stream, q.device, out, state_out)))
    return out, state_out
