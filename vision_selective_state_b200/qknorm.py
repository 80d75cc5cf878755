"""Norm of every query and key head with the position rotation in the same pass: binding of the
vscan_qknorm_* entry points.

    q, k     : [batch, tokens, heads, dim], torch.float32 or torch.bfloat16; token and image
               strides are free but not 0, the heads of one token are contiguous
    wq, wk   : [dim] float32, optional
    inv_freq : [pairs] float32, optional: channels p and p + pairs of a head are rotated by
               position * inv_freq[p]
    positions: int32 [tokens], [tokens, axes] or, one set per image, [batch, tokens(, axes)]
               (a shape that fits two of them is read as the first);
               with two axes (grid row, grid column) the first half of the pairs turns by the
               first, the second half by the second

stream is as in the delta rule's calls: the call runs, allocates and clears there, and waits for no
other stream.
"""
import ctypes

import torch

from . import _abi
from ._abi import VscanQkNormGrads, check
from .delta import check_dense, check_tensor, device_index, fresh, hand_over, head_strides, launching

NORMS = {"l2": 0, "rms": 1}


def _marshal(index, code, q, k, wq, wk, yq, yk, norm, eps, inv_freq, positions):
    """Packed vscan_qknorm_args."""
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {sorted(NORMS)}")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k are [batch, tokens, heads, dim]")
    dtype = q.dtype
    batch, tokens, hq, d = q.shape
    hk = k.shape[2]
    check_tensor("k", k, (batch, tokens, hk, d), dtype, index)
    check_tensor("yq (dyq)", yq, q.shape, dtype, index)
    check_tensor("yk (dyk)", yk, k.shape, dtype, index)
    if wq is not None:
        check_dense("wq", wq, (d,), torch.float32, index)
    if wk is not None:
        check_dense("wk", wk, (d,), torch.float32, index)
    pairs, axes, per_image = 0, 1, 0
    if (inv_freq is None) != (positions is None):
        raise ValueError("inv_freq and positions belong together")
    if inv_freq is not None:
        pairs = inv_freq.numel()
        check_dense("inv_freq", inv_freq, (pairs,), torch.float32, index)
        shape = positions.shape
        for lead in ((tokens,), (batch, tokens)):
            if shape == lead or (shape[:-1] == lead and shape[-1] in (1, 2)):
                axes, per_image = (1 if shape == lead else shape[-1]), len(lead) - 1
                break
        else:
            raise ValueError(f"positions shape {tuple(shape)} is not [tokens(, axes)] or [batch, tokens(, axes)]")
        check_dense("positions", positions, shape, torch.int32, index)
    return _abi.qknorm_forward.pack(
        batch, tokens, hq, hk, d, pairs, axes, code, NORMS[norm], eps,
        q.data_ptr(), k.data_ptr(), yq.data_ptr(), yk.data_ptr(), 0 if wq is None else wq.data_ptr(),
        0 if wk is None else wk.data_ptr(), inv_freq.data_ptr() if pairs else 0, positions.data_ptr() if pairs else 0,
        per_image, 0,
        *head_strides("q", q, q.is_contiguous()), *head_strides("k", k, k.is_contiguous()),
        *head_strides("yq", yq, yq.is_contiguous()), *head_strides("yk", yk, yk.is_contiguous()))


def qk_norm(q, k, wq=None, wk=None, *, norm="rms", eps=1e-6, inv_freq=None, positions=None, out=None, stream=None):
    """Normalised ("l2": unit length, "rms": unit mean square), weighted and rotated (yq, yk)
    (vscan_qknorm_forward). out: a pair of tensors to write to, each either its own input (in
    place) or memory that overlaps no input."""
    index, code = device_index(q)
    with launching(stream, index):
        if out is None:
            out = (fresh(q), fresh(k))
        args = _marshal(index, code, q, k, wq, wk, *out, norm, eps, inv_freq, positions)
        check(_abi.qknorm_forward.fn(args, torch._C._cuda_getCurrentRawStream(index)))
    if stream is not None:
        hand_over(stream, index, *out)
    return tuple(out)


def qk_norm_backward(q, k, wq=None, wk=None, *, dyq, dyk, norm="rms", eps=1e-6, inv_freq=None, positions=None,
                     want=("dq", "dk", "dwq", "dwk"), stream=None):
    """Gradients of qk_norm (vscan_qknorm_backward) in a dict: dq and dk (dense, in the dtype of
    q) and, where there is a weight, dwq and dwk (float32, summed over the tokens in a fixed
    order). dyq, dyk: dL/dyq and dL/dyk in the dtype of q, with free strides. `want` limits
    the keys computed."""
    like = {"dq": q, "dk": k, "dwq": wq, "dwk": wk}
    if not set(want) <= set(like):
        raise ValueError(f"want holds unknown gradients {sorted(set(want) - set(like))}")
    index, code = device_index(q)
    with launching(stream, index):
        args = _marshal(index, code, q, k, wq, wk, dyq, dyk, norm, eps, inv_freq, positions)
        grads, out = VscanQkNormGrads(), {}
        grads.dyq, grads.dyk = dyq.data_ptr(), dyk.data_ptr()
        for name in want:
            t = like[name]
            if t is not None:
                out[name] = fresh(t)
                setattr(grads, name, out[name].data_ptr())
        if "dwq" in out or "dwk" in out:
            need = ctypes.c_uint64()
            check(_abi.qknorm_backward_workspace_size.fn(args, ctypes.byref(need)))
            workspace = q.new_empty(need.value, dtype=torch.uint8)
            grads.workspace, grads.workspace_bytes = workspace.data_ptr(), need.value
        check(_abi.qknorm_backward.fn(args, ctypes.byref(grads), torch._C._cuda_getCurrentRawStream(index)))
    if stream is not None:
        hand_over(stream, index, *out.values())
    return out
