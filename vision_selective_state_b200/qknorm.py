"""Norm of every query and key head with the position rotation in the same pass: binding of the
vscan_qknorm_* entry points.

    q, k     : [batch, tokens, heads, dim], torch.float32 or torch.bfloat16; token and image
               strides are free, the heads of one token are contiguous
    wq, wk   : [dim] float32, optional
    inv_freq : [pairs] float32, optional: channels p and p + pairs of a head are rotated by
               position * inv_freq[p]
    positions: int32 [tokens], [tokens, axes] or, one set per image, [batch, tokens(, axes)];
               with two axes (grid row, grid column) the first half of the pairs turns by the
               first, the second half by the second
"""
import ctypes

import torch

from ._abi import VscanQkNormArgs, VscanQkNormGrads, check, lib
from .delta import _CODES, check_dense, check_tensor, head_strides, on_device, stream_handle

NORMS = {"l2": 0, "rms": 1}


def _marshal(q, k, wq, wk, yq, yk, norm, eps, inv_freq, positions):
    if q.dtype not in _CODES:
        raise TypeError(f"unsupported dtype {q.dtype} (float32 or bfloat16)")
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {sorted(NORMS)}")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k are [batch, tokens, heads, dim]")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device")
    batch, tokens, hq, d = q.shape
    hk = k.shape[2]
    check_tensor("k", k, (batch, tokens, hk, d), q.dtype, dev)
    for name, t in (("wq", wq), ("wk", wk)):
        if t is not None:
            check_dense(name, t, (d,), torch.float32, dev)
    pairs, axes, per_image = 0, 1, 0
    if (inv_freq is None) != (positions is None):
        raise ValueError("inv_freq and positions belong together")
    if inv_freq is not None:
        pairs = inv_freq.numel()
        check_dense("inv_freq", inv_freq, (pairs,), torch.float32, dev)
        shape = tuple(positions.shape)
        for lead in ((tokens,), (batch, tokens)):
            if shape == lead or (shape[:-1] == lead and shape[-1] in (1, 2)):
                axes, per_image = (1 if shape == lead else shape[-1]), len(lead) - 1
                break
        else:
            raise ValueError(f"positions shape {shape} is not [tokens(, axes)] or [batch, tokens(, axes)]")
        check_dense("positions", positions, shape, torch.int32, dev)
    return VscanQkNormArgs(
        batch, tokens, hq, hk, d, pairs, axes, _CODES[q.dtype], NORMS[norm], float(eps),
        q.data_ptr(), k.data_ptr(), yq.data_ptr(), yk.data_ptr(), None if wq is None else wq.data_ptr(),
        None if wk is None else wk.data_ptr(), inv_freq.data_ptr() if pairs else None,
        positions.data_ptr() if pairs else None, per_image, 0,
        *head_strides("q", q), *head_strides("k", k), *head_strides("yq", yq), *head_strides("yk", yk))


def qk_norm(q, k, wq=None, wk=None, *, norm="rms", eps=1e-6, inv_freq=None, positions=None, out=None, stream=None):
    """Normalised ("l2": unit length, "rms": unit mean square), weighted and rotated (yq, yk)
    (vscan_qknorm_forward). out: a pair of tensors to write to; (q, k) itself works in place."""
    if out is None:
        out = (torch.empty(q.shape, dtype=q.dtype, device=q.device), torch.empty(k.shape, dtype=k.dtype, device=k.device))
    for name, t, like in (("out[0]", out[0], q), ("out[1]", out[1], k)):
        check_tensor(name, t, like.shape, q.dtype, q.device)
    args = _marshal(q, k, wq, wk, *out, norm, eps, inv_freq, positions)
    with on_device(q.device):
        check(lib.vscan_qknorm_forward(ctypes.byref(args), stream_handle(stream, q.device, *out)))
    return tuple(out)


def qk_norm_backward(q, k, wq=None, wk=None, *, dyq, dyk, norm="rms", eps=1e-6, inv_freq=None, positions=None,
                     want=("dq", "dk", "dwq", "dwk"), stream=None):
    """Gradients of qk_norm (vscan_qknorm_backward) in a dict: dq and dk (dense, in the dtype of
    q) and, where there is a weight, dwq and dwk (float32, summed over the tokens in a fixed
    order). dyq, dyk: dL/dyq and dL/dyk in the dtype of q, with free strides. `want` limits
    the keys computed."""
    for name, t, like in (("dyq", dyq, q), ("dyk", dyk, k)):
        check_tensor(name, t, like.shape, q.dtype, q.device)
    args = _marshal(q, k, wq, wk, dyq, dyk, norm, eps, inv_freq, positions)
    like = {"dq": q, "dk": k, "dwq": wq, "dwk": wk}
    if not set(want) <= set(like):
        raise ValueError(f"want holds unknown gradients {sorted(set(want) - set(like))}")
    grads, out, dev = VscanQkNormGrads(), {}, q.device
    grads.dyq, grads.dyk = dyq.data_ptr(), dyk.data_ptr()
    for name in want:
        t = like[name]
        if t is not None:
            out[name] = torch.empty(t.shape, dtype=t.dtype, device=dev)
            setattr(grads, name, out[name].data_ptr())
    workspace = None
    if "dwq" in out or "dwk" in out:
        need = ctypes.c_uint64()
        check(lib.vscan_qknorm_backward_workspace_size(ctypes.byref(args), ctypes.byref(need)))
        workspace = torch.empty(need.value, dtype=torch.uint8, device=dev)
        grads.workspace, grads.workspace_bytes = workspace.data_ptr(), need.value
    with on_device(dev):
        check(lib.vscan_qknorm_backward(ctypes.byref(args), ctypes.byref(grads),
                                        stream_handle(stream, dev, workspace, *out.values())))
    return out
