"""Gradients of packed calls without a sequence: no step visits a row, so every row's are 0."""
import ctypes

import pytest
import torch

import delta_testlib as R

vs = pytest.importorskip("vision_selective_state_b200")
abi = pytest.importorskip("vision_selective_state_b200._abi")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOKENS, HK, HV, DK, DV = 37, 1, 2, 16, 24


def args_of(dtype):
    x = R.delta_inputs(1, 1, TOKENS, HK, HV, DK, DV, dtype)
    return [x[n].to(DEV, torch.float32 if n in ("A", "bias") else R.DT[dtype]) for n in
            ("q", "k", "v", "a", "b", "A", "bias")]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_sequence_clears_every_gradient(dtype):
    """Through the C interface, into memory that holds NaN."""
    q, k, v, a, b, A, bias = args_of(dtype)
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = abi.VscanDeltaArgs()
    args.batch, args.tokens, args.heads_k, args.heads_v, args.dim_k, args.dim_v = 0, TOKENS, HK, HV, DK, DV
    args.dtype, args.scale, args.beta_scale = (abi.F32 if dtype == "f32" else abi.BF16), 1.0, 1.0
    for n, t in zip(("q", "k", "v", "a", "b", "A", "bias"), (q, k, v, a, b, A, bias)):
        setattr(args, n, t.data_ptr())
    args.seq_offsets = none.data_ptr()
    grads, out = abi.VscanDeltaGrads(), {}
    for n, t in dict(dq=q, dk=k, dv=v, da=a, db=b, dA=A, dbias=bias).items():
        # a row of NaN before and behind: nothing but the gradient is written
        whole = torch.full((t.numel() + 128,), float("nan"), dtype=t.dtype, device=DEV)
        out[n] = whole
        setattr(grads, n, whole[64:].data_ptr())
    abi.check(abi.lib.vscan_delta_backward(None, ctypes.byref(args), v.data_ptr(), ctypes.byref(grads),
                                           torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    for n, whole in out.items():
        assert (whole[64:-64] == 0).all(), n
        assert whole[:64].isnan().all() and whole[-64:].isnan().all(), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_sequence_through_the_binding(dtype):
    args = args_of(dtype)
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    state = torch.zeros(0, HV, DK, DV, device=DEV)
    y, S = vs.delta_forward(*args, seq_offsets=none, initial_state=state, final_state=True)
    assert y.shape == args[2].shape and (y == 0).all() and S.shape == state.shape
    for _ in range(3):  # the allocator's memory holds NaN
        junk = [torch.full_like(t, float("nan")) for t in args for _ in range(4)]
        del junk
        got = vs.delta_backward(*args, dy=args[2], seq_offsets=none, initial_state=state, d_final_state=state)
        assert set(got) == {"dq", "dk", "dv", "da", "db", "dA", "dbias", "d_initial_state"}
        for n, t in got.items():
            assert (t == 0).all(), n
