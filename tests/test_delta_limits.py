"""Sizes at the ends of 32-bit counters are refused on the host: no GPU needed, no kernel launched."""
import ctypes

import pytest

abi = pytest.importorskip("vision_selective_state_b200._abi")

INVALID, UNSUPPORTED = -1, -4


@pytest.mark.parametrize("batch,heads_q,heads_k,ok", [
    (1, 2 ** 31 - 2, 1, False), (1, 1, 2 ** 31 - 2, False), (2 ** 30 - 1, 1, 1, False), (1, 2 ** 31 - 1025, 1, False),
    (1, 2 ** 31 - 1026, 1, True), (2 ** 30 - 513, 1, 1, True), (65536, 32768, 32767, False),
])
def test_rows_that_a_lane_counts_past_2_31(batch, heads_q, heads_k, ok):
    """A lane of the norm steps through images x heads rows, up to 512 behind the last."""
    a = abi.VscanQkNormArgs()
    a.batch, a.tokens, a.heads_q, a.heads_k, a.dim, a.axes, a.dtype, a.eps = batch, 1, heads_q, heads_k, 4, 1, abi.F32, 1e-6
    n, g = ctypes.c_uint64(), abi.VscanQkNormGrads()
    assert abi.lib.vscan_qknorm_backward_workspace_size(ctypes.byref(a), ctypes.byref(n)) == (0 if ok else UNSUPPORTED)
    # without pointers: refused for its size, or for the pointers that it lacks
    assert abi.lib.vscan_qknorm_forward(ctypes.byref(a), None) == (INVALID if ok else UNSUPPORTED)
    assert abi.lib.vscan_qknorm_backward(ctypes.byref(a), ctypes.byref(g), None) == (INVALID if ok else UNSUPPORTED)


@pytest.mark.parametrize("tokens,ok", [(2 ** 31 - 1, False), (2 ** 31 - 63, False), (2 ** 31 - 64, True), (2 ** 30, True)])
def test_tokens_that_do_not_round_up_to_chunks(tokens, ok):
    """The number of chunks of 64 steps rounds the tokens up, in 32 bits."""
    a = abi.VscanDeltaArgs()
    a.batch, a.tokens, a.heads_k, a.heads_v, a.dim_k, a.dim_v, a.dtype = 1, tokens, 1, 1, 8, 8, abi.BF16
    a.scale, a.beta_scale = 1.0, 1.0
    n = ctypes.c_uint64()
    assert abi.lib.vscan_delta_workspace_size(None, ctypes.byref(a), ctypes.byref(n)) == (0 if ok else UNSUPPORTED)
    if ok:
        assert n.value == -(-tokens // 64) * (2048 + 5 * 64 * 64 * 2)
    assert abi.lib.vscan_delta_backward_workspace_size(None, ctypes.byref(a), ctypes.byref(n)) == (0 if ok else UNSUPPORTED)
    # without pointers: refused for its size, or for the pointers that it lacks
    assert abi.lib.vscan_delta_forward(None, ctypes.byref(a), None) == (INVALID if ok else UNSUPPORTED)
