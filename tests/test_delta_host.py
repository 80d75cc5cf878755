"""Host-side checks of the delta rule and the query/key norm: no GPU needed, no kernel launched.
Every call here either is host-only by contract or fails its argument checks, which run before
the library's first CUDA call. No call with plausible-looking fake device pointers is ever
allowed to pass them."""
import ctypes

import pytest
import torch

import delta_testlib as R

abi = pytest.importorskip("vision_selective_state_b200._abi")
vs = pytest.importorskip("vision_selective_state_b200")

INVALID, SHAPE, ALIGNMENT, UNSUPPORTED, WORKSPACE = -1, -2, -3, -4, -6


def _delta(**kw):
    a = abi.VscanDeltaArgs()
    a.batch, a.tokens, a.heads_k, a.heads_v, a.dim_k, a.dim_v, a.dtype = 2, 100, 2, 4, 32, 48, abi.BF16
    a.scale, a.beta_scale = 1.0, 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _pointers(a):
    for n in ("q", "k", "v", "a", "b", "y", "A"):
        setattr(a, n, 4096)
    return a


def _size(a, route=None, name="vscan_delta_workspace_size"):
    n = ctypes.c_uint64()
    return getattr(abi.lib, name)(route, ctypes.byref(a), ctypes.byref(n)), n.value


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(abi.VscanDeltaArgs) == 8 * 4 + 11 * 8 + 2 * 4 + 12 * 8 + 3 * 8
    assert abi.VscanDeltaArgs.q.offset == 32 and abi.VscanDeltaArgs.scale.offset == 120
    assert abi.VscanDeltaArgs.q_tok_stride.offset == 128 and abi.VscanDeltaArgs.workspace.offset == 224
    assert abi.VscanDeltaArgs.status.offset == 240
    assert ctypes.sizeof(abi.VscanDeltaGrads) == 11 * 8
    assert ctypes.sizeof(abi.VscanQkNormArgs) == 10 * 4 + 8 * 8 + 2 * 4 + 8 * 8
    assert abi.VscanQkNormArgs.q.offset == 40 and abi.VscanQkNormArgs.q_tok_stride.offset == 112
    assert ctypes.sizeof(abi.VscanQkNormGrads) == 8 * 8


@pytest.mark.parametrize("field,value,status", [
    ("batch", -1, INVALID), ("tokens", -1, INVALID), ("heads_k", 0, INVALID), ("heads_v", 0, INVALID),
    ("heads_v", 3, SHAPE), ("dim_k", 0, INVALID), ("dim_v", 0, INVALID), ("dim_k", 20, ALIGNMENT), ("dim_v", 20, ALIGNMENT),
    ("dim_k", 136, UNSUPPORTED), ("dim_v", 264, UNSUPPORTED), ("dtype", 2, INVALID), ("direction", 1, SHAPE),
    ("direction", -1, SHAPE), ("scale", float("nan"), INVALID), ("beta_scale", float("inf"), INVALID),
    ("batch", 65536, UNSUPPORTED), ("q_tok_stride", 32, ALIGNMENT), ("k_tok_stride", 68, ALIGNMENT),
    ("v_batch_stride", 4, ALIGNMENT), ("y_tok_stride", -8, INVALID), ("a_batch_stride", -1, INVALID),
])
def test_bad_delta_arguments_fail_before_any_cuda_call(field, value, status):
    a = _pointers(_delta(**{field: value}))
    g = abi.VscanDeltaGrads()
    assert abi.lib.vscan_delta_forward(None, ctypes.byref(a), None) == status
    assert abi.lib.vscan_delta_backward(None, ctypes.byref(a), 4096, ctypes.byref(g), None) == status
    assert _size(a)[0] == status and _size(a, name="vscan_delta_backward_workspace_size")[0] == status
    a.tokens = 1 if field != "tokens" else value
    if field not in ("y_tok_stride",):
        assert abi.lib.vscan_delta_step(ctypes.byref(a), None) == status
    assert abi.lib.vscan_last_error().decode()


@pytest.mark.parametrize("name", ["q", "k", "v", "a", "b", "y", "A"])
def test_null_and_misaligned_delta_pointers(name):
    a = _pointers(_delta())
    setattr(a, name, None)
    assert abi.lib.vscan_delta_forward(None, ctypes.byref(a), None) == INVALID
    setattr(a, name, 4096 + 1)
    assert abi.lib.vscan_delta_forward(None, ctypes.byref(a), None) == ALIGNMENT
    a = _pointers(_delta(tokens=1))
    a.initial_state = a.final_state = 4096
    setattr(a, name, None)
    assert abi.lib.vscan_delta_step(ctypes.byref(a), None) == INVALID


def test_states_workspaces_and_status_words():
    a = _pointers(_delta())
    assert abi.lib.vscan_delta_forward(None, ctypes.byref(a), None) == WORKSPACE
    need = _size(a)[1]
    a.workspace, a.workspace_bytes = 4096, need - 1
    assert abi.lib.vscan_delta_forward(None, ctypes.byref(a), None) == WORKSPACE
    a.workspace, a.workspace_bytes = 4096 + 8, need
    assert abi.lib.vscan_delta_forward(None, ctypes.byref(a), None) == ALIGNMENT
    for field in ("initial_state", "final_state"):
        a = _pointers(_delta(**{field: 4096 + 4}))
        assert abi.lib.vscan_delta_forward(None, ctypes.byref(a), None) == ALIGNMENT
    for field in ("bias", "seq_offsets", "status"):
        a = _pointers(_delta(**{field: 4096 + 2}))
        assert abi.lib.vscan_delta_forward(None, ctypes.byref(a), None) == ALIGNMENT
    a = _pointers(_delta())
    g = abi.VscanDeltaGrads()
    assert abi.lib.vscan_delta_backward(None, ctypes.byref(a), None, ctypes.byref(g), None) == INVALID
    assert abi.lib.vscan_delta_backward(None, ctypes.byref(a), 4096, None, None) == INVALID
    assert abi.lib.vscan_delta_backward(None, ctypes.byref(a), 4096, ctypes.byref(g), None) == WORKSPACE
    g.d_final_state = g.d_initial_state = 4096
    assert abi.lib.vscan_delta_backward(None, ctypes.byref(a), 4096, ctypes.byref(g), None) == INVALID
    for field in ("dq", "dk", "dv", "d_initial_state", "d_final_state", "da", "dA"):
        g = abi.VscanDeltaGrads()
        setattr(g, field, 4096 + 1)
        assert abi.lib.vscan_delta_backward(None, ctypes.byref(a), 4096, ctypes.byref(g), None) == ALIGNMENT


def test_the_step_takes_one_token_and_both_states():
    a = _pointers(_delta())
    assert abi.lib.vscan_delta_step(ctypes.byref(a), None) == SHAPE
    a.tokens = 1
    assert abi.lib.vscan_delta_step(ctypes.byref(a), None) == INVALID
    a.initial_state = 4096
    assert abi.lib.vscan_delta_step(ctypes.byref(a), None) == INVALID
    a.final_state, a.seq_offsets = 4096, 4096
    assert abi.lib.vscan_delta_step(ctypes.byref(a), None) == UNSUPPORTED


def test_routes_of_the_delta_rule():
    r = vs.Route("cross4", 10, 10)
    a = _pointers(_delta(direction=4))
    assert abi.lib.vscan_delta_forward(r.handle, ctypes.byref(a), None) == SHAPE
    a.direction, a.tokens = 3, 99
    assert abi.lib.vscan_delta_forward(r.handle, ctypes.byref(a), None) == SHAPE
    a.tokens, a.seq_offsets = 100, 4096
    assert abi.lib.vscan_delta_forward(r.handle, ctypes.byref(a), None) == UNSUPPORTED
    a = _pointers(_delta(tokens=100))
    pooled = vs.Route("pool_w", 10, 10)
    assert abi.lib.vscan_delta_forward(pooled.handle, ctypes.byref(a), None) == UNSUPPORTED


def test_workspace_sizes_and_empty_calls():
    plane = 64 * 64 * 2
    r256 = lambda n: (n + 255) // 256 * 256  # noqa: E731
    assert _size(_delta()) == (0, r256(2 * 2 * 4 * (2048 + 5 * plane)))
    assert _size(_delta(dtype=abi.F32)) == (0, r256(2 * 2 * 4 * (2048 + 12 * plane)))
    assert _size(_delta(dtype=abi.F32, dim_k=128)) == (0, r256(2 * 2 * 4 * (2048 + 18 * plane)))
    assert _size(_delta(seq_offsets=4096)) == (0, r256((100 // 64 + 2 + 1) * 4 * (2048 + 5 * plane)))
    assert _size(_delta(batch=0)) == (0, 0) and _size(_delta(tokens=0)) == (0, 0)
    atrous = vs.Route("atrous2", 10, 10)  # 25 steps a direction: one chunk
    assert _size(_delta(), atrous.handle) == (0, r256(2 * 1 * 4 * (2048 + 5 * plane)))
    n = 2 * 2 * 4
    backward = (r256(n * (2048 + 6 * plane)) + r256(n * 64 * 64 * 4) + 2 * r256(n * 48 * 64 * 4) + 2 * r256(n * 64 * 48 * 4)
                + r256(n * 8) + 2 * r256(2 * 100 * 4 * 32 * 4))
    assert _size(_delta(), name="vscan_delta_backward_workspace_size") == (0, backward)
    # nothing to do: accepted without a pointer, and nothing is launched
    assert abi.lib.vscan_delta_forward(None, ctypes.byref(_delta(batch=0)), None) == 0
    assert abi.lib.vscan_delta_forward(None, ctypes.byref(_delta(tokens=0)), None) == 0
    assert abi.lib.vscan_delta_step(ctypes.byref(_delta(batch=0, tokens=1)), None) == 0


def _norm(**kw):
    a = abi.VscanQkNormArgs()
    a.batch, a.tokens, a.heads_q, a.heads_k, a.dim, a.pairs, a.axes, a.dtype, a.norm, a.eps = 2, 9, 3, 1, 64, 0, 1, abi.BF16, 1, 1e-6
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("fields,status", [
    ({"batch": -1}, INVALID), ({"tokens": -1}, INVALID), ({"heads_q": 0}, INVALID), ({"heads_k": 0}, INVALID),
    ({"dim": 0}, INVALID), ({"dim": 60}, ALIGNMENT), ({"dim": 264}, UNSUPPORTED), ({"dtype": 3}, INVALID), ({"norm": 2}, INVALID),
    ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID), ({"reserved": 1}, INVALID), ({"pos_per_image": 2}, INVALID),
    ({"pairs": 33}, SHAPE), ({"pairs": -1}, SHAPE), ({"axes": 3}, SHAPE), ({"pairs": 3, "axes": 2}, SHAPE), ({"pairs": 4}, INVALID),
    ({"pairs": 4, "inv_freq": 4096}, INVALID), ({"q_tok_stride": 64}, ALIGNMENT), ({"k_tok_stride": 68}, ALIGNMENT),
    ({"yq_batch_stride": -8}, INVALID), ({"wq": 4097}, ALIGNMENT), ({"q": None}, INVALID), ({"yk": None}, INVALID),
    ({"k": 4104}, ALIGNMENT), ({"yq": 4104}, ALIGNMENT),
])
def test_bad_norm_arguments_fail_before_any_cuda_call(fields, status):
    a = _norm(q=4096, k=4096, yq=4096, yk=4096)
    for k, v in fields.items():
        setattr(a, k, v)
    assert abi.lib.vscan_qknorm_forward(ctypes.byref(a), None) == status
    assert abi.lib.vscan_last_error().decode()
    if not set(fields) & {"yk", "yq"}:
        g = abi.VscanQkNormGrads()
        g.dyq = g.dyk = 4096
        assert abi.lib.vscan_qknorm_backward(ctypes.byref(a), ctypes.byref(g), None) == status


def test_norm_gradients_need_their_pointers_and_scratch():
    a = _norm(q=4096, k=4096)
    g = abi.VscanQkNormGrads()
    assert abi.lib.vscan_qknorm_backward(ctypes.byref(a), ctypes.byref(g), None) == INVALID
    assert abi.lib.vscan_qknorm_backward(ctypes.byref(a), None, None) == INVALID
    g.dyq = g.dyk = 4096
    g.dwq = 4096
    assert abi.lib.vscan_qknorm_backward(ctypes.byref(a), ctypes.byref(g), None) == WORKSPACE
    g.dwq = 4097
    assert abi.lib.vscan_qknorm_backward(ctypes.byref(a), ctypes.byref(g), None) == ALIGNMENT
    g.dwq, g.dq = None, 4104
    assert abi.lib.vscan_qknorm_backward(ctypes.byref(a), ctypes.byref(g), None) == ALIGNMENT
    n = ctypes.c_uint64()
    assert abi.lib.vscan_qknorm_backward_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
    assert n.value > 0 and n.value % (2 * 64 * 4) == 0
    assert abi.lib.vscan_qknorm_forward(ctypes.byref(_norm(batch=0)), None) == 0


def test_the_binding_refuses_what_it_cannot_marshal():
    q = torch.zeros(1, 4, 2, 16)
    g = torch.zeros(1, 4, 2)
    A = torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        vs.delta_forward(q, q, q, g, g, A)
    with pytest.raises(TypeError, match="dtype"):
        vs.delta_forward(q.half(), q, q, g, g, A)
    with pytest.raises(ValueError, match="CUDA"):
        vs.delta_step(q[:, 0], q[:, 0], q[:, 0], g[:, 0], g[:, 0], A, state=torch.zeros(1, 2, 16, 16))
    with pytest.raises(ValueError, match="CUDA"):
        vs.qk_norm(q, q)
    with pytest.raises(TypeError, match="dtype"):
        vs.qk_norm(q.double(), q.double())


def test_the_binding_refuses_an_expanded_axis():
    from vision_selective_state_b200.delta import _row_strides, head_strides
    x, row = torch.zeros(1, 1, 2, 16), torch.zeros(1, 1, 2)
    for shape in ((3, 1, 2, 16), (1, 3, 2, 16), (3, 5, 2, 16)):
        with pytest.raises(ValueError, match="stride of 0"):
            head_strides("q", x.expand(shape), False)
        with pytest.raises(ValueError, match="stride of 0"):
            _row_strides("a", row.expand(shape[:3]), False)
    assert head_strides("q", x.expand(1, 1, 2, 16), False) == (32, 32)


# ------------------------------------------------------------------ the float64 forms themselves
def test_the_reference_step_on_a_worked_example():
    """One head of width one: S = 2, decay 1/2, beta 1/2, k = 1, v = 3: S' = 1 + (3 - 1) / 2 = 2, y = 2 q."""
    one = torch.ones(1, 1, 1, 1, dtype=torch.float64)
    A = torch.tensor([-1.0], dtype=torch.float64)
    raw = torch.full((1, 1, 1), 0.0, dtype=torch.float64)  # softplus(0) = log 2: decay 1/2; sigmoid(0) = 1/2
    x = dict(q=5 * one, k=one, v=3 * one, a=raw, b=raw, A=A, bias=torch.zeros(1, dtype=torch.float64))
    y, S = R.delta_ref(x, state=2 * one, scale=1.0)
    assert abs(float(S) - 2.0) < 1e-15 and abs(float(y) - 10.0) < 1e-14


def test_the_reference_with_a_unit_key_stores_and_recalls():
    """beta = 1, no decay, orthonormal keys: reading with a key returns its value."""
    n = 8
    x = dict(q=torch.eye(n).double()[None, :, None], k=torch.eye(n).double()[None, :, None],
             v=torch.arange(n * 3).double().reshape(1, n, 1, 3), a=torch.zeros(1, n, 1).double(),
             b=torch.full((1, n, 1), 200.0).double(), A=torch.zeros(1).double(), bias=torch.zeros(1).double())
    y, S = R.delta_ref(x, scale=1.0)
    assert torch.allclose(y, x["v"], atol=1e-12) and torch.allclose(S[0, 0], x["v"][0, :, 0], atol=1e-12)


def test_the_reference_gradient_is_the_change_of_its_value():
    x = R.delta_inputs(3, 1, 5, 1, 2, 4, 4, "f32")
    g = torch.Generator().manual_seed(1)
    dy = torch.randn(x["v"].shape, generator=g).double()
    for n in ("q", "k", "v", "a", "b", "A", "bias"):
        leaf = x[n].clone().requires_grad_()
        (grad,) = torch.autograd.grad((R.delta_ref(dict(x, **{n: leaf}))[0] * dy).sum(), [leaf])
        u = torch.randn(x[n].shape, generator=g).double()
        fd = R.finite_difference(lambda z: (R.delta_ref(dict(x, **{n: z}))[0] * dy).sum(), x[n], u)
        assert abs(fd - float((grad * u).sum())) < 1e-7 * max(1.0, abs(fd)), n


def test_the_reference_orders_match_the_route_fixtures():
    from conftest import read_route_fixture

    for kind, name in (("cross4", "cross_scan_routes.txt"), ("atrous2", "atrous_routes.txt")):
        for (h, w), dirs in read_route_fixture(name).items():
            for k, want in dirs.items():
                assert R.order(kind, k, h, w, h * w) == want, (kind, h, w, k)
