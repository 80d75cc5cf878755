"""Chunked gated delta rule and its single-token step on the GPU against the definition in
float64, step by step."""
import pytest
import torch

import delta_testlib as R

vs = pytest.importorskip("vision_selective_state_b200")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def to_gpu(x, dtype):
    out = {n: x[n].to(DEV, R.DT[dtype]) for n in "qkvab"}
    out.update({n: x[n].to(DEV, torch.float32) for n in ("A", "bias")})
    return out


def f32(x):
    """A and bias as the float32 the kernels read."""
    return dict(x, A=x["A"].float().double(), bias=x["bias"].float().double())


def run(x, dtype, *, use_bias=True, **how):
    d = to_gpu(x, dtype)
    got = vs.delta_forward(d["q"], d["k"], d["v"], d["a"], d["b"], d["A"], d["bias"] if use_bias else None, **how)
    torch.cuda.synchronize()
    return got


SHAPES = [
    # batch, tokens, heads_k, heads_v, dim_k, dim_v
    (1, 1, 1, 1, 16, 16), (2, 2, 1, 2, 32, 48), (1, 63, 2, 2, 64, 64), (2, 64, 1, 1, 64, 128), (1, 65, 1, 1, 128, 16),
    (3, 129, 2, 4, 96, 80), (1, 197, 3, 3, 128, 128), (2, 100, 1, 3, 8, 8), (1, 130, 1, 2, 40, 200),
    (2, 77, 2, 2, 104, 256),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_plain_sequences(shape, dtype):
    batch, tokens, hk, hv, dk, dv = shape
    x = f32(R.delta_inputs(sum(shape), *shape, dtype))
    y, S = run(x, dtype, final_state=True)
    ry, rS = R.delta_ref(x)
    R.close(y, ry, dtype, R.ACC_FORWARD, "y")
    R.close(S, rS, "f32", R.ACC_FORWARD, "state")


def test_widths_off_the_tiles_in_fp32():
    for dk, dv in ((4, 4), (12, 20), (44, 52), (68, 132), (100, 252)):
        x = f32(R.delta_inputs(dk, 2, 70, 1, 2, dk, dv, "f32"))
        y, S = run(x, "f32", final_state=True)
        ry, rS = R.delta_ref(x)
        R.close(y, ry, "f32", R.ACC_FORWARD, f"y {dk} {dv}")
        R.close(S, rS, "f32", R.ACC_FORWARD, f"state {dk} {dv}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,h,w,cls", [("bidir", 9, 11, -1), ("bidir", 8, 9, 36), ("cross4", 7, 13, -1),
                                          ("cross4", 1, 70, -1), ("atrous2", 9, 15, -1), ("atrous2", 1, 1, -1),
                                          ("atrous2", 16, 18, -1)])
def test_every_direction_of_the_routes(kind, h, w, cls, dtype):
    r = vs.Route(kind, h, w, cls)
    x = f32(R.delta_inputs(h * w, 2, r.tokens, 1, 2, 24, 40, dtype))
    state = torch.randn(2, 2, 24, 40, generator=torch.Generator().manual_seed(1)) * 0.5
    for direction in range(r.K):
        y, S = run(x, dtype, route=r, direction=direction, initial_state=state.to(DEV), final_state=True)
        ry, rS = R.delta_ref(x, kind=kind, direction=direction, h=h, w=w, state=state.double())
        R.close(y, ry, dtype, R.ACC_FORWARD, f"y, direction {direction}")
        R.close(S, rS, "f32", R.ACC_FORWARD, f"state, direction {direction}")


def test_atrous_directions_fill_one_output_between_them():
    r = vs.Route("atrous2", 7, 10)
    x = f32(R.delta_inputs(3, 1, r.tokens, 1, 1, 16, 16, "f32"))
    d = to_gpu(x, "f32")
    out = torch.full((1, r.tokens, 1, 16), 7.0, device=DEV)
    for direction in range(4):
        vs.delta_forward(*(d[n] for n in ("q", "k", "v", "a", "b", "A", "bias")), route=r, direction=direction, out=out)
    ref = sum(R.delta_ref(x, kind="atrous2", direction=i, h=7, w=10)[0] for i in range(4))
    R.close(out, ref, "f32", R.ACC_FORWARD, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,behind", [([5, 0, 64, 1, 130], 0), ([0, 0, 0], 3), ([63, 65, 2], 9), ([200], 70),
                                            ([1] * 40, 5)])
def test_packed_sequences_and_rows_behind_them(lengths, behind, dtype):
    off = R.lengths_to_offsets(lengths)
    n = off[-1] + behind
    x = f32(R.delta_inputs(n, 1, n, 1, 2, 32, 24, dtype))
    d = to_gpu(x, dtype)
    # what lies behind the last sequence is neither read nor written
    for name in "qkvab":
        d[name][:, off[-1]:] = float("nan")
    state = torch.randn(len(lengths), 2, 32, 24, generator=torch.Generator().manual_seed(2)) * 0.5
    out = torch.full((1, n, 2, 24), 3.0, device=DEV, dtype=R.DT[dtype])
    y, S = vs.delta_forward(*(d[m] for m in ("q", "k", "v", "a", "b", "A", "bias")),
                            seq_offsets=torch.tensor(off, dtype=torch.int32, device=DEV), initial_state=state.to(DEV),
                            final_state=True, out=out)
    torch.cuda.synchronize()
    assert y is out and (out[:, off[-1]:] == 3.0).all()
    ry, rS = R.delta_ref(x, offsets=off, state=state.double())
    R.close(y[:, :off[-1]], ry[:, :off[-1]], dtype, R.ACC_FORWARD, "y")
    R.close(S, rS, "f32", R.ACC_FORWARD, "state")


def test_packed_equals_one_by_one():
    lengths = [70, 3, 128]
    off = R.lengths_to_offsets(lengths)
    x = f32(R.delta_inputs(9, 1, off[-1], 2, 2, 64, 64, "bf16"))
    d = to_gpu(x, "bf16")
    names = ("q", "k", "v", "a", "b")
    packed = vs.delta_forward(*(d[n] for n in names), d["A"], d["bias"],
                              seq_offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
    for o0, o1 in zip(off[:-1], off[1:]):
        one = vs.delta_forward(*(d[n][:, o0:o1] for n in names), d["A"], d["bias"])
        assert torch.equal(one, packed[:, o0:o1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_views_and_no_bias(dtype):
    batch, tokens, hk, hv, dk, dv = 2, 90, 2, 4, 32, 16
    x = f32(R.delta_inputs(5, batch, tokens, hk, hv, dk, dv, dtype))
    d = to_gpu(x, dtype)
    width = 2 * hk * dk + hv * dv + 2 * hv + 16
    packed = torch.full((batch, tokens + 3, width), float("nan"), device=DEV, dtype=R.DT[dtype])
    views, at = {}, 0
    for name, heads, dim in (("q", hk, dk), ("k", hk, dk), ("v", hv, dv)):
        views[name] = packed[:, :tokens, at:at + heads * dim].unflatten(2, (heads, dim))
        at += heads * dim
    for name in "ab":
        views[name] = packed[:, :tokens, at:at + hv]
        at += hv
    for name in "qkvab":
        views[name].copy_(d[name])
    out = torch.zeros(batch, tokens, 2 * hv, dv, device=DEV, dtype=R.DT[dtype])
    y = vs.delta_forward(*(views[n] for n in "qkvab"), d["A"], out=out[:, :, hv:], scale=0.7, beta_scale=1.5)
    torch.cuda.synchronize()
    ry, _ = R.delta_ref(x, use_bias=False, scale=0.7, beta_scale=1.5)
    R.close(y, ry, dtype, R.ACC_FORWARD, "y")
    assert (out[:, :, :hv] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_neighbouring_keys_that_point_the_same_way(dtype):
    x = f32(R.delta_inputs(6, 1, 256, 1, 1, 64, 64, dtype, correlated=True, decay=0.05))
    y, S = run(x, dtype, final_state=True)
    ry, rS = R.delta_ref(x)
    # the triangle's inverse has entries of both signs up to 1: a factor of two on the bound
    R.close(y, ry, dtype, 2 * R.ACC_FORWARD, "y")
    R.close(S, rS, "f32", 2 * R.ACC_FORWARD, "state")


def test_extreme_decays_and_strengths():
    x = f32(R.delta_inputs(7, 1, 150, 1, 4, 32, 32, "f32"))
    x["a"][0, 10] = 200.0   # forgets everything
    x["a"][0, 70:90] = -200.0  # keeps everything
    x["a"][0, 100, 0] = 3e4
    x["b"][0, 20:30] = -200.0  # writes nothing
    x["b"][0, 40:50] = 200.0
    x["A"][1] = 0.0           # the ungated rule
    x["A"][2] = -1000.0
    x["A"] = x["A"].float().double()
    y, S = run(x, "f32", final_state=True)
    ry, rS = R.delta_ref(x)
    for h in range(4):  # head by head: their magnitudes differ
        R.close(y[:, :, h], ry[:, :, h], "f32", R.ACC_FORWARD, f"y, head {h}")
        R.close(S[:, h], rS[:, h], "f32", R.ACC_FORWARD, f"state, head {h}")


def test_two_halves_carry_the_state():
    x = f32(R.delta_inputs(8, 2, 150, 1, 1, 48, 48, "f32"))
    d = to_gpu(x, "f32")
    names = ("q", "k", "v", "a", "b")
    first, S = vs.delta_forward(*(d[n][:, :70] for n in names), d["A"], d["bias"], final_state=True)
    second, S2 = vs.delta_forward(*(d[n][:, 70:] for n in names), d["A"], d["bias"], initial_state=S, final_state=S)
    assert S2 is S
    ry, rS = R.delta_ref(x)
    R.close(torch.cat([first, second], 1), ry, "f32", R.ACC_FORWARD, "y")
    R.close(S, rS, "f32", R.ACC_FORWARD, "state")


def test_empty_batches_and_sequences():
    for batch, tokens in ((0, 5), (2, 0)):
        x = f32(R.delta_inputs(1, batch, tokens, 1, 1, 16, 16, "bf16"))
        state = torch.randn(batch, 1, 16, 16)
        y, S = run(x, "bf16", initial_state=state.to(DEV), final_state=True)
        assert y.shape == (batch, tokens, 1, 16) and torch.equal(S.cpu(), state)
    y = run(f32(R.delta_inputs(1, 2, 0, 1, 1, 16, 16, "bf16")), "bf16")
    assert y.shape == (2, 0, 1, 16)


def test_runs_are_identical_and_graphs_replay_them():
    x = f32(R.delta_inputs(11, 2, 300, 2, 2, 64, 64, "bf16"))
    d = to_gpu(x, "bf16")
    args = [d[n] for n in ("q", "k", "v", "a", "b", "A", "bias")]
    eager = vs.delta_forward(*args)
    assert torch.equal(eager, vs.delta_forward(*args))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = vs.delta_forward(*args)
    y.zero_()
    d["v"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, vs.delta_forward(*args)) and not torch.equal(y, eager)


def test_another_stream():
    x = f32(R.delta_inputs(12, 1, 200, 1, 1, 64, 64, "bf16"))
    d = to_gpu(x, "bf16")
    args = [d[n] for n in ("q", "k", "v", "a", "b", "A", "bias")]
    eager = vs.delta_forward(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = vs.delta_forward(*args, stream=s)
    junk = [torch.full((1 << 20,), 1.0, device=DEV) for _ in range(4)]  # would reuse freed scratch
    s.synchronize()
    assert torch.equal(y, eager) and len(junk) == 4


# ------------------------------------------------------------------ one token
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16, 16), (3, 2, 6, 72, 104), (5, 1, 2, 128, 256), (2, 3, 3, 64, 64),
                                   (1, 1, 1, 8, 8), (130, 1, 1, 24, 40)], ids=str)
def test_step(shape, dtype):
    batch, hk, hv, dk, dv = shape
    x = f32(R.delta_inputs(sum(shape), batch, 1, hk, hv, dk, dv, dtype))
    state = torch.randn(batch, hv, dk, dv, generator=torch.Generator().manual_seed(3))
    d = to_gpu(x, dtype)
    args = [d[n][:, 0] for n in "qkvab"] + [d["A"], d["bias"]]
    ry, rS = R.delta_ref(x, state=state.double())
    S = state.to(DEV)
    new = torch.empty_like(S)
    y, out = vs.delta_step(*args, state=S, state_out=new)
    assert out is new and torch.equal(S.cpu(), state)
    # sums of dk products: each of at most 16 register and 5 tree additions rounds by 2^-24
    R.close(y, ry[:, 0], dtype, 2 * 21 * 2.0 ** -24 * 8, "y")
    R.close(new, rS, "f32", 2 * 21 * 2.0 ** -24 * 8, "state")
    y2, out = vs.delta_step(*args, state=S)  # in place
    assert out is S and torch.equal(S, new) and torch.equal(y2, y)


def test_steps_continue_a_chunked_pass():
    x = f32(R.delta_inputs(13, 2, 140, 1, 2, 64, 64, "f32"))
    d = to_gpu(x, "f32")
    names = ("q", "k", "v", "a", "b")
    y, S = vs.delta_forward(*(d[n][:, :130] for n in names), d["A"], d["bias"], final_state=True)
    ys = [y]
    for t in range(130, 140):
        y, S = vs.delta_step(*(d[n][:, t] for n in names), d["A"], d["bias"], state=S)
        ys.append(y[:, None])
    ry, rS = R.delta_ref(x)
    R.close(torch.cat(ys, 1), ry, "f32", R.ACC_FORWARD, "y")
    R.close(S, rS, "f32", R.ACC_FORWARD, "state")


# ------------------------------------------------------------------ calls that are easy to get wrong
def test_offsets_that_make_no_sense_stay_inside_their_arrays():
    """Decreasing, negative and too large offsets are clamped: the call ends, and what lies around
    its outputs is as it was (the outputs themselves are not defined)."""
    n, hv, d = 200, 2, 32
    x = f32(R.delta_inputs(14, 1, n, 1, hv, d, d, "bf16"))
    d_ = to_gpu(x, "bf16")
    around = torch.full((1, n + 128, hv, d), 5.0, device=DEV, dtype=torch.bfloat16)
    for offsets in ([0, 300, -7, 150], [150, 100, 50, 0], [-100, -1, 2 ** 31 - 1, 3], [200, 200, 200, 200]):
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        states = torch.full((5, hv, d, d), 9.0, device=DEV)
        vs.delta_forward(*(d_[m] for m in ("q", "k", "v", "a", "b", "A", "bias")), seq_offsets=off,
                         out=around[:, 64:64 + n], final_state=states[1:4])
        torch.cuda.synchronize()
        assert (around[:, :64] == 5.0).all() and (around[:, 64 + n:] == 5.0).all()
        assert (states[0] == 9.0).all() and (states[4] == 9.0).all()
        got = vs.delta_backward(*(d_[m] for m in ("q", "k", "v", "a", "b", "A", "bias")), seq_offsets=off, dy=d_["v"])
        torch.cuda.synchronize()
        assert got["dq"].shape == d_["q"].shape


def test_two_calls_at_once_and_graphs_that_share_a_workspace():
    xs = [to_gpu(f32(R.delta_inputs(seed, 1, 700, 2, 2, 64, 64, "bf16")), "bf16") for seed in (15, 16)]
    args = [[d[n] for n in ("q", "k", "v", "a", "b", "A", "bias")] for d in xs]
    want = [vs.delta_forward(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [vs.delta_forward(*a, stream=s) for a, s in zip(args, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    # one workspace, two captured calls, replayed in turn on one stream
    workspace = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)
    held, graphs = [], []
    for a in args:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(vs.delta_forward(*a, workspace=workspace))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(h, w) for h, w in zip(held, want))


def test_image_strides_beyond_32_bits():
    batch, n, h, d = 2, 66, 1, 16
    x = f32(R.delta_inputs(17, batch, n, h, h, d, d, "bf16"))
    dd = to_gpu(x, "bf16")
    stride = 2 ** 31 + 64
    far = torch.empty(stride + n * h * d, dtype=torch.bfloat16, device=DEV)
    views = {}
    for m in ("q", "v"):  # one buffer each in turn would be larger: q and v share it, at different places
        at = 0 if m == "q" else n * h * d
        views[m] = torch.as_strided(far, (batch, n, h, d), (stride - n * h * d, h * d, d, 1), at)
        views[m].copy_(dd[m])
    near = vs.delta_forward(*(dd[m] for m in ("q", "k", "v", "a", "b", "A", "bias")))
    got = vs.delta_forward(views["q"], dd["k"], views["v"], dd["a"], dd["b"], dd["A"], dd["bias"])
    assert torch.equal(near, got)


def test_a_later_token_does_not_touch_an_earlier_chunk():
    x = f32(R.delta_inputs(18, 1, 192, 1, 1, 32, 32, "f32"))
    d = to_gpu(x, "f32")
    args = lambda: [d[n] for n in ("q", "k", "v", "a", "b", "A", "bias")]  # noqa: E731
    first = vs.delta_forward(*args())
    for n in ("q", "k", "v"):
        d[n][:, 130:] = float("inf")
    second = vs.delta_forward(*args())
    assert torch.equal(first[:, :128], second[:, :128])


def test_one_head_shared_by_many_and_sizes_at_the_limits():
    for hk, hv, dk, dv in ((1, 7, 128, 256), (1, 1, 4, 4), (3, 3, 64, 4), (1, 2, 128, 132)):
        x = f32(R.delta_inputs(hv + dk, 1, 67, hk, hv, dk, dv, "f32"))
        y, S = run(x, "f32", final_state=True)
        ry, rS = R.delta_ref(x)
        R.close(y, ry, "f32", R.ACC_FORWARD, f"y {hk} {hv} {dk} {dv}")
        R.close(S, rS, "f32", R.ACC_FORWARD, "state")


def test_expanded_inputs_and_foreign_workspaces_are_refused():
    x = to_gpu(f32(R.delta_inputs(3, 2, 5, 1, 1, 16, 16, "f32")), "f32")
    names = ("q", "k", "v", "a", "b", "A", "bias")
    for name in ("q", "k", "v", "a", "b"):
        for axis in (0, 1):
            one = x[name].narrow(axis, 0, 1).expand(x[name].shape)
            with pytest.raises(ValueError, match="stride of 0"):
                vs.delta_forward(*(one if n == name else x[n] for n in names))
    step = [x[n] if n in ("A", "bias") else x[n][:, 0].contiguous() for n in names]
    state = torch.zeros(2, 1, 16, 16, device=DEV)
    step[0] = step[0][:1].expand(step[0].shape)
    with pytest.raises(ValueError, match="stride of 0"):
        vs.delta_step(*step, state=state)
    with pytest.raises(ValueError, match="stride of 0"):
        vs.qk_norm(x["q"], x["k"][:1].expand(x["k"].shape))
    with pytest.raises(ValueError, match="workspace"):
        vs.delta_forward(*(x[n] for n in names), workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace"):
        vs.delta_backward(*(x[n] for n in names), dy=x["v"], workspace=torch.zeros(1 << 20, dtype=torch.uint8))
