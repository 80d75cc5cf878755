"""Gradients of the gated delta rule on the GPU against those of the float64 definition."""
import pytest
import torch

import delta_testlib as R

vs = pytest.importorskip("vision_selective_state_b200")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KEYS = {"dq": "q", "dk": "k", "dv": "v", "da": "a", "db": "b", "dA": "A", "dbias": "bias", "d_initial_state": "state"}


def f32(x):
    return dict(x, A=x["A"].float().double(), bias=x["bias"].float().double())


def case(x, dtype, seed, *, rows, state=False, dstate=False, route=None, direction=0, kind=None, h=0, w=0, offsets=None,
         use_bias=True, **how):
    """(gradients of the library, gradients of the definition)."""
    g = torch.Generator().manual_seed(seed)
    hv, dk, dv = x["v"].shape[2], x["q"].shape[3], x["v"].shape[3]
    dy = torch.randn(x["v"].shape, generator=g).to(R.DT[dtype]).double()
    S0 = torch.randn(rows, hv, dk, dv, generator=g) * 0.5 if state else None
    dS = torch.randn(rows, hv, dk, dv, generator=g) * 0.5 if dstate else None
    # A and bias per token: their gradients are the terms of dA and dbias
    leaves = {n: (t.expand(x["a"].shape) if n in ("A", "bias") else t).clone().requires_grad_() for n, t in x.items()}
    if state:
        leaves["state"] = S0.double().requires_grad_()
    y, S = R.delta_ref({n: leaves[n] for n in x}, kind=kind, direction=direction, h=h, w=w, offsets=offsets,
                       state=leaves.get("state"), use_bias=use_bias, **how)
    loss = (y * dy).sum() + ((S * dS.double()).sum() if dstate else 0)
    ref = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)))
    ref = {n: torch.zeros_like(leaves[n]) if r is None else r for n, r in ref.items()}
    d = {n: x[n].to(DEV, R.DT[dtype]) for n in "qkvab"}
    d.update({n: x[n].to(DEV, torch.float32) for n in ("A", "bias")})
    got = vs.delta_backward(d["q"], d["k"], d["v"], d["a"], d["b"], d["A"], d["bias"] if use_bias else None,
                            dy=dy.to(DEV, R.DT[dtype]), route=route, direction=direction,
                            seq_offsets=None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV),
                            initial_state=None if S0 is None else S0.to(DEV),
                            d_final_state=None if dS is None else dS.to(DEV), **how)
    torch.cuda.synchronize()
    return got, ref


def compare(got, ref, dtype, acc=R.ACC_BACKWARD):
    for key, n in KEYS.items():
        if key not in got:
            continue
        if key in ("dA", "dbias"):
            R.close(got[key], ref[n].sum((0, 1)), "f32", acc, key, size=R.sum_size(ref[n]))
        else:
            R.close(got[key], ref[n], "f32" if key == "d_initial_state" else dtype, acc, key)


SHAPES = [(1, 1, 1, 1, 16, 16), (2, 2, 1, 2, 32, 48), (1, 64, 1, 1, 64, 64), (2, 65, 1, 1, 128, 128), (1, 129, 2, 4, 96, 80),
          (1, 70, 1, 3, 8, 8), (1, 100, 1, 2, 40, 200), (2, 150, 2, 2, 104, 256)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_plain_sequences(shape, dtype):
    x = f32(R.delta_inputs(sum(shape), *shape, dtype))
    got, ref = case(x, dtype, 1, rows=shape[0], state=True, dstate=True)
    assert set(got) == set(KEYS)
    compare(got, ref, dtype)


@pytest.mark.parametrize("dk,dv", [(4, 4), (12, 20), (44, 52), (68, 132)])
def test_widths_off_the_tiles_in_fp32(dk, dv):
    x = f32(R.delta_inputs(dk, 2, 70, 1, 2, dk, dv, "f32"))
    got, ref = case(x, "f32", 2, rows=2)
    assert "d_initial_state" not in got
    compare(got, ref, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,h,w,cls", [("bidir", 8, 9, 36), ("cross4", 7, 13, -1), ("atrous2", 9, 15, -1)])
def test_every_direction_of_the_routes(kind, h, w, cls, dtype):
    r = vs.Route(kind, h, w, cls)
    x = f32(R.delta_inputs(h * w, 2, r.tokens, 1, 2, 24, 40, dtype))
    for direction in range(r.K):
        got, ref = case(x, dtype, 3, rows=2, state=True, dstate=True, route=r, direction=direction, kind=kind, h=h, w=w)
        compare(got, ref, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,behind,heads", [([5, 0, 64, 1, 130], 0, (1, 2)), ([0, 0, 0], 3, (1, 1)),
                                                  ([63, 65, 2], 9, (2, 2))])
def test_packed_sequences(lengths, behind, heads, dtype):
    off = R.lengths_to_offsets(lengths)
    n = off[-1] + behind
    x = f32(R.delta_inputs(n, 1, n, *heads, 32, 24, dtype))
    got, ref = case(x, dtype, 4, rows=len(lengths), state=True, dstate=True, offsets=off)
    for key in ("dq", "dk", "dv", "da", "db"):
        assert (got[key][:, off[-1]:] == 0).all()
    compare(got, ref, dtype)


def test_no_bias_scales_and_a_choice_of_gradients():
    x = f32(R.delta_inputs(5, 2, 90, 2, 4, 32, 16, "f32"))
    got, ref = case(x, "f32", 5, rows=2, use_bias=False, scale=0.7, beta_scale=1.5)
    ref["bias"] = ref["a"]  # a bias of zero has the raw step's gradients
    compare(got, ref, "f32")
    d = {n: x[n].to(DEV, torch.float32) for n in x}
    dy = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(5)).to(DEV)
    args = [d[n] for n in ("q", "k", "v", "a", "b", "A")]
    for want in ([n] for n in ("dq", "dk", "dv", "da", "db", "dA", "dbias")):
        some = vs.delta_backward(*args, dy=dy, want=want, scale=0.7, beta_scale=1.5)
        assert list(some) == want and torch.equal(some[want[0]], got[want[0]])


def test_neighbouring_keys_that_point_the_same_way():
    x = f32(R.delta_inputs(6, 1, 200, 1, 1, 64, 64, "f32", correlated=True, decay=0.05))
    got, ref = case(x, "f32", 6, rows=1, state=True, dstate=True)
    compare(got, ref, "f32", 2 * R.ACC_BACKWARD)  # T's entries of both signs: as in the forward pass


def test_extreme_decays_and_strengths():
    x = f32(R.delta_inputs(7, 1, 150, 1, 4, 32, 32, "f32"))
    x["a"][0, 10] = 200.0
    x["a"][0, 70:90] = -200.0
    x["b"][0, 20:30] = -200.0
    x["b"][0, 40:50] = 200.0
    x["A"][1] = 0.0
    x["A"][2] = -1000.0
    got, ref = case(x, "f32", 7, rows=1, state=True, dstate=True)
    compare(got, ref, "f32")


def test_against_differences():
    """The library's gradient along a direction equals the change of the float64 loss along it."""
    x = f32(R.delta_inputs(8, 1, 80, 1, 2, 16, 24, "f32"))
    g = torch.Generator().manual_seed(9)
    dy = torch.randn(x["v"].shape, generator=g)
    d = {n: x[n].to(DEV, torch.float32) for n in x}
    got = vs.delta_backward(*(d[n] for n in ("q", "k", "v", "a", "b", "A", "bias")), dy=dy.to(DEV))
    for key, n in KEYS.items():
        if n == "state":
            continue
        u = torch.randn(x[n].shape, generator=g).double()

        def loss(z):
            return (R.delta_ref(dict(x, **{n: z}))[0] * dy.double()).sum()

        fd = R.finite_difference(loss, x[n], u)
        along = float((got[key].double().cpu() * u).sum())
        size = float(got[key].double().norm().cpu() * u.norm())
        # central differences in float64 at step 1e-6 are good to about 1e-9 of the loss's curvature
        assert abs(along - fd) <= (R.ACC_BACKWARD + 1e-6) * size, key


def test_runs_are_identical_strided_dy_and_graphs():
    x = f32(R.delta_inputs(11, 2, 200, 2, 4, 64, 64, "bf16"))
    d = {n: x[n].to(DEV, torch.bfloat16) for n in "qkvab"}
    d.update({n: x[n].to(DEV, torch.float32) for n in ("A", "bias")})
    args = [d[n] for n in ("q", "k", "v", "a", "b", "A", "bias")]
    wide = torch.randn(2, 200, 8, 64, device=DEV).bfloat16()
    dy = wide[:, :, 2:6]
    one, two = vs.delta_backward(*args, dy=dy), vs.delta_backward(*args, dy=dy.contiguous())
    assert all(torch.equal(one[n], two[n]) for n in one)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = vs.delta_backward(*args, dy=dy)
    wide.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    now = vs.delta_backward(*args, dy=dy)
    assert all(torch.equal(held[n], now[n]) for n in now) and not torch.equal(held["dq"], one["dq"])


def test_empty_batches_and_sequences():
    for batch, tokens in ((0, 5), (2, 0)):
        x = f32(R.delta_inputs(1, batch, tokens, 1, 1, 16, 16, "bf16"))
        d = {n: x[n].to(DEV, torch.bfloat16) for n in "qkvab"}
        A = x["A"].to(DEV, torch.float32)
        dS = torch.randn(batch, 1, 16, 16, device=DEV)
        got = vs.delta_backward(*(d[n] for n in "qkvab"), A, dy=d["v"], initial_state=torch.zeros_like(dS),
                                d_final_state=dS)
        assert torch.equal(got["d_initial_state"], dS) and (got["dA"] == 0).all() and got["dq"].shape == d["q"].shape
