"""Query/key norm with position rotation on the GPU against the float64 form, and a run of the
operators together."""
import pytest
import torch

import delta_testlib as R

vs = pytest.importorskip("vision_selective_state_b200")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6

# float32 work on one row: the sum of up to 256 squares (8 lane levels of additions over 16
# products: 24 roundings), root, reciprocal, two products and a rotation of three roundings, the
# angle reduced in float64 and rounded once (|t| <= pi: 2^-23 absolute): 40 roundings of 2^-24
ACC = 40 * 2.0 ** -24


def inputs(seed, batch, tokens, hq, hk, d, dtype):
    g = torch.Generator().manual_seed(seed)
    x = {n: (torch.randn(batch, tokens, h, d, generator=g) * 1.5).to(R.DT[dtype]) for n, h in (("q", hq), ("k", hk))}
    x.update({"d" + n: torch.randn(x[n].shape, generator=g).to(R.DT[dtype]) for n in "qk"})
    x.update({"w" + n: 1 + 0.3 * torch.randn(d, generator=g) for n in "qk"})
    return x


def rotation(seed, batch, tokens, pairs, axes, per_image, far=1000):
    if not pairs:
        return None, None
    g = torch.Generator().manual_seed(seed + 1)
    per = pairs // axes
    inv = (10000.0 ** (-(torch.arange(pairs) % per).double() / per)).float()
    shape = ((batch,) if per_image else ()) + ((tokens,) if axes == 1 else (tokens, axes))
    return inv, torch.randint(-far, far, shape, generator=g, dtype=torch.int32)


def both(x, norm, weight, inv, pos, axes, backward=False):
    """(library, float64) outputs; with gradients of both for backward."""
    d = {n: t.to(DEV) for n, t in x.items()}
    how = dict(norm=norm, eps=EPS, inv_freq=None if inv is None else inv.to(DEV), positions=None if pos is None else pos.to(DEV))
    w = (d["wq"], d["wk"]) if weight else (None, None)
    leaves = {n: x[n].double().requires_grad_() for n in ("q", "k", "wq", "wk")}
    ref = [R.norm_ref(leaves[n], leaves["w" + n] if weight else None, norm, EPS, inv, pos, axes) for n in "qk"]
    if not backward:
        return vs.qk_norm(d["q"], d["k"], *w, **how), ref
    loss = sum((r * x["d" + n].double()).sum() for n, r in zip("qk", ref))
    names = list(leaves) if weight else ["q", "k"]
    grads = dict(zip(["d" + n for n in names], torch.autograd.grad(loss, [leaves[n] for n in names])))
    return vs.qk_norm_backward(d["q"], d["k"], *w, dyq=d["dq"], dyk=d["dk"], **how), grads


CASES = [
    # batch, tokens, hq, hk, d, pairs, axes, per_image
    (1, 1, 1, 1, 16, 8, 1, False), (2, 5, 3, 1, 64, 32, 2, False), (3, 7, 2, 4, 72, 12, 2, True),
    (2, 9, 1, 2, 128, 5, 1, False), (1, 33, 6, 6, 256, 128, 1, False), (70, 3, 2, 1, 32, 0, 1, False),
    (2, 4, 2, 2, 8, 4, 1, True), (1, 3, 1, 1, 248, 62, 2, False), (2, 2, 1, 1, 200, 6, 1, False),
    (2, 3, 5, 2, 256, 1, 1, True), (1, 2000, 1, 1, 24, 12, 1, False), (2, 3, 1, 1, 40, 16, 1, False),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm,weight", [("rms", True), ("l2", False), ("l2", True)])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(case, norm, weight, dtype):
    batch, tokens, hq, hk, d, pairs, axes, per_image = case
    x = inputs(sum(case), batch, tokens, hq, hk, d, dtype)
    inv, pos = rotation(sum(case), batch, tokens, pairs, axes, per_image)
    got, ref = both(x, norm, weight, inv, pos, axes)
    for g, r in zip(got, ref):
        R.close(g, r, dtype, ACC, "y")
    got, ref = both(x, norm, weight, inv, pos, axes, backward=True)
    assert set(got) == set(ref)
    for n in ref:
        if n.startswith("dw"):  # a sum over all rows: the errors of its terms add up
            rows = x["q"].shape[0] * x["q"].shape[1] * x[n[2:]].shape[2]
            R.close(got[n], ref[n], "f32", ACC, n, size=rows ** 0.5 * 4 * ref[n].square().mean().sqrt() + 4 * rows ** 0.5)
        else:
            # dx = r (u - x f): the two parts cancel where x and u are parallel, each as large as r |u|
            size = 2 * x[n].double().abs().max() * 1.9 * ((d ** 0.5 if norm == "rms" else 1.0) /
                                                          x[n[1:]].double().norm(dim=-1).min())
            R.close(got[n], ref[n], dtype, ACC, n, size=size)


def test_far_positions():
    x = inputs(3, 1, 6, 1, 1, 32, "f32")
    inv = torch.full((16,), 0.999, dtype=torch.float32)
    pos = torch.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64).to(torch.int32)
    got, ref = both(x, "rms", False, inv, pos, 1)
    for g, r in zip(got, ref):
        R.close(g, r, "f32", ACC, "y")


def test_zero_rows_have_finite_values_and_gradients():
    x = inputs(4, 2, 3, 2, 1, 64, "bf16")
    x["q"][0, 1] = 0
    x["k"][1, 2] = 0
    inv, pos = rotation(4, 2, 3, 32, 1, False)
    for norm in ("rms", "l2"):
        got, ref = both(x, norm, True, inv, pos, 1)
        assert (got[0][0, 1] == 0).all() and (got[1][1, 2] == 0).all()
        for g, r in zip(got, ref):
            R.close(g, r, "bf16", ACC, "y")
        got, ref = both(x, norm, True, inv, pos, 1, backward=True)
        for n in ("dq", "dk"):  # zero rows: dy w / sqrt(eps), a thousand times the others
            R.close(got[n], ref[n], "bf16", ACC, n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_views_in_place_and_streams(dtype):
    x = inputs(5, 2, 40, 3, 2, 48, dtype)
    inv, pos = (t.to(DEV) for t in rotation(5, 2, 40, 24, 2, False))
    q, k = x["q"].to(DEV), x["k"].to(DEV)
    packed = torch.cat([q, k], 2)
    views = packed[:, :, :3], packed[:, :, 3:]
    plain = vs.qk_norm(q, k, inv_freq=inv, positions=pos)
    fresh = vs.qk_norm(*views, inv_freq=inv, positions=pos)
    assert all(torch.equal(a, b) for a, b in zip(plain, fresh))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = vs.qk_norm(*views, inv_freq=inv, positions=pos, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(plain, other))
    vs.qk_norm(*views, inv_freq=inv, positions=pos, out=views)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(plain, views))


def test_empty_calls():
    for batch, tokens in ((0, 4), (3, 0)):
        q = torch.zeros(batch, tokens, 2, 16, device=DEV)
        w = torch.ones(16, device=DEV)
        assert vs.qk_norm(q, q, w, w)[0].shape == q.shape
        got = vs.qk_norm_backward(q, q, w, w, dyq=q, dyk=q)
        assert (got["dwq"] == 0).all() and (got["dwk"] == 0).all()


def test_graph_replays_the_backward_pass():
    x = inputs(6, 4, 50, 2, 2, 64, "bf16")
    d = {n: t.to(DEV) for n, t in x.items()}
    args, how = (d["q"], d["k"], d["wq"], d["wk"]), dict(dyq=d["dq"], dyk=d["dk"])
    eager = vs.qk_norm_backward(*args, **how)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = vs.qk_norm_backward(*args, **how)
    d["dq"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    now = vs.qk_norm_backward(*args, **how)
    assert all(torch.equal(held[n], now[n]) for n in now)
    assert torch.equal(held["dwq"], -eager["dwq"]) and torch.equal(held["dwk"], eager["dwk"])


def test_mixer_with_its_gradients_and_decoding():
    """One packed projection through norm and rotation, the delta rule, and back; then the last
    tokens again one at a time."""
    batch, h, w, hk, hv, dk, dv = 2, 6, 9, 2, 4, 32, 48
    route = vs.Route("cross4", h, w)
    n = route.tokens
    g = torch.Generator().manual_seed(8)
    packed = torch.randn(batch, n, 2 * hk * dk + hv * dv, generator=g)
    a, b = torch.randn(batch, n, hv, generator=g), torch.randn(batch, n, hv, generator=g)
    A, bias = -torch.rand(hv, generator=g), torch.randn(hv, generator=g)
    wq, wk = 1 + 0.2 * torch.randn(dk, generator=g), 1 + 0.2 * torch.randn(dk, generator=g)
    dy = torch.randn(batch, n, hv, dv, generator=g)
    inv = (100.0 ** (-(torch.arange(16) % 8).double() / 8)).float()
    t = torch.arange(n)
    pos = torch.stack([t // w, t % w], -1).to(torch.int32)

    def split(z):
        q, k, v = z.split([hk * dk, hk * dk, hv * dv], -1)
        return q.unflatten(2, (hk, dk)), k.unflatten(2, (hk, dk)), v.unflatten(2, (hv, dv))

    z = packed.double().requires_grad_()
    w64 = [u.double().requires_grad_() for u in (wq, wk)]
    q, k, v = split(z)
    qn = R.norm_ref(q, w64[0], "rms", EPS, inv, pos, 2)
    kn = R.norm_ref(k, w64[1], "l2", EPS, inv, pos, 2)
    x = dict(q=qn, k=kn, v=v, a=a.double(), b=b.double(), A=A.double(), bias=bias.double())
    y_ref, S_ref = R.delta_ref(x, kind="cross4", direction=2, h=h, w=w)
    dz_ref, *dw_ref = torch.autograd.grad((y_ref * dy.double()).sum(), [z, *w64])

    P, dyd = packed.to(DEV), dy.to(DEV)
    ad, bd, Ad, biasd, wqd, wkd, invd, posd = (u.to(DEV) for u in (a, b, A, bias, wq, wk, inv, pos))
    q, k, v = split(P)
    rot = dict(inv_freq=invd, positions=posd)
    q1, _ = vs.qk_norm(q, k, wqd, wkd, norm="rms", **rot)
    _, k1 = vs.qk_norm(q, k, wqd, wkd, norm="l2", **rot)
    how = dict(route=route, direction=2)
    y, S = vs.delta_forward(q1, k1, v, ad, bd, Ad, biasd, final_state=True, **how)
    R.close(y, y_ref, "f32", R.ACC_FORWARD + 4 * ACC, "y")
    R.close(S, S_ref, "f32", R.ACC_FORWARD + 4 * ACC, "state")
    got = vs.delta_backward(q1, k1, v, ad, bd, Ad, biasd, dy=dyd, **how)
    gq = vs.qk_norm_backward(q, k, wqd, wkd, dyq=got["dq"], dyk=got["dk"], norm="rms", **rot)
    gk = vs.qk_norm_backward(q, k, wqd, wkd, dyq=got["dq"], dyk=got["dk"], norm="l2", **rot)
    dq, dkey, dvalue = split(dz_ref)
    for name, have, want in (("dq", gq["dq"], dq), ("dk", gk["dk"], dkey), ("dv", got["dv"], dvalue)):
        R.close(have, want, "f32", 2 * (R.ACC_BACKWARD + 4 * ACC), name)
    for name, have, want in (("dwq", gq["dwq"], dw_ref[0]), ("dwk", gk["dwk"], dw_ref[1])):
        R.close(have, want, "f32", R.ACC_BACKWARD + 4 * ACC, name, size=batch * n * hk * want.abs().max())

    # decoding: the state before the last three steps, then one token at a time
    order = torch.tensor(R.order("cross4", 2, h, w, n))
    seq = [u[:, order.to(DEV)] for u in (q1, k1, v.contiguous(), ad, bd)]
    _, S = vs.delta_forward(*(u[:, :-3] for u in seq), Ad, biasd, final_state=True)
    for i in range(n - 3, n):
        yt, S = vs.delta_step(*(u[:, i] for u in seq), Ad, biasd, state=S)
        R.close(yt, y_ref[:, order[i]], "f32", R.ACC_FORWARD + 4 * ACC, f"token {i}")
    R.close(S, S_ref, "f32", R.ACC_FORWARD + 4 * ACC, "state after the steps")
