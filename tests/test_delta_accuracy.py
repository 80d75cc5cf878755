"""The delta rule's float32 results hold float32 accuracy: a bound on the rms error, which the loss of
one bf16 term of one operand exceeds. (The bounds on single elements beside it are those of the worst
case, which such a loss stays within.)"""
import pytest
import torch

import delta_testlib as R

# Every product adds 16 summed indices at a time to a float32 accumulator that the tensor core
# truncates: up to 2^-23 of the running sum, 2^-24 on average, always towards 0. Four such additions of
# the large terms (64 channels or 64 steps) whose running sum grows as the root of their number
# leave (1 + sqrt 2 + sqrt 3 + 2) / 2 = 3.1 of 2^-24; the small terms are 2^-8 of that. y has been
# through three products in a row (k S, T X, P W), the state it reads through three more (k S, T X,
# k^T W): 6 * 3.1 = 19 if no error of one met another's with the other sign. The errors of a product are of
# both signs as its results are, so they add as squares after the first: below 16 of 2^-24. The backward pass
# reads W and S of the forward pass and has a chain of its own of the same length: twice that.
FORWARD = 16 * 2.0 ** -24
BACKWARD = 2 * FORWARD

SHAPE = (1, 400, 1, 2, 64, 64)
KEYS = {"dq": "q", "dk": "k", "dv": "v", "da": "a", "db": "b", "dA": "A", "dbias": "bias", "d_initial_state": "state"}


def inputs():
    """Keys that lean one way and slow decays: the state and the triangle's inverse count in every output."""
    x = R.delta_inputs(3, *SHAPE, "f32", decay=0.01)
    g = torch.Generator().manual_seed(103)
    for n in "qk":
        z = x[n] + torch.nn.functional.normalize(torch.randn(1, 1, 1, SHAPE[4], generator=g), dim=-1).double()
        x[n] = (z / z.norm(dim=-1, keepdim=True)).float().double()
    x.update(A=x["A"].float().double(), bias=x["bias"].float().double())
    x["state"] = (torch.randn(1, SHAPE[3], SHAPE[4], SHAPE[5], generator=g) * 0.5).double()
    dy = torch.randn(x["v"].shape, generator=g).double()
    return x, dy, (torch.randn(x["state"].shape, generator=g) * 0.5).double()


def gradients(f, x, dy, dstate):
    leaves = {n: t.clone().requires_grad_() for n, t in x.items()}
    y, S = f(leaves)
    got = torch.autograd.grad((y * dy).sum() + (S * dstate).sum(), list(leaves.values()))
    return (y.detach(), S.detach()), dict(zip(leaves, got))


def definition(x):
    return R.delta_ref(x, state=x["state"])


def off(got, ref):
    """rms error over rms."""
    got, ref = got.double().cpu(), ref.double()
    return float(((got - ref).square().mean() / ref.square().mean()).sqrt())


# ------------------------------------------------------------------ what a lost term does
def two_terms(x, cut):
    """The first two of three bf16 terms, cut or rounded."""
    rest, out = x.float(), torch.zeros_like(x.float())
    for _ in range(2):
        h = (rest.view(torch.int32) & -65536).view(torch.float32) if cut else rest.bfloat16().float()
        out, rest = out + h, rest - h
    return out.double()


class Lossy(torch.autograd.Function):
    """An operand of a product that has lost its third term, on the way forward or back."""

    @staticmethod
    def forward(ctx, x, cut, back):
        ctx.cut, ctx.back = cut, back
        return x.clone() if back else two_terms(x, cut)

    @staticmethod
    def backward(ctx, g):
        return (two_terms(g, ctx.cut) if ctx.back else g), None, None


def chunked(x, lost, cut, back):
    """The definition's chunked form in float64 with one operand that lost a term."""
    def operand(name, t):
        return Lossy.apply(t, cut, back) if name == lost else t

    group = x["v"].shape[2] // x["q"].shape[2]
    q, k, v = (x[n][0].repeat_interleave(1 if n == "v" else group, 1).transpose(0, 1) for n in "qkv")
    g = (x["A"] * torch.logaddexp(x["a"][0] + x["bias"], torch.zeros(()).double())).T
    beta, scale = torch.sigmoid(x["b"][0]).T[..., None], q.shape[-1] ** -0.5
    S, ys = x["state"][0], []
    for c in range(0, v.shape[1], 64):
        Q, K, V, B, G = q[:, c:c + 64], k[:, c:c + 64], v[:, c:c + 64], beta[:, c:c + 64], g[:, c:c + 64].cumsum(-1)
        low = torch.ones(G.shape[1], G.shape[1]).tril().bool()
        decay = torch.where(low, G[:, :, None] - G[:, None, :], torch.tensor(-1e30).double()).exp()
        T = operand("T", torch.linalg.inv(torch.eye(G.shape[1]).double() + B * (K @ K.mT) * decay * low.tril(-1)))
        P, eG, onward = operand("P", scale * (Q @ K.mT) * decay), G.exp()[..., None], (G[:, -1:] - G).exp()[..., None]
        entering = operand("S", S)
        W = T @ operand("X", B * (V - eG * (K @ entering)))
        if back:  # dW is one operand, the sum of both products' parts
            W = operand("W", W)
        ys.append(scale * eG * (Q @ entering) + P @ (W if back else operand("W", W)))
        S = G[:, -1, None, None].exp() * S + K.mT @ operand("D", onward * W)
    return torch.cat(ys, 1).transpose(0, 1)[None], S[None]


def test_the_chunked_form_is_the_definition():
    x, dy, dS = inputs()
    ref, grads = gradients(definition, x, dy, dS)
    got, mine = gradients(lambda z: chunked(z, None, True, False), x, dy, dS)
    assert max(off(a, b) for a, b in zip(got, ref)) < 1e-13
    assert max(off(mine[n], grads[n]) for n in grads) < 1e-12


@pytest.mark.parametrize("cut", [True, False], ids=["cut", "rounded"])
@pytest.mark.parametrize("lost", "STXPWD")
def test_a_lost_term_is_outside_the_bounds(lost, cut):
    x, dy, dS = inputs()
    ref, grads = gradients(definition, x, dy, dS)
    got, _ = gradients(lambda z: chunked(z, lost, cut, False), x, dy, dS)
    assert max(off(a, b) for a, b in zip(got, ref)) > FORWARD
    if lost in "SXWD":  # operands whose gradients are operands of the products on the way back
        _, mine = gradients(lambda z: chunked(z, lost, cut, True), x, dy, dS)
        assert max(off(mine[n], grads[n]) for n in grads) > BACKWARD


# ------------------------------------------------------------------ the kernels
@pytest.mark.gpu
def test_float32_results_hold_float32_accuracy():
    import vision_selective_state_b200 as vs

    x, dy, dS = inputs()
    (y_ref, S_ref), ref = gradients(definition, x, dy, dS)
    d = {n: t.to("cuda:0", torch.float32) for n, t in x.items()}
    args = [d[n] for n in ("q", "k", "v", "a", "b", "A", "bias")]
    y, S = vs.delta_forward(*args, initial_state=d["state"], final_state=True)
    got = vs.delta_backward(*args, dy=dy.to("cuda:0", torch.float32), initial_state=d["state"],
                            d_final_state=dS.to("cuda:0", torch.float32))
    errors = {"y": off(y, y_ref), "state": off(S, S_ref), **{key: off(got[key], ref[n]) for key, n in KEYS.items()}}
    assert errors["y"] <= FORWARD and errors["state"] <= FORWARD, errors
    # dA and dbias are sums over all tokens, whose terms are those of da
    assert all(errors[key] <= BACKWARD for key in KEYS if key not in ("dA", "dbias")), errors
