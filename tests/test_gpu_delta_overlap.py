"""The gated delta rule beside other work on the GPU: results do not depend on what runs at the
same time."""
import pytest
import torch

import delta_testlib as R

vs = pytest.importorskip("vision_selective_state_b200")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAMES = ("q", "k", "v", "a", "b", "A", "bias")


def on_gpu(seed, *shape, dtype):
    x = R.delta_inputs(seed, *shape, dtype)
    x = dict(x, A=x["A"].float().double(), bias=x["bias"].float().double())
    return x, [x[n].to(DEV, torch.float32 if n in ("A", "bias") else R.DT[dtype]) for n in NAMES]


def two_term_products(x):
    """Sum over j of |P_ij w_j| for every element of y of plain sequences, float64, in chunks of 64.

    y of a bf16 call has P and w in two bf16 terms, each rounded. A bf16 holds 8 bits: in steps of 2^-7
    of the power of two below a value, so the first term leaves at most 2^-8 of that power, a number whose own
    power is one less at least, and the second at most 2^-17. Left out is the product of both second
    terms, 2^-8 of each: 2^-16. Together 2^-17 + 2^-17 + 2^-16 = 2^-15 of |P_ij w_j|, summed over j."""
    group, out = x["v"].shape[2] // x["q"].shape[2], []
    for i in range(x["v"].shape[0]):
        q, k, v = (x[n][i].repeat_interleave(1 if n == "v" else group, 1).transpose(0, 1) for n in "qkv")
        g = (x["A"] * torch.logaddexp(x["a"][i] + x["bias"], torch.zeros(()).double())).T
        beta, scale, rows = torch.sigmoid(x["b"][i]).T[..., None], q.shape[-1] ** -0.5, []
        S = q.new_zeros(v.shape[0], q.shape[2], v.shape[2])
        for c in range(0, v.shape[1], 64):
            Q, K, V, B, G = q[:, c:c + 64], k[:, c:c + 64], v[:, c:c + 64], beta[:, c:c + 64], g[:, c:c + 64].cumsum(-1)
            low = torch.ones(G.shape[1], G.shape[1]).tril().bool()
            decay = torch.where(low, G[:, :, None] - G[:, None, :], torch.tensor(-1e30).double()).exp()
            T = torch.linalg.inv(torch.eye(G.shape[1]).double() + B * (K @ K.mT) * decay * low.tril(-1))
            W = T @ (B * (V - G.exp()[..., None] * (K @ S)))
            rows.append((scale * (Q @ K.mT) * decay).abs() @ W.abs())
            S = G[:, -1, None, None].exp() * S + K.mT @ ((G[:, -1:] - G).exp()[..., None] * W)
        out.append(torch.cat(rows, 1).transpose(0, 1))
    return torch.stack(out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (96, 200)])
def test_a_busy_tensor_core_changes_nothing(dk, dv, dtype):
    """The last product of a chunk reads its stage while the next chunks' copies wait for it. Other
    calls' tensor-core work on the same SMs makes that product late; the copies have to be late as well."""
    x, args = on_gpu(dk + dv, 2, 700, 2, 4, dk, dv, dtype=dtype)
    _, busy = on_gpu(1, 64, 256, 6, 6, 64, 64, dtype="bf16")
    quiet, state = vs.delta_forward(*args, final_state=True)
    ref, ref_state = R.delta_ref(x)
    size = torch.maximum(ref.abs(), ref.square().mean().sqrt())
    if dtype == "bf16":
        size = size + two_term_products(x) * (2.0 ** -15 / R.ACC_FORWARD)
    R.close(quiet, ref, dtype, R.ACC_FORWARD, "y", size=size)
    R.close(state, ref_state, "f32", R.ACC_FORWARD, "state")
    here, there = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(there):
            for _ in range(6):
                vs.delta_forward(*busy)
        with torch.cuda.stream(here):
            got = [vs.delta_forward(*args, final_state=True) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, quiet) and torch.equal(s, state) for y, s in got)
