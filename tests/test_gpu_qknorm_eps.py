"""The query/key norm without an epsilon: rows that are not there must not reach the weights' gradients."""
import pytest
import torch

import delta_testlib as R

vs = pytest.importorskip("vision_selective_state_b200")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# as in the norm's other tests: at most 40 roundings of 2^-24 a value
ACC = 40 * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("batch,tokens,hq,hk,d,pairs", [(1, 5, 3, 1, 64, 16), (2, 33, 5, 2, 72, 0), (3, 4, 1, 1, 256, 128),
                                                        (1, 2, 1, 1, 8, 3)])
def test_no_epsilon(batch, tokens, hq, hk, d, pairs, norm, dtype):
    g = torch.Generator().manual_seed(d + pairs)
    x = {n: torch.randn(batch, tokens, h, d, generator=g).to(R.DT[dtype]) for n, h in (("q", hq), ("k", hk))}
    dy = {n: torch.randn(x[n].shape, generator=g).to(R.DT[dtype]) for n in "qk"}
    w = {n: 1 + 0.3 * torch.randn(d, generator=g) for n in "qk"}
    inv, pos = (torch.rand(pairs, generator=g), torch.arange(tokens, dtype=torch.int32)) if pairs else (None, None)
    leaves = {n: t.double().requires_grad_() for n, t in (*x.items(), ("wq", w["q"]), ("wk", w["k"]))}
    ref = {n: R.norm_ref(leaves[n], leaves["w" + n], norm, 0.0, inv, pos) for n in "qk"}
    loss = sum((ref[n] * dy[n].double()).sum() for n in "qk")
    grads = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    q, k, wq, wk, dq, dk = (t.to(DEV) for t in (x["q"], x["k"], w["q"], w["k"], dy["q"], dy["k"]))
    how = dict(norm=norm, eps=0.0, inv_freq=None if inv is None else inv.to(DEV), positions=None if pos is None else pos.to(DEV))
    for n, y in zip("qk", vs.qk_norm(q, k, wq, wk, **how)):
        R.close(y, ref[n], dtype, ACC, n)
    got = vs.qk_norm_backward(q, k, wq, wk, dyq=dq, dyk=dk, **how)
    for n in "qk":
        rows = x[n].numel() // d
        # a sum of `rows` terms dn x r, |x r| <= sqrt d (rms) or 1 (l2), |dn| <= 6: each off by ACC of itself
        R.close(got["dw" + n], grads["w" + n], "f32", ACC, "dw" + n, size=rows * 6 * (d ** 0.5 if norm == "rms" else 1.0))
        # dx = r (u - x f): the two parts cancel where x and u are parallel, each as large as r |u|
        size = 2 * 6 * 1.9 * (d ** 0.5 if norm == "rms" else 1.0) / x[n].double().norm(dim=-1).min()
        R.close(got["d" + n], grads[n], dtype, ACC, "d" + n, size=size)
