"""Calls of the delta rule and of the norm with arguments of the wrong form raise what says so, before
anything is allocated or launched."""
import pytest
import torch

vs = pytest.importorskip("vision_selective_state_b200")


def tensors(device, batch=1, tokens=6, hk=1, hv=2, dk=16, dv=8):
    def zeros(*shape):
        return torch.zeros(shape, device=device)

    return dict(q=zeros(batch, tokens, hk, dk), k=zeros(batch, tokens, hk, dk), v=zeros(batch, tokens, hv, dv),
                a=zeros(batch, tokens, hv), b=zeros(batch, tokens, hv), A=zeros(hv), bias=zeros(hv))


def test_the_shapes_that_a_call_looks_at_first():
    from vision_selective_state_b200.delta import _rows

    x = tensors("cpu")
    assert _rows(x["q"], x["v"], None) == 1
    assert _rows(x["q"], x["v"], torch.zeros(4, dtype=torch.int32)) == 3
    for q, v, offsets, what in ((x["q"][0], x["v"], None, "are"), (x["q"], x["v"][0], None, "are"),
                                (x["q"], x["v"], torch.zeros(0, dtype=torch.int32), "one more"),
                                (x["q"], x["v"], torch.zeros(2, 2, dtype=torch.int32), "one more"),
                                (x["q"], x["v"], torch.tensor(3, dtype=torch.int32), "one more"),
                                (x["q"].expand(2, -1, -1, -1), x["v"], torch.zeros(2, dtype=torch.int32), "batch")):
        with pytest.raises(ValueError, match=what):
            _rows(q, v, offsets)


@pytest.mark.gpu
@pytest.mark.parametrize("final_state", [False, True])
def test_wrong_forms_on_the_gpu(final_state):
    x = tensors("cuda:0")

    def forward(**other):
        y = dict(x, **{n: t for n, t in other.items() if n in x})
        how = {n: t for n, t in other.items() if n not in x}
        return vs.delta_forward(*y.values(), final_state=final_state, **how)

    forward()
    for other, what in (({"v": x["v"][0]}, "v is"), ({"q": x["q"][0]}, "q and k are"),
                        ({"seq_offsets": torch.zeros(0, dtype=torch.int32, device="cuda:0")}, "one more"),
                        ({"seq_offsets": torch.tensor(0, dtype=torch.int32, device="cuda:0")}, "one more"),
                        ({"out": x["v"][:, :, :1]}, "y"), ({"out": x["v"].cpu()}, "y")):
        with pytest.raises(ValueError, match=what):
            forward(**other)
    with pytest.raises(vs.VscanError, match="dim_k 0"):
        forward(q=x["q"][..., :0], k=x["k"][..., :0])
    with pytest.raises(ValueError, match="dy"):
        vs.delta_backward(*x.values(), dy=x["v"][:, :, :1])
    with pytest.raises(vs.VscanError, match="dim_k 0"):
        vs.delta_step(*(t if n in ("A", "bias") else t[:, 0, ..., :0] if n in "qk" else t[:, 0] for n, t in x.items()),
                      state=torch.zeros(1, 2, 0, 8, device="cuda:0"))
