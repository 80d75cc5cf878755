"""Calls of the delta rule and of the query/key norm on another stream than the current one: what
such a call allocates and clears belongs to its own stream."""
import pytest
import torch

import delta_testlib as R

vs = pytest.importorskip("vision_selective_state_b200")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAMES = ("q", "k", "v", "a", "b", "A", "bias")
LONG = 100_000_000  # cycles: at least 50 ms of work in front of what the current stream gets next


def on_gpu(seed, *shape, dtype="bf16"):
    x = R.delta_inputs(seed, *shape, dtype)
    return [x[n].to(DEV, torch.float32 if n in ("A", "bias") else R.DT[dtype]) for n in NAMES]


def offsets(*lengths):
    return torch.tensor(R.lengths_to_offsets(lengths), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["packed", "atrous2", "plain"])
def test_rows_that_a_call_leaves_are_cleared_before_its_others_are_written(kind, dtype):
    if kind == "packed":
        args, how = on_gpu(1, 1, 200, 1, 2, 32, 32, dtype=dtype), dict(seq_offsets=offsets(70, 0, 100))
    else:
        route = vs.Route("atrous2", 9, 15) if kind == "atrous2" else None
        args = on_gpu(2, 2, 135, 1, 2, 32, 32, dtype=dtype)
        how = dict(route=route, direction=2 if route else 0)
    want, want_state = vs.delta_forward(*args, **how, final_state=True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(LONG)  # the current stream is busy: a fill queued there would come last
        got, state = vs.delta_forward(*args, **how, final_state=True, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(state, want_state)


def calls():
    args = on_gpu(3, 2, 300, 2, 2, 64, 64)
    dy = torch.randn_like(args[2])
    step = [t if n in ("A", "bias") else t[:, 0].contiguous() for n, t in zip(NAMES, args)]
    state = torch.zeros(2, 2, 64, 64, device=DEV)
    new = torch.empty_like(state)  # the caller's own: made before, not while the current stream is busy
    w = torch.ones(64, device=DEV)
    return {
        "forward": lambda **how: vs.delta_forward(*args, final_state=True, **how),
        "backward": lambda **how: vs.delta_backward(*args, dy=dy, **how),
        "step": lambda **how: vs.delta_step(*step, state=state, state_out=new, **how),
        "norm": lambda **how: vs.qk_norm(args[0], args[1], w, w, **how),
        "norm gradients": lambda **how: vs.qk_norm_backward(args[0], args[1], w, w, dyq=dy, dyk=dy, **how),
    }


@pytest.mark.parametrize("name", ["forward", "backward", "step", "norm", "norm gradients"])
def test_memory_that_the_current_stream_still_reads_is_not_written(name):
    """Tensors freed here while the current stream has yet to read them: a call on another stream,
    which does not wait for that, must not be given their memory."""
    call = calls()[name]
    want = call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for size in (1 << 12, 1 << 15, 1 << 17, 1 << 19, 1 << 22):
        old = [torch.full((size,), 7.0, device=DEV) for _ in range(16)]
        torch.cuda.synchronize()
        torch.cuda._sleep(LONG // 4)
        read = [t.clone() for t in old]
        del old
        got = call(stream=s)
        torch.cuda.synchronize()
        assert all((t == 7.0).all() for t in read), size
        pairs = zip(got.values(), want.values()) if isinstance(got, dict) else zip(got, want)
        assert all(torch.equal(g, w) for g, w in pairs)
        del read, got


@pytest.mark.parametrize("name", ["forward", "backward", "norm", "norm gradients"])
def test_results_read_on_the_current_stream_live_until_it_has_read_them(name):
    """A result made on another stream, read here and dropped: the other stream's next call must not
    be given its memory before it has been read."""
    call = calls()[name]
    want = call()
    values = lambda got: list(got.values()) if isinstance(got, dict) else list(got)  # noqa: E731
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = values(call(stream=s))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(LONG)
    read = [t.clone() for t in got]
    del got
    with torch.cuda.stream(s):
        junk = [torch.full_like(t, 9.0) for t in read for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(r, w) for r, w in zip(read, values(want))) and junk
