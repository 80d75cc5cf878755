"""Plain float64 forms of the gated delta rule and of the query/key norm with rotation, and
the inputs of their tests (CPU, torch only; nothing here comes from the library)."""
import math

import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def half_step(dtype):
    """Largest relative error of one rounding to a type."""
    return torch.finfo(DT[dtype]).eps / 2


# Accumulated error of the delta rule's float32 results, relative to the magnitude of the
# summed terms. A product of the chunked form adds at most 8 key slices x 6 split terms into
# one float32 accumulator, which the tensor core truncates: 48 * 2^-23 of the running sum.
# Four such products follow one another in a chunk (k S, T X, P W, k^T W), and the state that
# is handed on has been through the same four: 4 * 48 * 2^-23 = 2.3e-5. The backward pass
# reads W and S of the forward pass and runs four more: twice that.
ACC_FORWARD = 4 * 48 * 2.0 ** -23
ACC_BACKWARD = 2 * ACC_FORWARD


def close(got, ref, dtype, acc, what="", size=None):
    """got within a rounding to its type plus acc of the tensor's magnitude (its rms, or the
    element where that is larger, or `size`) of ref."""
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    assert torch.isfinite(got).all(), what
    rms = ref.square().mean().sqrt()
    bound = half_step(dtype) * ref.abs() + acc * (torch.maximum(ref.abs(), rms) if size is None else size)
    off = ((got - ref).abs() - bound).max()
    worst = ((got - ref).abs() / torch.maximum(ref.abs(), rms).clamp(min=1e-300)).max()
    assert off <= 0, f"{what}: error {worst:.3e} of the magnitude, bound {half_step(dtype):.1e} + {acc:.1e}"


# ------------------------------------------------------------------ orders
def order(kind, direction, h, w, tokens):
    """Token visited at each step (-1: a padding slot of the atrous grid)."""
    if kind is None:
        return list(range(tokens))
    if kind == "bidir":
        s = list(range(tokens))
        return s if direction == 0 else s[::-1]
    if kind == "cross4":
        s = [r * w + c for r in range(h) for c in range(w)]
        if direction >= 2:
            s = [r * w + c for c in range(w) for r in range(h)]
        return s[::-1] if direction % 2 else s
    rows, cols = (h + 1) // 2, (w + 1) // 2
    m, n = direction & 1, direction >> 1
    cells = ([(r, c) for c in range(cols) for r in range(rows)] if direction & 1 else
             [(r, c) for r in range(rows) for c in range(cols)])
    out = []
    for r, c in cells:
        y, x = 2 * r + m, 2 * c + n
        out.append(y * w + x if y < h and x < w else -1)
    return out


# ------------------------------------------------------------------ inputs
def delta_inputs(seed, batch, tokens, hk, hv, dk, dv, dtype, correlated=False, decay=1.0):
    """Float64 inputs whose values the I/O type holds exactly."""
    g = torch.Generator().manual_seed(seed)

    def draw(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).double()

    x = {}
    for n in "qk":
        z = torch.randn(batch, tokens, hk, dk, generator=g)
        if correlated:  # keys of one image that point nearly the same way
            z = z * 0.2 + torch.randn(1, 1, hk, dk, generator=g)
        x[n] = (z / z.norm(dim=-1, keepdim=True).clamp(min=1e-6)).to(DT[dtype]).double()
    x["v"] = draw(batch, tokens, hv, dv)
    x["a"], x["b"] = draw(batch, tokens, hv, scale=0.5), draw(batch, tokens, hv)
    x["A"] = -(torch.rand(hv, generator=g) * 2 * decay).double()
    x["bias"] = (torch.randn(hv, generator=g) - 1).double()
    return x


# ------------------------------------------------------------------ the definition
def _one(q, k, v, a, b, A, bias, S, scale, beta_scale):
    """Steps [L, heads, .] of one sequence in float64; q and k per value head. A and bias are
    per head, or per step and head."""
    x = a + (0 if bias is None else bias)
    decay = torch.exp(A * torch.logaddexp(x, torch.zeros_like(x)))
    beta = beta_scale * torch.sigmoid(b)
    ys = []
    for t in range(q.shape[0]):
        S = S * decay[t, :, None, None]
        w = beta[t, :, None] * (v[t] - (k[t, :, :, None] * S).sum(1))
        S = S + k[t, :, :, None] * w[:, None, :]
        ys.append(scale * (q[t, :, :, None] * S).sum(1))
    return (torch.stack(ys) if ys else v.new_zeros(v.shape)), S


def delta_ref(x, *, kind=None, direction=0, h=0, w=0, offsets=None, scale=None, beta_scale=1.0, state=None,
              use_bias=True):
    """(y, final state) of the definition, token by token. Rows that no step visits are 0."""
    q, k, v = x["q"], x["k"], x["v"]
    group = v.shape[2] // q.shape[2]
    q, k = q.repeat_interleave(group, 2), k.repeat_interleave(group, 2)
    scale = q.shape[3] ** -0.5 if scale is None else scale
    bias = x["bias"] if use_bias else None
    y = torch.zeros_like(v)
    seqs = []
    if offsets is not None:
        seqs = [(0, list(range(o0, o1))) for o0, o1 in zip(offsets[:-1], offsets[1:])]
    else:
        o = order(kind, direction, h, w, v.shape[1])
        seqs = [(i, o) for i in range(v.shape[0])]
    states = []
    for n, (i, rows) in enumerate(seqs):
        idx = torch.tensor(rows, dtype=torch.long)
        live = idx >= 0
        at = idx.clamp(min=0)

        def take(z):
            s = z[i][at]
            return s * live.reshape((-1,) + (1,) * (s.dim() - 1))

        S0 = v.new_zeros(v.shape[2], q.shape[3], v.shape[3]) if state is None else state[n]
        A, c = (z if z is None or z.dim() == 1 else z[i][at] for z in (x["A"], bias))
        ys, S = _one(take(q), take(k), take(v), take(x["a"]), take(x["b"]), A, c, S0, scale, beta_scale)
        y = y.index_put((torch.tensor(i), at[live]), ys[live])
        states.append(S)
    return y, (torch.stack(states) if states else v.new_zeros(0, v.shape[2], q.shape[3], v.shape[3]))


# ------------------------------------------------------------------ norm and rotation
def norm_ref(x, weight, norm, eps, inv_freq=None, positions=None, axes=1):
    """[batch, tokens, heads, d] float64 -> normalised, weighted, rotated."""
    d = x.shape[-1]
    m = x.square().sum(-1, keepdim=True)
    y = x / torch.sqrt((m / d if norm == "rms" else m) + eps)
    if weight is not None:
        y = y * weight
    if inv_freq is not None and inv_freq.numel():
        pairs = inv_freq.numel()
        per = pairs // axes
        pos = positions.double().reshape((-1, x.shape[1], axes))
        cols = []
        for p in range(pairs):
            angle = pos[:, :, p // per] * inv_freq[p].double()
            cols.append(angle)
        t = torch.stack(cols, -1)[:, :, None]
        u, v = y[..., :pairs], y[..., pairs:2 * pairs]
        y = torch.cat([u * t.cos() - v * t.sin(), u * t.sin() + v * t.cos(), y[..., 2 * pairs:]], -1)
    return y


def sum_size(terms):
    """Magnitude of a sum over tokens, per head: each term [batch, tokens, heads] is off by its
    accumulated error, relative to the larger of itself and the terms' rms, and the errors of a
    sum add up whatever its terms' signs, so a sum that cancels is off by more of its own value."""
    rms = terms.square().mean().sqrt()
    return torch.maximum(terms.abs(), rms).sum((0, 1))


def finite_difference(f, x, direction, eps=1e-6):
    """Central difference of a scalar function along a direction."""
    return float((f(x + eps * direction) - f(x - eps * direction)) / (2 * eps))


def lengths_to_offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


__all__ = [n for n in dir() if not n.startswith("_") and n not in ("math", "torch")]
