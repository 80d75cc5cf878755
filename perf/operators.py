"""Measured cases of the gated delta rule (chunked, its gradient, and the single-token step) and
of the per-head query/key norm with position rotation, with their plain forms.

The operators and their arguments, per image (or packed sequence) and value head h:

    g_t = A_h softplus(a_t + bias_h)            log decay (A_h <= 0)
    beta_t = sigmoid(b_t)                        write strength
    S_t = e^{g_t} S_{t-1} + beta_t k_t (v_t - e^{g_t} S_{t-1}^T k_t)^T      [dk, dv]
    y_t = dk^-1/2 S_t^T q_t

with q, k shared by hv / hk value heads; tokens are visited in the order of one direction of a
route, or packed sequences one after the other; and

    n = x / sqrt(sum x^2 (/ d) + eps) * w,  then pairs (p, p + r/2) of the first r channels
    rotated by position * inv_freq[p]

for q and k. `own` chooses between the plain torch forms and the framework's operators.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CHUNK = 64
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _delta(name, op, batch, h, w, cls, route, direction, hk, hv, dk, dv, dtype, state=False, ragged=False):
    return {"name": name, "op": op, "batch": batch, "h": h, "w": w, "cls": cls, "route": route,
            "direction": direction, "hk": hk, "hv": hv, "dk": dk, "dv": dv, "dtype": dtype, "state": state,
            "ragged": ragged}


def _step(name, batch, hk, hv, dk, dv, dtype):
    return {"name": name, "op": "step", "batch": batch, "hk": hk, "hv": hv, "dk": dk, "dv": dv, "dtype": dtype}


def _norm(name, op, batch, h, w, cls, hq, hk, d, rot, axes, norm, weight, dtype):
    return {"name": name, "op": op, "batch": batch, "h": h, "w": w, "cls": cls, "hq": hq, "hk": hk, "d": d,
            "rot": rot, "axes": axes, "norm": norm, "weight": weight, "dtype": dtype}


def listed():
    return [
        # one Vim-Tiny image (14x14 patches + CLS, width 384) in fp32: latency of the smallest call
        _delta("delta 14x14+cls b1 f32", "delta", 1, 14, 14, True, "bidir", 0, 6, 6, 64, 64, "f32"),
        # SS2D's column-major traversal of a 56x56 stage of width 192
        _delta("delta 56x56 cross4 b16", "delta", 16, 56, 56, False, "cross4", 2, 3, 3, 64, 64, "bf16"),
        # a packed batch of images of mixed resolutions (up to 48x48), shared key heads, states carried over
        _delta("delta packed ragged b24", "delta", 24, 48, 48, False, "none", 0, 3, 6, 64, 128, "bf16", True, True),
        # Vim-Small at 1024^2: 64x64 patches + CLS, width 768, batch 64; the reversed direction
        _delta("delta 64x64+cls b64 bf16", "delta", 64, 64, 64, True, "bidir", 1, 6, 6, 128, 128, "bf16"),
        # a training step's gradients on a small batch of 14x14 images
        _delta("grad 14x14+cls b8 bf16", "grad", 8, 14, 14, True, "bidir", 1, 6, 6, 64, 64, "bf16"),
        # odd sizes in fp32: shared key heads, head widths off the tile sizes, carried state
        _delta("grad 21x37 odd heads b3 f32", "grad", 3, 21, 37, False, "cross4", 3, 2, 4, 48, 80, "f32", True),
        # a training step's gradients at high resolution
        _delta("grad 64x64+cls b16 bf16", "grad", 16, 64, 64, True, "bidir", 0, 6, 6, 128, 128, "bf16"),
        # one token of one sequence: pure latency
        _step("step b1 f32", 1, 6, 6, 64, 64, "f32"),
        # one token of each of many sequences: the state's read and write
        _step("step b256 bf16", 256, 3, 6, 128, 128, "bf16"),
        # queries and keys of one Vim-Tiny image, as views of a packed projection
        _norm("norm 14x14+cls b1 f32", "norm", 1, 14, 14, True, 6, 6, 64, 64, 1, "rms", True, "f32"),
        # Vim-Small at 1024^2, grid rotation on half of the channels, unit-length keys
        _norm("norm 64x64+cls b64 bf16", "norm", 64, 64, 64, True, 6, 6, 128, 64, 2, "l2", False, "bf16"),
        # its gradients with learned weights
        _norm("normgrad 56x56 b16 bf16", "normgrad", 16, 56, 56, False, 12, 4, 72, 48, 2, "rms", True, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "grad", "grad", "step", "norm", "normgrad"])
    dtype = rng.choice(["f32", "bf16", "bf16"])
    wide = 4 if dtype == "f32" else 8
    if op in ("norm", "normgrad"):
        d = wide * rng.randint(16 // wide, 128 // wide)
        c = _norm("", op, 1, rng.randint(1, 64), rng.randint(1, 64), False, rng.randint(1, 12), rng.randint(1, 12), d,
                  4 * rng.randint(0, d // 4), rng.choice([1, 2]), rng.choice(["rms", "l2"]), rng.random() < 0.5, dtype)
        c["cls"] = rng.random() < 0.5
        cap = 64 * 4097 * 12 * 128 // (4 if op == "normgrad" else 1)
        c["batch"] = min(_log(rng, 1, 64), max(1, cap // (c["h"] * c["w"] * (c["hq"] + c["hk"]) * d)))
    elif op == "step":
        hk, group = rng.randint(1, 6), rng.choice([1, 1, 2, 3])
        c = _step("", _log(rng, 1, 256), hk, hk * group, wide * rng.randint(16 // wide, 128 // wide),
                  wide * rng.randint(16 // wide, 128 // wide), dtype)
        c["batch"] = max(1, min(c["batch"], 256 * 6 * 128 * 128 // (c["hv"] * c["dk"] * c["dv"])))
    else:
        hk, group = rng.randint(1, 4), rng.choice([1, 1, 2])
        route = rng.choice(["none", "bidir", "cross4"])
        directions = {"none": 1, "bidir": 2, "cross4": 4}[route]
        c = _delta("", op, 1, _log(rng, 1, 64), _log(rng, 1, 64), route == "bidir" and rng.random() < 0.5, route,
                   rng.randrange(directions), hk, hk * group, wide * rng.randint(16 // wide, 128 // wide),
                   wide * rng.randint(16 // wide, 128 // wide), dtype, rng.random() < 0.5,
                   route == "none" and rng.random() < 0.7)
        # at most a sixteenth of the largest listed call in fp32 or backward, a quarter otherwise
        cap = 64 * 4097 * 6 * 128 * 128 // (4 if op == "delta" and dtype == "bf16" else 16)
        c["batch"] = max(1, min(_log(rng, 1, 64), cap // (c["h"] * c["w"] * c["hv"] * c["dk"] * c["dv"])))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _tokens(c):
    return c["h"] * c["w"] + (1 if c["cls"] else 0)


def _lengths(c):
    """Tokens of each packed image: sizes spread over the range, one of them empty."""
    n, b = _tokens(c), c["batch"]
    lengths = [max(1, int(n * ((7 * i + 5) % b / b + 0.5 / b) ** 2)) for i in range(b)]
    if b > 2:
        lengths[1] = 0
    return lengths


def _order(c, device):
    """Token visited at each step of the route's direction."""
    n = _tokens(c)
    t = torch.arange(n, device=device)
    if c["route"] == "cross4":
        s = n - 1 - t if c["direction"] % 2 else t
        return s if c["direction"] < 2 else (s % c["h"]) * c["w"] + s // c["h"]
    return n - 1 - t if c["direction"] == 1 else t


def _unit_keys(shape, gen, device, dtype):
    """Unit vectors as a SiLU and a norm leave them: not centred, so neighbours correlate."""
    x = torch.nn.functional.silu(torch.randn(shape, generator=gen, device=device) + 0.3)
    return (x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt()).to(dtype)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device=dev) * scale

    s = {"case": dict(c)}
    if c["op"] in ("norm", "normgrad"):
        b, n, d = c["batch"], _tokens(c), c["d"]
        # q and k are neighbouring slices of one projection's output
        packed = randn(b, n, c["hq"] + c["hk"], d, scale=1.5).to(dt)
        s["q"], s["k"] = packed[:, :, :c["hq"]], packed[:, :, c["hq"]:]
        s["wq"], s["wk"] = (1 + randn(d, scale=0.2), 1 + randn(d, scale=0.2)) if c["weight"] else (None, None)
        pairs = c["rot"] // 2
        s["inv_freq"] = s["positions"] = None
        if pairs:
            per_axis = pairs // c["axes"] if pairs % c["axes"] == 0 else pairs
            s["axes"] = c["axes"] if pairs % c["axes"] == 0 else 1
            p = torch.arange(pairs, device=dev) % per_axis
            s["inv_freq"] = (10000.0 ** (-p.double() / per_axis)).float()
            t = torch.arange(c["h"] * c["w"], device=dev)
            pos = torch.stack([t // c["w"], t % c["w"]], -1) if s["axes"] == 2 else t[:, None]
            if c["cls"]:  # the class token sits in the middle, at position 0
                half = c["h"] * c["w"] // 2
                pos = torch.cat([pos[:half], torch.zeros_like(pos[:1]), pos[half:]])
            s["positions"] = pos.to(torch.int32).contiguous()
        if c["op"] == "normgrad":
            s["dq"], s["dk"] = randn(b, n, c["hq"], d).to(dt), randn(b, n, c["hk"], d).to(dt)
        return s

    hk, hv, dk, dv = c["hk"], c["hv"], c["dk"], c["dv"]
    s["A"] = -torch.exp(randn(hv, scale=0.7))
    dt0 = torch.rand(hv, generator=gen, device=dev) * 0.099 + 0.001
    s["bias"] = torch.log(torch.expm1(dt0))
    if c["op"] == "step":
        b = c["batch"]
        s["q"], s["k"] = (_unit_keys((b, hk, dk), gen, dev, dt) for _ in "qk")
        s["v"] = randn(b, hv, dv).to(dt)
        s["a"], s["b"] = randn(b, hv, scale=0.5).to(dt), randn(b, hv).to(dt)
        s["state"] = randn(b, hv, dk, dv, scale=0.3)
        return s
    b, n = c["batch"], _tokens(c)
    nseq = b
    if c["ragged"]:
        # the images' tokens one after the other in one row
        lengths = _lengths(c)
        offsets = [0]
        for x in lengths:
            offsets.append(offsets[-1] + x)
        b, n, longest = 1, offsets[-1], max(lengths)
        s["seq_offsets"] = torch.tensor(offsets, dtype=torch.int32, device=dev)
        at = torch.arange(longest, device=dev)
        first = s["seq_offsets"].long()
        live = at < (first[1:] - first[:-1])[:, None]
        s["live"], s["gather"] = live, torch.where(live, first[:-1, None] + at, 0)
    else:
        s["order"] = _order(c, dev)
    s["q"], s["k"] = (_unit_keys((b, n, hk, dk), gen, dev, dt) for _ in "qk")
    s["v"] = randn(b, n, hv, dv).to(dt)
    s["a"], s["b"] = randn(b, n, hv, scale=0.5).to(dt), randn(b, n, hv).to(dt)
    s["state"] = randn(nseq, hv, dk, dv, scale=0.3) if c["state"] else None
    if c["op"] == "grad":
        s["dy"] = randn(b, n, hv, dv).to(dt)
        s["dstate"] = randn(nseq, hv, dk, dv, scale=0.3) if c["state"] else None
    return s


# ------------------------------------------------------------------ plain forms
def _to_steps(s, x):
    """[b, n, ...] tokens to [sequence, step, ...] in visiting order; nothing behind a sequence's end."""
    if "gather" in s:
        y = x[0][s["gather"]]
        return torch.where(s["live"].reshape(s["live"].shape + (1,) * (y.dim() - 2)), y, torch.zeros_like(y))
    return x[:, s["order"]]


def _to_tokens(s, y):
    if "gather" in s:
        return y[s["live"]][None]
    back = torch.empty_like(y)
    back[:, s["order"]] = y
    return back


def _plain_steps(q, k, v, g, beta, state):
    """Chunked gated delta rule on [B, L, H, .] fp32 in visiting order; returns y and the last state."""
    B, n, H, dk = q.shape
    dv = v.shape[-1]
    C = min(CHUNK, max(n, 1))
    m = -(-n // C)
    pad = m * C - n

    def chunks(x):  # [B, n, H, .] -> [B, H, m, C, .]
        x = torch.cat([x, x.new_zeros((B, pad) + x.shape[2:])], 1) if pad else x
        return x.unflatten(1, (m, C)).movedim(3, 1)

    q, k, v, g, beta = chunks(q), chunks(k), chunks(v), chunks(g[..., None])[..., 0], chunks(beta[..., None])
    G = g.double().cumsum(-1)  # differences of these sums are exponents
    tril = torch.ones(C, C, device=q.device, dtype=torch.bool).tril()
    decay = torch.where(tril, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    eG, eD, eC = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None], G[..., -1].exp().float()
    P = (q @ k.transpose(-1, -2)) * decay
    low = beta * (k @ k.transpose(-1, -2)) * decay * tril.tril(-1)
    rows = [torch.zeros_like(low[..., 0, :])]
    rows[0][..., 0] = 1
    unit = torch.eye(C, device=q.device)
    for i in range(1, C):  # (I + low)^-1, row after row
        rows.append(unit[i] - (low[..., i, None, :i] @ torch.stack(rows, -2))[..., 0, :])
    T = torch.stack(rows, -2)
    S = q.new_zeros(B, H, dk, dv) if state is None else state
    y = []
    for t in range(m):
        kc = k[:, :, t]
        X = beta[:, :, t] * (v[:, :, t] - eG[:, :, t] * (kc @ S))
        W = T[:, :, t] @ X
        y.append(eG[:, :, t] * (q[:, :, t] @ S) + P[:, :, t] @ W)
        S = eC[:, :, t, None, None] * S + (eD[:, :, t] * kc).transpose(-1, -2) @ W
    y = torch.stack(y, 2) * dk ** -0.5
    return y.movedim(1, 3).flatten(1, 2)[:, :n], S


def _plain_delta(s, q, k, v, a, b, A, bias, state):
    c = s["case"]
    group = c["hv"] // c["hk"]
    q, k = (x.repeat_interleave(group, 2) if group > 1 else x for x in (q, k))
    x = a + bias
    g = A * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))
    beta = 1 / (1 + torch.exp(-b))
    y, S = _plain_steps(*(_to_steps(s, t) for t in (q, k, v, g, beta)), state)
    return _to_tokens(s, y), S


def _run_plain_delta(s):
    dt = DTYPES[s["case"]["dtype"]]
    y, S = _plain_delta(s, *(s[n].float() for n in "qkvab"), s["A"], s["bias"], s["state"])
    return (y.to(dt), S) if s["state"] is not None else (y.to(dt),)


def _run_plain_grad(s):
    dt = DTYPES[s["case"]["dtype"]]
    leaves = {n: s[n].float().detach().requires_grad_() for n in ("q", "k", "v", "a", "b", "A", "bias")}
    if s["state"] is not None:
        leaves["state"] = s["state"].detach().requires_grad_()
    y, S = _plain_delta(s, *leaves.values(), *(() if "state" in leaves else (None,)))
    outs, grads = [y], [s["dy"].float()]
    if s["dstate"] is not None:
        outs, grads = outs + [S], grads + [s["dstate"]]
    got = torch.autograd.grad(outs, list(leaves.values()), grads)
    return {"d" + n: x.to(dt) if n in "qkvab" else x for n, x in zip(leaves, got)}


def _run_plain_step(s):
    c = s["case"]
    group = c["hv"] // c["hk"]
    q, k = (s[n].float().repeat_interleave(group, 1) if group > 1 else s[n].float() for n in "qk")
    x = s["a"].float() + s["bias"]
    g = s["A"] * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))
    beta = 1 / (1 + torch.exp(-s["b"].float()))
    S = s["state"] * torch.exp(g)[..., None, None]
    w = beta[..., None] * (s["v"].float() - (k[..., None] * S).sum(-2))
    S = S + k[..., None] * w[..., None, :]
    return ((q[..., None] * S).sum(-2) * c["dk"] ** -0.5).to(s["v"].dtype), S


def _angles(s):
    """cos and sin of position * inv_freq; far positions need the 64-bit angle."""
    pairs = s["inv_freq"].numel()
    axis = torch.arange(pairs, device=s["inv_freq"].device) // (pairs // s["axes"])
    t = s["positions"].double()[:, axis] * s["inv_freq"].double()
    return t.cos().float()[:, None], t.sin().float()[:, None]


def _rotate(x, cos, sin):
    h = cos.shape[-1]
    u, v = x[..., :h], x[..., h:2 * h]
    return torch.cat([u * cos - v * sin, u * sin + v * cos, x[..., 2 * h:]], -1)


def _run_plain_norm(s):
    c = s["case"]
    out = []
    for name in "qk":
        x = s[name].float()
        m = x.square().sum(-1, keepdim=True)
        y = x / ((m / c["d"] if c["norm"] == "rms" else m) + EPS).sqrt()
        if s["w" + name] is not None:
            y = y * s["w" + name]
        if s["inv_freq"] is not None:
            y = _rotate(y, *_angles(s))
        out.append(y.to(s[name].dtype))
    return tuple(out)


def _run_plain_normgrad(s):
    c = s["case"]
    out = {}
    for name in "qk":
        x, dy, w = s[name].float(), s["d" + name].float(), s["w" + name]
        if s["inv_freq"] is not None:
            cos, sin = _angles(s)
            dy = _rotate(dy, cos, -sin)
        m = x.square().sum(-1, keepdim=True)
        r = 1 / ((m / c["d"] if c["norm"] == "rms" else m) + EPS).sqrt()
        if w is not None:
            out["dw" + name] = (dy * x * r).flatten(0, 2).double().sum(0).float()
            dy = dy * w
        inner = (dy * x).sum(-1, keepdim=True)
        out["d" + name] = (r * (dy - x * (r * r * (inner / c["d"] if c["norm"] == "rms" else inner)))).to(s[name].dtype)
    return out


# ------------------------------------------------------------------ the framework's operators
_routes = {}


def _route(c):
    """The route handle a program keeps, by its geometry."""
    import vision_selective_state_b200 as vs

    key = (c["route"], c["h"], c["w"], c["cls"])
    if key not in _routes:
        _routes[key] = None if c["route"] == "none" else vs.Route(c["route"], c["h"], c["w"],
                                                                  c["h"] * c["w"] // 2 if c["cls"] else -1)
    return _routes[key]


def _run_own(s):
    import vision_selective_state_b200 as vs

    c = s["case"]
    if c["op"] == "step":
        # the state is carried on in place; each pass starts from the same one, so it goes to a new tensor
        return vs.delta_step(s["q"], s["k"], s["v"], s["a"], s["b"], s["A"], s["bias"], state=s["state"],
                             state_out=torch.empty_like(s["state"]))
    if c["op"] in ("delta", "grad"):
        args = (s["q"], s["k"], s["v"], s["a"], s["b"], s["A"], s["bias"])
        how = dict(route=_route(c), direction=c["direction"], seq_offsets=s.get("seq_offsets"),
                   initial_state=s["state"])
        if c["op"] == "delta":
            out = vs.delta_forward(*args, **how, final_state=c["state"])
            return out if c["state"] else (out,)
        got = vs.delta_backward(*args, **how, dy=s["dy"], d_final_state=s["dstate"])
        names = {"dq": "dq", "dk": "dk", "dv": "dv", "da": "da", "db": "db", "dA": "dA", "dbias": "dbias"}
        if c["state"]:
            names["dstate"] = "d_initial_state"
        return {n: got[m] for n, m in names.items()}
    how = dict(norm=c["norm"], eps=EPS, inv_freq=s["inv_freq"], positions=s["positions"])
    if c["op"] == "norm":
        return vs.qk_norm(s["q"], s["k"], s["wq"], s["wk"], **how)
    got = vs.qk_norm_backward(s["q"], s["k"], s["wq"], s["wk"], dyq=s["dq"], dyk=s["dk"], **how)
    return {n: got[n] for n in (("dq", "dk", "dwq", "dwk") if c["weight"] else ("dq", "dk"))}


_PLAIN = {"delta": _run_plain_delta, "grad": _run_plain_grad, "step": _run_plain_step, "norm": _run_plain_norm,
          "normgrad": _run_plain_normgrad}


def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the least work
def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("norm", "normgrad"):
        x = c["batch"] * _tokens(c) * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": x * e * (2 if c["op"] == "norm" else 3), "flops": x * (8 if c["op"] == "norm" else 16)}
    hk, hv, dk, dv = c["hk"], c["hv"], c["dk"], c["dv"]
    rows = 2 * hk * dk + 2 * hv * dv + 2 * hv  # q, k, v, y, a, b of one token
    if c["op"] == "step":
        return {"bytes": c["batch"] * (rows * e + 8 * hv * dk * dv), "flops": c["batch"] * hv * 7 * dk * dv}
    n = sum(_lengths(c)) if c["ragged"] else c["batch"] * _tokens(c)
    states = c["batch"] * hv * dk * dv * 4 * (2 if c["state"] else 0)
    if c["op"] == "delta":
        return {"bytes": n * rows * e + states, "flops": n * hv * 6 * dk * dv}
    # q, k, v, a, b, dy in and dq, dk, dv, da, db out; k^T S and the update again, then six products with S, dS
    return {"bytes": n * e * (4 * hk * dk + 3 * hv * dv + 4 * hv) + 2 * states, "flops": n * hv * 16 * dk * dv}


# ------------------------------------------------------------------ the definitions in 64 bits
def _steps64(s, names):
    """fp64 [sequence, step, heads, ...] tensors, q and k repeated for their value heads."""
    c = s["case"]
    out = []
    for n in names:
        x = s[n].double()
        if n in "qk":
            x = x.repeat_interleave(c["hv"] // c["hk"], 2)
        out.append(_to_steps(s, x))
    return out


def _live(s, like):
    if "live" in s:
        return s["live"].double()[..., None]
    return torch.ones(like.shape[:2] + (1,), dtype=torch.float64, device=like.device)


def _gates64(s, a, b):
    x = a + s["bias"].double()
    soft = torch.logaddexp(x, torch.zeros_like(x))
    live = _live(s, a)
    return torch.exp(s["A"].double() * soft * live), torch.sigmoid(b) * live, soft, x, live


def _step64(S, q, k, v, decay, beta):
    """One step of the definition: (state, delta-corrected write)."""
    S = S * decay[..., None, None]
    w = beta[..., None] * (v - torch.einsum("bhkv,bhk->bhv", S, k))
    return S + torch.einsum("bhk,bhv->bhkv", k, w), w


def _first64(s, q, v):
    if s["state"] is not None:
        return s["state"].double()
    return torch.zeros(q.shape[0], q.shape[2], q.shape[3], v.shape[3], dtype=torch.float64, device=q.device)


def _exact_delta(s):
    q, k, v, a, b = _steps64(s, "qkvab")
    decay, beta, *_ = _gates64(s, a, b)
    S = _first64(s, q, v)
    y = torch.empty_like(v)
    for t in range(v.shape[1]):
        S, _ = _step64(S, q[:, t], k[:, t], v[:, t], decay[:, t], beta[:, t])
        y[:, t] = torch.einsum("bhkv,bhk->bhv", S, q[:, t]) * s["case"]["dk"] ** -0.5
    y = _to_tokens(s, y)
    return (y, S) if s["state"] is not None else (y,)


def _exact_grad(s):
    c = s["case"]
    q, k, v, a, b = _steps64(s, "qkvab")
    dy = _to_steps(s, s["dy"].double()) * c["dk"] ** -0.5
    decay, beta, soft, x, live = _gates64(s, a, b)
    n = v.shape[1]
    seg = max(1, math.isqrt(n))
    S = _first64(s, q, v)
    starts = []
    for t in range(n):
        if t % seg == 0:
            starts.append(S)
        S, _ = _step64(S, q[:, t], k[:, t], v[:, t], decay[:, t], beta[:, t])
    dS = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double().clone()
    dq, dk, dv, dg, db = (torch.zeros_like(z) for z in (q, k, v, a, b))
    for first in reversed(range(0, n, seg)):
        before, last = [starts[first // seg]], min(first + seg, n)
        writes = []
        for t in range(first, last):
            S, w = _step64(before[-1], q[:, t], k[:, t], v[:, t], decay[:, t], beta[:, t])
            before.append(S)
            writes.append(w)
        for t in reversed(range(first, last)):
            S0, S, w = before[t - first], before[t - first + 1], writes[t - first]
            kt, bt, gt = k[:, t], beta[:, t], decay[:, t]
            # y = S^T q
            dq[:, t] = torch.einsum("bhkv,bhv->bhk", S, dy[:, t])
            dS = dS + torch.einsum("bhk,bhv->bhkv", q[:, t], dy[:, t])
            # S = decay S0 + k w^T
            dw = torch.einsum("bhkv,bhk->bhv", dS, kt)
            D = S0 * gt[..., None, None]
            r = v[:, t] - torch.einsum("bhkv,bhk->bhv", D, kt)
            dr = bt[..., None] * dw  # w = beta r, r = v - D^T k
            dv[:, t] = dr
            db[:, t] = (dw * r).sum(-1) * bt * (1 - torch.sigmoid(b[:, t]))
            dk[:, t] = torch.einsum("bhkv,bhv->bhk", dS, w) - torch.einsum("bhkv,bhv->bhk", D, dr)
            dD = dS - torch.einsum("bhk,bhv->bhkv", kt, dr)
            dg[:, t] = (dD * D).sum((-1, -2)) * live[:, t]
            dS = dD * gt[..., None, None]
    group = c["hv"] // c["hk"]
    da = dg * s["A"].double() * torch.sigmoid(x)
    out = {"dq": dq.unflatten(2, (c["hk"], group)).sum(3), "dk": dk.unflatten(2, (c["hk"], group)).sum(3), "dv": dv,
           "da": da, "db": db}
    out = {m: _to_tokens(s, z) for m, z in out.items()}
    out["dA"], out["dbias"] = (dg * soft).sum((0, 1)), da.sum((0, 1))
    if s["state"] is not None:
        out["dstate"] = dS
    return out


def _exact_step(s):
    group = s["case"]["hv"] // s["case"]["hk"]
    q, k = (s[n].double().repeat_interleave(group, 1) for n in "qk")
    x = s["a"].double() + s["bias"].double()
    decay = torch.exp(s["A"].double() * torch.logaddexp(x, torch.zeros_like(x)))
    S, _ = _step64(s["state"].double(), q, k, s["v"].double(), decay, torch.sigmoid(s["b"].double()))
    return torch.einsum("bhkv,bhk->bhv", S, q) * s["case"]["dk"] ** -0.5, S


def _exact_norm(s):
    """The norm's value and, with dy given, its gradients: complex numbers turn the pairs."""
    c = s["case"]
    fwd, grad = [], {}
    for name in "qk":
        x = s[name].double()
        w = torch.ones(c["d"], dtype=torch.float64, device=x.device) if s["w" + name] is None else s["w" + name].double()
        length = ((x * x).mean(-1, keepdim=True) if c["norm"] == "rms" else (x * x).sum(-1, keepdim=True)) + EPS
        unit = x / length.sqrt()
        pairs = c["rot"] // 2
        turn = None
        if pairs:
            axis = torch.arange(pairs, device=x.device) * s["axes"] // pairs
            t = s["positions"].double()[:, axis] * s["inv_freq"].double()
            turn = torch.complex(t.cos(), t.sin())[:, None]

        def turned(z, by):
            if by is None:
                return z
            u = torch.complex(z[..., :pairs], z[..., pairs:2 * pairs]) * by
            return torch.cat([u.real, u.imag, z[..., 2 * pairs:]], -1)

        if c["op"] == "norm":
            fwd.append(turned(unit * w, turn))
            continue
        dn = turned(s["d" + name].double(), None if turn is None else turn.conj())
        grad["dw" + name] = (dn * unit).sum((0, 1, 2)) if s["w" + name] is not None else None
        dn = dn * w
        along = (dn * unit).mean(-1, keepdim=True) if c["norm"] == "rms" else (dn * unit).sum(-1, keepdim=True)
        grad["d" + name] = (dn - unit * along) / length.sqrt()
    return tuple(fwd) if c["op"] == "norm" else {n: x for n, x in grad.items() if x is not None}


def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "grad": _exact_grad, "step": _exact_step, "norm": _exact_norm,
            "normgrad": _exact_norm}[case["op"]](s)
