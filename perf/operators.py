"""Cases of the sequence operators over voxel tokens: rotary positions, the root-mean-square norm and linear
attention with a decay for each head.

A sparse-voxel model that reads its grids as sequences takes the active voxels of a batch in canonical order: one
row per voxel, grid after grid, with an int64 offset per grid.  ``run`` computes an operator either in its plain
form (elementary torch operations in 32 bits) or, where ``own`` is true, by the calls a user makes of the package.

A case is one call of one operator ("op"), or a training step's forward and backward calls."""
import math
import random

import torch

own = False

TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


def listed():
    return [
        # one new token for each of 32 streams of a generator, before its cache or state is touched: latency
        dict(name="rotary_step", op="rotary", tokens=32, heads=16, kv_heads=4, dim=128, rotated=128, axes=1,
             layout="half", type="bfloat16", span=131072, stretch=1.0, backward=False),
        # the queries and keys of 16 shell grids at resolution 64 (7.8k voxels each), turned by their voxel coordinates
        dict(name="rotary_voxels", op="rotary", tokens=124807, heads=8, kv_heads=8, dim=64, rotated=64, axes=3,
             layout="half", type="bfloat16", span=8192, stretch=1.0, backward=False),
        # the gradient of a partly rotated head in interleaved layout, with positions stretched for a longer context
        dict(name="rotary_part_backward", op="rotary", tokens=20011, heads=12, kv_heads=4, dim=96, rotated=64, axes=1,
             layout="interleaved", type="float32", span=500000, stretch=8.0, backward=True),
        # the norm before an 8-bit projection, one token for each of 16 streams: latency
        dict(name="norm_step_fp8", op="norm", tokens=16, width=2048, type="bfloat16", residual=True, fp8=True,
             backward=False),
        # the norm of a block over all voxels of 16 shell grids, with the residual stream's addition
        dict(name="norm_voxels", op="norm", tokens=124807, width=1024, type="bfloat16", residual=True, fp8=False,
             backward=False),
        # the same block in training: gradients of the rows and of the weight
        dict(name="norm_voxels_backward", op="norm", tokens=60013, width=1536, type="bfloat16", residual=True,
             fp8=False, backward=True),
        # an odd width in 32 bits: rows that start at no vector boundary
        dict(name="norm_odd", op="norm", tokens=4099, width=1001, type="float32", residual=False, fp8=False,
             backward=False),
        # one new token for each of 2 streams: the smallest recurrent step
        dict(name="attention_step", op="step", streams=2, heads=8, key=64, value=64, type="bfloat16"),
        # one new token for each of 256 streams of a generator: the states' bytes
        dict(name="attention_step_many", op="step", streams=256, heads=16, key=128, value=128, type="bfloat16"),
        # one long scan prompt with the state that generation starts from: few rows, one long axis
        dict(name="attention_prompt", op="attention", grids=1, tokens=65537, heads=16, key=128, value=128,
             type="bfloat16", state=True, backward=False),
        # a training step over 16 grids of unequal size, two of them empty: output and all gradients
        dict(name="attention_train", op="attention", grids=16, tokens=124807, heads=8, key=64, value=64,
             type="bfloat16", state=False, backward=True),
        # a few short sequences with odd head sizes in 32 bits, states and their gradients carried through
        dict(name="attention_short_fp32", op="attention", grids=5, tokens=1333, heads=3, key=40, value=72,
             type="float32", state=True, backward=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "norm", "step", "attention", "attention"])
    kind = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    if op == "rotary":
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4])
        dim = rng.choice([32, 48, 64, 80, 96, 128])
        most = int(3e8 / ((heads + kv) * dim * 4))
        return dict(op=op, tokens=_log(rng, 1, min(most, 125000)), heads=heads, kv_heads=kv, dim=dim,
                    rotated=rng.choice([dim, dim, dim // 2]), axes=rng.choice([1, 3]),
                    layout=rng.choice(["half", "interleaved"]), type=kind, span=_log(rng, 64, 1000000),
                    stretch=rng.choice([1.0, 4.0]), backward=rng.random() < 0.4)
    if op == "norm":
        width = _log(rng, 64, 8192)
        width = width // 64 * 64 if rng.random() < 0.6 else width
        back = rng.random() < 0.4
        return dict(op=op, tokens=_log(rng, 1, min(125000, 1.2e8 / width)), width=width, type=kind,
                    residual=rng.random() < 0.6, fp8=not back and rng.random() < 0.4, backward=back)
    size = lambda: rng.choice([32, 40, 64, 64, 72, 96, 128, 128])  # noqa: E731
    if op == "step":
        return dict(op=op, streams=_log(rng, 1, 256), heads=rng.randint(1, 16), key=size(), value=size(), type=kind)
    heads = rng.randint(1, 8)
    most = 65000 if kind == "bfloat16" else 20000
    return dict(op=op, grids=_log(rng, 1, 48), tokens=_log(rng, 1, most), heads=heads, key=size(), value=size(),
                type=kind, state=rng.random() < 0.5, backward=rng.random() < 0.5)


def work(case):
    size = 4 if case["type"] == "float32" else 2
    if case["op"] == "rotary":
        n = case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * n * case["dim"] * size + 4 * case["tokens"] * case["axes"],
                "flops": 3 * n * case["rotated"]}
    if case["op"] == "norm":
        n = case["tokens"] * case["width"]
        if case["backward"]:
            return {"bytes": n * size * (4 if case["residual"] else 3) + 2 * case["width"] * size, "flops": 10 * n}
        out = (1 if case["fp8"] else size) + (2 * size if case["residual"] else 0)
        return {"bytes": n * (size + out) + case["width"] * size + (4 * case["tokens"] if case["fp8"] else 0),
                "flops": 5 * n}
    dk, dv = case["key"], case["value"]
    if case["op"] == "step":
        rows = case["streams"] * case["heads"]
        return {"bytes": rows * (8 * dk * dv + (2 * dk + 2 * dv) * size), "flops": 5 * rows * dk * dv}
    rows = case["tokens"] * case["heads"]
    states = 4 * case["grids"] * case["heads"] * dk * dv if case["state"] else 0
    got = {"bytes": rows * (2 * dk + 2 * dv) * size + 2 * states, "flops": 4 * rows * dk * dv}
    if case["backward"]:
        got = {"bytes": got["bytes"] + rows * (4 * dk + 3 * dv) * size + 3 * states,
               "flops": got["flops"] + 10 * rows * dk * dv}
    return got


# ------------------------------------------------------------------------------------------------------- the inputs

def _lengths(grids, tokens, seed):
    """Unequal lengths with the given sum; from five grids on, one in eight is empty."""
    r = random.Random(seed)
    weight = [r.uniform(0.25, 2.0) for _ in range(grids)]
    if grids >= 5:
        for b in r.sample(range(grids), max(1, grids // 8)):
            weight[b] = 0.0
    cut, total, at = [0], sum(weight), 0.0
    for w in weight:
        at += w
        cut.append(int(round(tokens * at / total)))
    cut[-1] = tokens
    return [b - a for a, b in zip(cut, cut[1:])]


def _sections(pairs, axes):
    """Pairs of a head per position axis, as even as they come."""
    return [pairs // axes + (a < pairs % axes) for a in range(axes)]


def _turns(rotated, axes, stretch):
    """Turns per unit of position for each rotated pair, as 64-bit fixed-point fractions."""
    table = []
    for n in _sections(rotated // 2, axes):
        table += [int(10000.0 ** (-i / n) / stretch / (2 * math.pi) * 2.0 ** 64) for i in range(n)]
    return table


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    kind = TYPES[case["type"]]

    def normal(*shape, scale=1.0, to=kind):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(to)

    s = {"case": case}
    if case["op"] == "rotary":
        t, h, kv, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        if case["backward"]:
            s["q"], s["k"] = normal(t, h, d), normal(t, kv, d)
        else:  # a packed projection, as it comes
            qkv = normal(t, h + 2 * kv, d)
            s["q"], s["k"] = qkv[:, :h], qkv[:, h:h + kv]
        lo = 0 if case["axes"] == 1 else -(case["span"] // 2)
        shape = (t,) if case["axes"] == 1 else (t, case["axes"])
        s["positions"] = torch.randint(lo, lo + case["span"], shape, generator=g, device=dev, dtype=torch.int32)
        s["turns"] = torch.tensor(_turns(case["rotated"], case["axes"], case["stretch"]), dtype=torch.int64, device=dev)
        s["sections"] = tuple(_sections(case["rotated"] // 2, case["axes"]))
        s["axis"] = torch.tensor([a for a, n in enumerate(s["sections"]) for _ in range(n)], device=dev)
        s["amplitude"] = 0.1 * math.log(case["stretch"]) + 1.0
    elif case["op"] == "norm":
        t, c = case["tokens"], case["width"]
        s["x"] = normal(t, c, scale=2.0)
        s["weight"] = normal(c, scale=0.2, to=torch.float32).add(1.0).to(kind)
        s["residual"] = normal(t, c, scale=3.0) if case["residual"] else None
        s["dy"] = normal(t, c, scale=0.05) if case["backward"] else None
    else:
        h, dk, dv = case["heads"], case["key"], case["value"]
        s["decay"] = 1.0 - 2.0 ** -(1.0 + 9.0 * torch.arange(h, device=dev) / max(1, h - 1))
        if case["op"] == "step":
            n = case["streams"]
            s["state"] = normal(n, h, dk, dv, to=torch.float32)
        else:
            n = case["tokens"]
            lengths = _lengths(case["grids"], n, seed)
            s["longest"] = max(lengths)
            ends = [0]
            for x in lengths:
                ends.append(ends[-1] + x)
            s["offsets"] = torch.tensor(ends, dtype=torch.int64, device=dev)
            s["state"] = normal(case["grids"], h, dk, dv, to=torch.float32) if case["state"] else None
            s["do"] = normal(n, h, dv) if case["backward"] else None
            s["dstate"] = normal(case["grids"], h, dk, dv, to=torch.float32) \
                if case["backward"] and case["state"] else None
        qkv = normal(n, h * (2 * dk + dv))
        s["q"], s["k"], s["v"] = (x.unflatten(1, (h, -1)) for x in qkv.split([h * dk, h * dk, h * dv], 1))
        s["scale"] = dk ** -0.5
    return s


# ---------------------------------------------------------------------------------------------------- the plain form

def _plain_rotary(s):
    case, sign = s["case"], -1.0 if s["case"]["backward"] else 1.0
    at = s["positions"].reshape(case["tokens"], -1)
    phase = at.to(torch.int64)[:, s["axis"]] * s["turns"]  # whole turns wrap around
    angle = (phase >> 32).to(torch.float32) * (math.pi / 2 ** 31)
    cos = (torch.cos(angle) * s["amplitude"])[:, None]
    sin = (torch.sin(angle) * (s["amplitude"] * sign))[:, None]
    rotated, half = case["rotated"], case["layout"] == "half"

    def turn(x):
        y = x.float()
        r = y[..., :rotated]
        a, b = (r[..., :rotated // 2], r[..., rotated // 2:]) if half else (r[..., 0::2], r[..., 1::2])
        c, d = a * cos - b * sin, b * cos + a * sin
        r = torch.cat([c, d], -1) if half else torch.stack([c, d], -1).flatten(-2)
        return torch.cat([r, y[..., rotated:]], -1).to(x.dtype)

    return [turn(s["q"]), turn(s["k"])]


def _plain_norm(s, eps=1e-6):
    case, x, w = s["case"], s["x"].float(), s["weight"].float()
    kind = s["x"].dtype
    if case["backward"]:
        dy = s["dy"].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
        wd = dy * w
        dx = r * wd - x * (r * r * r * (wd * x).mean(-1, keepdim=True))
        if s["residual"] is not None:  # the gradient that comes down the residual stream
            dx = dx + s["residual"].float()
        return [dx.to(kind), (dy * x * r).sum(0).to(kind)]
    if s["residual"] is not None:
        x = x + s["residual"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w
    out = [x.to(kind)] if s["residual"] is not None else []
    if case["fp8"]:
        scale = y.abs().amax(-1) / 448.0
        return [(y / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale] + out
    return [y.to(kind)] + out


def _chunked(q, k, v, decay, state, first):
    """Rows [B, L, H, D] in 32 bits, by chunks: sum over j <= i of decay^(i-j) (q_i . k_j) v_j
    + decay^(i+first) q_i . state."""
    b, n, h, dk = q.shape
    c = 256 if n <= 20000 else 512
    m = -(-n // c)
    cut = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, m * c - n)).unflatten(1, (m, c)).permute(0, 3, 1, 2, 4)  # noqa: E731
    q, k, v = cut(q), cut(k), cut(v)
    at = torch.arange(c, device=q.device, dtype=torch.float32)
    pow_ = lambda e: torch.where(e >= 0, decay[:, None, None] ** e.clamp(min=0), 0.0)  # noqa: E731
    o = ((q @ k.transpose(-1, -2)) * pow_(at[:, None] - at[None, :])[:, None]) @ v
    part = (k * (decay[:, None] ** (c - 1 - at))[:, None, :, None]).transpose(-1, -2) @ v  # each chunk's own state
    step = torch.arange(m, device=q.device, dtype=torch.float32)
    before = pow_((step[:, None] - step[None, :] - 1) * c)  # from a chunk's end to a later chunk's start
    part = (before @ part.flatten(-2)).unflatten(-1, part.shape[-2:])
    o = o + (q * (decay[:, None] ** (at + 1))[:, None, :, None]) @ part
    if state is not None:
        along = (decay[:, None] ** (torch.arange(m * c, device=q.device, dtype=torch.float32) + first)).unflatten(1, (m, c))
        o = o + (q * along[..., None]) @ state[:, :, None]
    return o.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :n]


def _plain_attention(s):
    off, n = s["offsets"], max(1, s["longest"])
    size = off[1:] - off[:-1]
    at = torch.arange(n, device=off.device)
    real = at[None, :] < size[:, None]
    ahead = (off[:-1, None] + at[None, :])[real]
    rows = (off[1:, None] - 1 - at[None, :])[real]  # the same places, read from each grid's end

    def padded(x, order):
        y = torch.zeros((size.numel(), n) + x.shape[1:], device=x.device)
        y[real] = x.float()[order]
        return y

    def jagged(y, order, kind):
        x = torch.empty((order.numel(),) + y.shape[2:], device=y.device, dtype=kind)
        x[order] = y[real].to(kind)
        return x

    decay, scale, state, kind = s["decay"], s["scale"], s["state"], s["q"].dtype
    turned = lambda x: None if x is None else x.transpose(-1, -2)  # noqa: E731
    q, k, v = (padded(s[x], ahead) for x in "qkv")
    out = [jagged(_chunked(q, k, v, decay, state, 1.0) * scale, ahead, kind)]
    through = (decay[None, :] ** size[:, None])[..., None, None]
    if state is not None:
        left = torch.where(real, size[:, None] - 1 - at[None, :], 0).float()
        w = torch.where(real[..., None], decay ** left[..., None], 0.0)
        out.append(through * state + (k * w[..., None]).permute(0, 2, 3, 1) @ v.transpose(1, 2))
    if s["do"] is not None:
        do = padded(s["do"], ahead)
        out.append(jagged(_chunked(do, v, k, decay, turned(state), 1.0) * scale, ahead, kind))
        w = torch.where(real[..., None], decay ** (at[None, :, None] + 1.0), 0.0)
        first = (q * w[..., None]).permute(0, 2, 3, 1) @ do.transpose(1, 2) * scale
        q, k, v, do = (padded(s[x], rows) for x in ("q", "k", "v", "do"))
        out.append(jagged(_chunked(v, do * scale, q, decay, turned(s["dstate"]), 0.0), rows, kind))
        out.append(jagged(_chunked(k, q * scale, do, decay, s["dstate"], 0.0), rows, kind))
        if state is not None:
            out.append(first + through * s["dstate"])
    return out


def _plain_step(s):
    state = s["state"]
    state.mul_(s["decay"][:, None, None]).add_(s["k"].float()[..., None] * s["v"].float()[..., None, :])
    o = (s["q"].float()[..., None, :] @ state)[..., 0, :] * s["scale"]
    return [o.to(s["q"].dtype), state]


# ---------------------------------------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"rotary": _plain_rotary, "norm": _plain_norm, "step": _plain_step,
                "attention": _plain_attention}[op](s)
    import sparse_voxel_grid_leaf_gb300 as tb
    if op == "rotary":
        call = tb.rotary_backward if case["backward"] else tb.rotary
        return list(call(s["q"], s["k"], s["positions"], s["turns"], layout=case["layout"], sections=s["sections"],
                         amplitude=s["amplitude"]))
    if op == "norm":
        if case["backward"]:
            return list(tb.rms_norm_backward(s["dy"], s["x"], s["weight"], dh=s["residual"], eps=1e-6))
        if case["fp8"]:
            q, scale, h = tb.rms_norm_fp8(s["x"], s["weight"], s["residual"], eps=1e-6)
            return [q, scale] + ([h] if s["residual"] is not None else [])
        y, h = tb.rms_norm(s["x"], s["weight"], s["residual"], eps=1e-6)
        return [y] + ([h] if s["residual"] is not None else [])
    if op == "step":
        o = tb.linear_attention_step(s["q"], s["k"], s["v"], s["decay"], s["state"], scale=s["scale"])
        return [o, s["state"]]
    args = (s["q"], s["k"], s["v"], s["decay"], s["offsets"])
    o, last = tb.linear_attention(*args, state=s["state"], scale=s["scale"], return_state=case["state"])
    out = [o] + ([last] if case["state"] else [])
    if case["backward"]:
        dq, dk, dv, first = tb.linear_attention_backward(s["do"], *args, state=s["state"], scale=s["scale"],
                                                         dstate=s["dstate"])
        out += [dq, dk, dv] + ([first] if case["state"] else [])
    return out


# -------------------------------------------------------------------------------------------- the values, in 64 bits

def _exact_attention(case, s):
    """The recurrence itself, token by token, for all grids and heads at once."""
    off = s["offsets"].tolist()
    size = [b - a for a, b in zip(off, off[1:])]
    grids, heads, dk, dv = len(size), case["heads"], case["key"], case["value"]
    dev = s["q"].device
    decay = s["decay"].double()[None, :, None, None]
    start, length = s["offsets"][:-1], s["offsets"][1:] - s["offsets"][:-1]
    order = sorted(range(grids), key=lambda b: -size[b])  # the grids still running at step t come first
    rank = torch.tensor(order, device=dev)
    start, length = start[rank], length[rank]
    alive = [sum(1 for b in order if size[b] > t) for t in range(max(size))]
    double = {x: s[x].double() for x in ("q", "k", "v", "do") if s.get(x) is not None}
    q, k, v, scale = double["q"], double["k"], double["v"], s["scale"]
    zero = lambda: torch.zeros(grids, heads, dk, dv, dtype=torch.float64, device=dev)  # noqa: E731
    state = s["state"].double()[rank].clone() if s["state"] is not None else zero()
    o = torch.zeros_like(v)
    dq, gk, gv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    back = case["backward"]
    for t, n in enumerate(alive):
        at = start[:n] + t
        live = state[:n]
        live.mul_(decay).add_(k[at][..., None] * v[at][..., None, :])
        o[at] = torch.matmul(q[at][..., None, :], live)[..., 0, :] * scale
        if back:
            dq[at] = torch.matmul(live, double["do"][at][..., None])[..., 0] * scale
    out = [o] + ([state[torch.argsort(rank)]] if case["state"] else [])
    if back:
        grad = s["dstate"].double()[rank].clone() if s["dstate"] is not None else zero()
        for t, n in enumerate(alive):
            at = start[:n] + length[:n] - 1 - t
            live = grad[:n]
            if t:
                live.mul_(decay)
            live.add_(q[at][..., None] * (double["do"][at] * scale)[..., None, :])
            gk[at] = torch.matmul(live, v[at][..., None])[..., 0]
            gv[at] = torch.matmul(k[at][..., None, :], live)[..., 0, :]
        out += [dq, gk, gv]
        if case["state"]:
            ran = (length > 0)[:, None, None, None]
            out.append(torch.where(ran, grad * decay, grad)[torch.argsort(rank)])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(case, s)
    if case["op"] == "step":
        state = s["state"].double() * s["decay"].double()[:, None, None]
        state += torch.einsum("nhk,nhv->nhkv", s["k"].double(), s["v"].double())
        return [torch.einsum("nhk,nhkv->nhv", s["q"].double(), state) * s["scale"], state]
    if case["op"] == "rotary":
        rotated, outs = case["rotated"], []
        parts, at, col = [], s["positions"].reshape(case["tokens"], -1).double(), 0
        for a, n in enumerate(s["sections"]):
            rate = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device=at.device) / n) / case["stretch"]
            parts.append(at[:, a:a + 1] * rate)
        turn = torch.polar(torch.full((), s["amplitude"], dtype=torch.float64, device=at.device).expand(parts[0].shape[0], rotated // 2).contiguous(),
                           torch.cat(parts, 1) * (-1.0 if case["backward"] else 1.0))[:, None]
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            first = slice(0, rotated // 2) if case["layout"] == "half" else slice(0, rotated, 2)
            second = slice(rotated // 2, rotated) if case["layout"] == "half" else slice(1, rotated, 2)
            z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
            y[..., first], y[..., second] = z.real, z.imag
            outs.append(y)
        return outs
    x, w = s["x"].double(), s["weight"].double()
    if case["backward"]:  # through the norm's Jacobian: (I - u u^T / C) / r, with u the row over its root mean square
        r = (x.square().sum(-1, keepdim=True) / case["width"] + 1e-6).sqrt()
        u, d = x / r, s["dy"].double()
        along = torch.einsum("tc,tc->t", u, d * w)[:, None] / case["width"]
        dx = (d * w - u * along) / r
        if s["residual"] is not None:
            dx += s["residual"].double()
        return [dx, torch.einsum("tc,tc->c", d, u)]
    if s["residual"] is not None:
        x = x + s["residual"].double()
    y = x / (x.square().sum(-1, keepdim=True) / case["width"] + 1e-6).sqrt() * w
    rest = [x] if s["residual"] is not None else []
    if case["fp8"]:
        top = y.abs().max(-1).values / 448.0
        return [y / top[:, None], top] + rest
    return [y] + rest
