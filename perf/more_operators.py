"""Cases of the state-space operators over voxel tokens: the short causal convolution, the selective scan and the layer
norm, which make up a block of a state-space model that reads a batch's voxels as jagged sequences.

A sparse-voxel model that reads its grids as sequences takes the active voxels of a batch in canonical order: one row
per voxel, grid after grid, with an int64 offset per grid.  ``run`` computes an operator either in its plain form
(elementary torch operations in 32 bits) or, where ``own`` is true, by the calls a user makes of the package.

A case is one call of one operator ("op"), or a training step's forward and backward calls."""
import math
import random

import torch

own = False

TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


def listed():
    return [
        # one new token for each of 32 streams of a generator, before the scan's step: latency
        dict(name="conv_step", op="conv_step", streams=32, channels=1024, taps=4, type="bfloat16", silu=True),
        # the convolution over all voxels of 16 shell grids at resolution 64 (7.8k voxels each), one half of a packed
        # projection
        dict(name="conv_voxels", op="conv", grids=16, tokens=124807, channels=1024, taps=4, type="bfloat16", silu=True,
             state=False, backward=False),
        # the same in training, over a batch of grids of which some are empty: output and all gradients
        dict(name="conv_train", op="conv", grids=16, tokens=60013, channels=1536, taps=4, type="bfloat16", silu=True,
             state=False, backward=True),
        # many short sequences with odd sizes in 32 bits, states and their gradients carried through
        dict(name="conv_short_fp32", op="conv", grids=48, tokens=4099, channels=333, taps=3, type="float32", silu=False,
             state=True, backward=True),
        # one new token for each of 2 streams: the smallest recurrent step
        dict(name="scan_step", op="scan_step", streams=2, channels=512, states=16, groups=1, type="bfloat16", gate=True),
        # one new token for each of 256 streams of a generator: the states' bytes
        dict(name="scan_step_many", op="scan_step", streams=256, channels=2048, states=16, groups=1, type="bfloat16",
             gate=True),
        # one long scan prompt with the state that generation starts from: few rows, one long axis
        dict(name="scan_prompt", op="scan", grids=1, tokens=65537, channels=2048, states=16, groups=1, type="bfloat16",
             gate=True, state=True, backward=False),
        # a training step over 16 grids of unequal size, two of them empty: output and all gradients
        dict(name="scan_train", op="scan", grids=16, tokens=124807, channels=1024, states=16, groups=1, type="bfloat16",
             gate=True, state=False, backward=True),
        # a few short sequences with odd sizes in 32 bits, two groups, states and their gradients carried through
        dict(name="scan_short_fp32", op="scan", grids=5, tokens=1333, channels=202, states=12, groups=2, type="float32",
             gate=False, state=True, backward=True),
        # the norm of a block over all voxels of 16 shell grids, with the residual stream's addition
        dict(name="norm_voxels", op="norm", tokens=124807, width=1024, type="bfloat16", residual=True, backward=False),
        # the same block in training: gradients of the rows, the weight and the bias
        dict(name="norm_voxels_backward", op="norm", tokens=60013, width=1536, type="bfloat16", residual=True,
             backward=True),
        # an odd width in 32 bits: rows that start at no vector boundary
        dict(name="norm_odd", op="norm", tokens=4099, width=1001, type="float32", residual=False, backward=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv", "conv_step", "scan", "scan", "scan", "scan_step", "norm", "norm"])
    kind = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    if op == "norm":
        width = _log(rng, 64, 8192)
        width = width // 64 * 64 if rng.random() < 0.6 else width
        return dict(op=op, tokens=_log(rng, 1, min(125000, 1.2e8 / width)), width=width, type=kind,
                    residual=rng.random() < 0.6, backward=rng.random() < 0.5)
    channels = _log(rng, 24, 2048)
    channels = max(32, channels // 32 * 32) if rng.random() < 0.7 else channels
    if op == "conv_step":
        return dict(op=op, streams=_log(rng, 1, 256), channels=channels, taps=rng.choice([2, 3, 4, 4]), type=kind,
                    silu=rng.random() < 0.8)
    if op == "conv":
        return dict(op=op, grids=_log(rng, 1, 64), tokens=_log(rng, 1, min(125000, 9e7 / channels)), channels=channels,
                    taps=rng.choice([2, 3, 4, 4]), type=kind, silu=rng.random() < 0.8, state=rng.random() < 0.5,
                    backward=rng.random() < 0.5)
    groups = rng.choice([1, 1, 1, 2])
    channels = channels // groups * groups
    states = rng.choice([4, 8, 12, 16, 16, 16, 16, 24, 32, 64])
    if op == "scan_step":
        return dict(op=op, streams=_log(rng, 1, 256), channels=channels, states=min(states, 16), groups=groups, type=kind,
                    gate=rng.random() < 0.7)
    back = rng.random() < 0.5
    most = (6e8 if back else 1e9) / (channels * states)
    return dict(op=op, grids=_log(rng, 1, 48), tokens=_log(rng, 1, min(65000, most)), channels=channels, states=states,
                groups=groups, type=kind, gate=rng.random() < 0.7, state=rng.random() < 0.5, backward=back)


def work(case):
    size = 4 if case["type"] == "float32" else 2
    if case["op"] == "norm":
        n, c = case["tokens"] * case["width"], case["width"]
        if case["backward"]:
            return {"bytes": n * size * (4 if case["residual"] else 3) + 3 * c * size, "flops": 14 * n}
        return {"bytes": n * size * (4 if case["residual"] else 2) + 2 * c * size, "flops": 8 * n}
    c = case["channels"]
    if case["op"] == "conv_step":
        n, k = case["streams"] * c, case["taps"]
        return {"bytes": size * (n * 2 * k + c * (k + 1)), "flops": n * (2 * k + 4)}
    if case["op"] == "conv":
        n, k = case["tokens"] * c, case["taps"]
        ends = size * case["grids"] * (k - 1) * c * 2 if case["state"] else 0
        got = {"bytes": size * (2 * n + c * (k + 1)) + ends, "flops": n * (2 * k + 4)}
        if case["backward"]:
            got = {"bytes": got["bytes"] + size * (3 * n + 2 * c * (k + 1)) + ends, "flops": got["flops"] + n * (6 * k + 10)}
        return got
    states, groups = case["states"], case["groups"]
    rows = 4 if case["gate"] else 3  # x, dt, y and the gate
    if case["op"] == "scan_step":
        n = case["streams"]
        return {"bytes": size * n * (rows * c + 2 * groups * states) + 8 * n * c * states + 4 * c * (states + 2),
                "flops": n * c * (7 * states + 20)}
    n = case["tokens"]
    ends = 8 * case["grids"] * c * states if case["state"] else 0
    got = {"bytes": size * n * (rows * c + 2 * groups * states) + ends + 4 * c * (states + 2),
           "flops": n * c * (7 * states + 20)}
    if case["backward"]:  # x, dt, the gate and dy in, dx, ddt and the gate's gradient out, b and c and theirs
        got = {"bytes": got["bytes"] + size * n * ((7 if case["gate"] else 5) * c + 4 * groups * states) + ends
               + 8 * c * (states + 2), "flops": got["flops"] + n * c * (20 * states + 30)}
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


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    kind, op = TYPES[case["type"]], case["op"]

    def normal(*shape, scale=1.0, to=kind):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(to)

    s = {"case": case}
    if op == "norm":
        t, c = case["tokens"], case["width"]
        s["x"] = (torch.randn(t, c, generator=g, device=dev) * 2.0
                  + 0.5 * torch.randn(t, 1, generator=g, device=dev)).to(kind)
        s["weight"] = normal(c, scale=0.2, to=torch.float32).add(1.0).to(kind)
        s["bias"] = normal(c, scale=0.2)
        s["residual"] = normal(t, c, scale=3.0) if case["residual"] else None
        s["dy"] = normal(t, c, scale=0.05) if case["backward"] else None
        return s
    c = case["channels"]
    if op in ("conv", "scan"):
        n = case["tokens"]
        lengths = _lengths(case["grids"], n, seed)
        ends = [0]
        for x in lengths:
            ends.append(ends[-1] + x)
        s["lengths"] = lengths
        s["offsets"] = torch.tensor(ends, dtype=torch.int64, device=dev)
    else:
        n = case["streams"]
    if op in ("conv", "conv_step"):
        k = case["taps"]
        s["x"] = normal(n, 2 * c)[:, :c]  # a packed projection, as it comes: the convolution's half and the gate's
        s["weight"] = normal(c, k, scale=k ** -0.5)
        s["bias"] = normal(c, scale=0.2)
        s["activation"] = "silu" if case["silu"] else None
        if op == "conv_step":
            s["state"] = normal(n, k - 1, c)
        else:
            s["state"] = normal(case["grids"], k - 1, c) if case["state"] else None
            s["dy"] = normal(n, c, scale=0.5) if case["backward"] else None
            s["dstate"] = normal(case["grids"], k - 1, c) if case["backward"] and case["state"] else None
        return s
    states, groups = case["states"], case["groups"]
    s["x"] = normal(n, c)
    xz = normal(n, 2 * c)  # a packed projection whose second half is the gate
    s["z"] = xz[:, c:] if case["gate"] else None
    s["dt"] = normal(n, c, scale=0.5)
    rest = normal(n, 2 * groups * states)  # b and c come packed from their projection
    s["b"], s["c"] = (r.unflatten(1, (groups, states)) for r in rest.chunk(2, 1))
    # steps of 0.001 to 0.1 at dt = 0, rates of -1 to -states
    step = torch.exp(torch.rand(c, generator=g, device=dev) * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    rate = torch.arange(1, states + 1, device=dev, dtype=torch.float32)
    s["a"] = -(rate * torch.exp(0.1 * torch.randn(c, states, generator=g, device=dev)))
    s["d"] = 1.0 + 0.2 * torch.randn(c, generator=g, device=dev)
    if op == "scan_step":
        s["state"] = normal(n, c, states, to=torch.float32)
    else:
        s["state"] = normal(case["grids"], c, states, to=torch.float32) if case["state"] else None
        s["dy"] = normal(n, c, scale=0.5) if case["backward"] else None
        s["dstate"] = normal(case["grids"], c, states, to=torch.float32) if case["backward"] and case["state"] else None
    return s


# ---------------------------------------------------------------------------------------------------- the plain form

def _places(s):
    """Every row's grid, and its place in it."""
    at = torch.arange(s["x"].shape[0], device=s["x"].device)
    grid = torch.searchsorted(s["offsets"], at, right=True) - 1
    return grid, at - s["offsets"][grid]


def _plain_conv(s):
    case, off = s["case"], s["offsets"]
    k, c, kind = case["taps"], case["channels"], s["x"].dtype
    x, w, bias = s["x"].float(), s["weight"].float(), s["bias"].float()
    grid, place = _places(s)
    size = off[1:] - off[:-1]
    left = size[grid] - 1 - place  # rows of the grid that follow
    state = None if s["state"] is None else s["state"].float()

    def before(back):
        """The rows `back` before each one: the grid's, its state's or zeros."""
        y = torch.roll(x, back, 0)
        early = (place < back)[:, None]
        if state is None:
            return torch.where(early, 0.0, y)
        return torch.where(early, state[grid, (k - 1 - back + place).clamp(max=k - 2)], y)

    window = [x] + [before(back) for back in range(1, k)]
    pre = bias + sum(w[:, k - 1 - back] * window[back] for back in range(k))
    sig = torch.sigmoid(pre)
    out = [(pre * sig if case["silu"] else pre).to(kind)]
    if state is not None:  # the last k - 1 rows of state and grid together
        row = size[:, None] + torch.arange(k - 1, device=x.device)  # in them, counted from the state's first
        both = torch.where((row < k - 1)[..., None], state.gather(1, row.clamp(max=k - 2)[..., None].expand(-1, -1, c)),
                           x[(off[:-1, None] + row - (k - 1)).clamp(min=0)])
        out.append(both.to(kind))
    if case["backward"]:
        dpre = s["dy"].float()
        if case["silu"]:
            dpre = dpre * (sig * (1.0 + pre * (1.0 - sig)))
        ahead = [dpre] + [torch.where((left >= far)[:, None], torch.roll(dpre, -far, 0), 0.0) for far in range(1, k)]
        dx = sum(w[:, k - 1 - far] * ahead[far] for far in range(k))
        dw = torch.stack([(dpre * window[k - 1 - j]).sum(0) for j in range(k)], 1)
        first = None
        if s["dstate"] is not None:
            dlast = s["dstate"].float()
            dx = dx + torch.where((left < k - 1)[:, None], dlast[grid, (k - 2 - left).clamp(min=0)], 0.0)
            # a state's row m is the tap m - p of the row at place p, and goes on into the last rows of short grids
            rows = [[torch.where((size > p)[:, None], dpre[(off[:-1] + p).clamp(max=max(0, x.shape[0] - 1))], 0.0)
                     * w[:, m - p] for p in range(m + 1)] for m in range(k - 1)]
            first = torch.stack([sum(r) for r in rows], 1)
            row = torch.arange(k - 1, device=x.device) - size[:, None]
            first = first + torch.where((row >= 0)[..., None],
                                        dlast.gather(1, row.clamp(min=0)[..., None].expand(-1, -1, c)), 0.0)
        out += [dx.to(kind), dw.to(kind), dpre.sum(0).to(kind)] + ([first.to(kind)] if first is not None else [])
    return out


def _plain_conv_step(s):
    state, kind = s["state"], s["x"].dtype
    rows = torch.cat([state, s["x"][:, None]], 1)
    pre = s["bias"].float() + (rows.float() * s["weight"].float().t()).sum(1)
    state.copy_(rows[:, 1:])
    return [(pre * torch.sigmoid(pre) if s["case"]["silu"] else pre).to(kind), state]


def _recurrence(e, u, chunk=64):
    """h_t = e_t h_(t-1) + u_t along the first dimension, from zero; e and u are used up.  The loop is over the places
    of a chunk, all chunks at once; the chunks' ends are the same recurrence again."""
    n = e.shape[0]
    if n > chunk:
        m = -(-n // chunk)
        pad = [0, 0] * (e.dim() - 1) + [0, m * chunk - n]
        e = torch.nn.functional.pad(e, pad).unflatten(0, (m, chunk)).transpose(0, 1)
        u = torch.nn.functional.pad(u, pad).unflatten(0, (m, chunk)).transpose(0, 1)
    for t in range(1, min(n, chunk)):
        u[t] += e[t] * u[t - 1]
        e[t] *= e[t - 1]
    if n > chunk:
        ends = _recurrence(e[-1].clone(), u[-1].clone(), chunk)
        u[:, 1:] += e[:, 1:] * ends[:-1]
        u = u.transpose(0, 1).flatten(0, 1)[:n]
    return u


def _steps(s):
    """The rows' steps before and after the softplus, in 32 bits."""
    raw = s["dt"].float() + s["dt_bias"]
    return raw, raw.clamp(min=0.0) + torch.log1p(torch.exp(-raw.abs()))


def _plain_scan(s):
    case, off = s["case"], s["offsets"]
    n, kind, a = case["tokens"], s["x"].dtype, s["a"]
    per = case["channels"] // case["groups"]
    x, state = s["x"].float(), s["state"]
    raw, delta = _steps(s)
    grid, place = _places(s)
    size = off[1:] - off[:-1]
    enters, leaves = place == 0, place == size[grid] - 1
    wide = lambda r: r.float()[:, :, None].expand(-1, -1, per, -1).flatten(1, 2)  # noqa: E731  a group's rows for each channel

    def decays():
        return torch.exp(delta[..., None] * a)

    def at(where, values):  # a grid's values at one of its rows, zeros at the others
        return torch.where(where[:, None, None], values[grid], 0.0)

    e = decays()
    u = (delta * x)[..., None] * wide(s["b"])
    if state is not None:
        u += e * at(enters, state)
    h = _recurrence(torch.where(enters[:, None, None], 0.0, e), u)
    del e, u
    through = (h * wide(s["c"])).sum(-1) + s["d"] * x
    z = None if s["z"] is None else s["z"].float()
    gate = 1.0 if z is None else z * torch.sigmoid(z)
    out = [(through * gate).to(kind)]
    if state is not None:
        full = (size > 0)[:, None, None]
        out.append(torch.where(full, h[(off[1:] - 1).clamp(min=0)], state))
    if not case["backward"]:
        return out
    dy = s["dy"].float()
    ds, dz = dy * gate, None
    if z is not None:
        sig = torch.sigmoid(z)
        dz = (dy * through * (sig * (1.0 + z * (1.0 - sig)))).to(kind)
    u = ds[..., None] * wide(s["c"])
    if s["dstate"] is not None:
        u += at(leaves, s["dstate"])
    e = torch.roll(torch.where(enters[:, None, None], 0.0, decays()), -1, 0)  # the next row's; no grid's goes past its end
    g = _recurrence(e.flip(0), u.flip(0)).flip(0)
    del e, u
    by_group = lambda r: r.unflatten(1, (case["groups"], per)).sum(2)  # noqa: E731
    dc = by_group(ds[..., None] * h).to(kind)
    h = torch.where(enters[:, None, None], 0.0, torch.roll(h, 1, 0))  # the states before the rows
    if state is not None:
        h += at(enters, state)
    h *= decays()
    h *= g
    db = by_group(g * (delta * x)[..., None]).to(kind)
    into = (g * wide(s["b"])).sum(-1)
    dx = (s["d"] * ds + delta * into).to(kind)
    ddelta = (h * a).sum(-1) + x * into
    ddt = ddelta * torch.sigmoid(raw)
    h *= delta[..., None]
    out += [dx, ddt.to(kind), h.sum(0), db, dc, (ds * x).sum(0), ddt.sum(0)]
    if dz is not None:
        out.append(dz)
    if state is not None:
        row = off[:-1].clamp(max=max(0, n - 1))
        first = torch.exp(delta[row][..., None] * a) * g[row]
        out.append(torch.where(full, first, s["dstate"]))
    return out


def _plain_scan_step(s):
    case, state = s["case"], s["state"]
    per = case["channels"] // case["groups"]
    x = s["x"].float()
    delta = _steps(s)[1]
    wide = lambda r: r.float().repeat_interleave(per, 1)  # noqa: E731
    state.mul_(torch.exp(delta[..., None] * s["a"])).add_((delta * x)[..., None] * wide(s["b"]))
    y = (state * wide(s["c"])).sum(-1) + s["d"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return [y.to(s["x"].dtype), state]


def _plain_norm(s, eps=1e-5):
    case, x, w = s["case"], s["x"].float(), s["weight"].float()
    kind = s["x"].dtype
    if not case["backward"] and s["residual"] is not None:
        x = x + s["residual"].float()
    centred = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((centred * centred).mean(-1, keepdim=True) + eps)
    unit = centred * r
    if not case["backward"]:
        return [(unit * w + s["bias"].float()).to(kind)] + ([x.to(kind)] if s["residual"] is not None else [])
    dy = s["dy"].float()
    wd = dy * w
    dx = r * (wd - wd.mean(-1, keepdim=True) - unit * (wd * unit).mean(-1, keepdim=True))
    if s["residual"] is not None:  # the gradient that comes down the residual stream
        dx = dx + s["residual"].float()
    return [dx.to(kind), (dy * unit).sum(0).to(kind), dy.sum(0).to(kind)]


# ---------------------------------------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan, "scan_step": _plain_scan_step,
                "norm": _plain_norm}[op](s)
    import sparse_voxel_grid_leaf_gb300 as tb
    if op == "norm":
        if case["backward"]:
            return list(tb.layer_norm_backward(s["dy"], s["x"], s["weight"], dh=s["residual"], eps=1e-5))
        y, h = tb.layer_norm(s["x"], s["weight"], s["bias"], s["residual"], eps=1e-5)
        return [y] + ([h] if s["residual"] is not None else [])
    if op == "conv_step":
        y = tb.causal_conv_step(s["x"], s["weight"], s["state"], s["bias"], activation=s["activation"])
        return [y, s["state"]]
    if op == "scan_step":
        y = tb.selective_scan_step(s["x"], s["dt"], s["a"], s["b"], s["c"], s["state"], d=s["d"], z=s["z"],
                                   dt_bias=s["dt_bias"], softplus=True)
        return [y, s["state"]]
    if op == "conv":
        how = dict(offsets=s["offsets"], state=s["state"], activation=s["activation"])
        y, last = tb.causal_conv(s["x"], s["weight"], s["bias"], return_state=case["state"], **how)
        out = [y] + ([last] if case["state"] else [])
        if case["backward"]:
            dx, dw, dbias, first = tb.causal_conv_backward(s["dy"], s["x"], s["weight"], s["bias"], dstate=s["dstate"], **how)
            out += [dx, dw, dbias] + ([first] if case["state"] else [])
        return out
    rows = (s["x"], s["dt"], s["a"], s["b"], s["c"])
    how = dict(d=s["d"], z=s["z"], dt_bias=s["dt_bias"], softplus=True, offsets=s["offsets"], state=s["state"])
    y, last = tb.selective_scan(*rows, return_state=case["state"], **how)
    out = [y] + ([last] if case["state"] else [])
    if case["backward"]:
        dx, ddt, da, db, dc, dd, dz, dbias, first = tb.selective_scan_backward(s["dy"], *rows, dstate=s["dstate"], **how)
        out += [dx, ddt, da, db, dc, dd, dbias] + ([dz] if case["gate"] else []) + ([first] if case["state"] else [])
    return out


# -------------------------------------------------------------------------------------------- the values, in 64 bits

def _silu_and_slope(v):
    low = torch.exp(-v.abs())
    sig = torch.where(v >= 0, 1 / (1 + low), low / (1 + low))
    return v * sig, sig + v * sig * (1 - sig)


def _exact_conv(case, s):
    """Grid by grid, over the state's rows and the grid's as one sequence."""
    k, c = case["taps"], case["channels"]
    dev = s["x"].device
    w, bias = s["weight"].double(), s["bias"].double()
    x = s["x"].double()
    back = case["backward"]
    dy = s["dy"].double() if back else None
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    last, first = [], []
    dw, dbias = torch.zeros(c, k, dtype=torch.float64, device=dev), torch.zeros(c, dtype=torch.float64, device=dev)
    begin = 0
    for b, n in enumerate(s["lengths"]):
        lead = s["state"][b].double() if case["state"] else torch.zeros(k - 1, c, dtype=torch.float64, device=dev)
        row = torch.cat([lead, x[begin:begin + n]])
        last.append(row[n:])
        grad = torch.zeros_like(row)
        if back and s["dstate"] is not None:
            grad[n:] += s["dstate"][b].double()
        if n:
            view = row.unfold(0, k, 1)  # [n, c, k]
            pre = torch.einsum("tck,ck->tc", view, w) + bias
            value, slope = _silu_and_slope(pre) if case["silu"] else (pre, torch.ones_like(pre))
            y[begin:begin + n] = value
            if back:
                d = dy[begin:begin + n] * slope
                dw += torch.einsum("tc,tck->ck", d, view)
                dbias += d.sum(0)
                for j in range(k):
                    grad[j:j + n] += d * w[:, j]
        dx[begin:begin + n] = grad[k - 1:]
        first.append(grad[:k - 1])
        begin += n
    out = [y] + ([torch.stack(last)] if case["state"] else [])
    if back:
        out += [dx, dw, dbias] + ([torch.stack(first)] if case["state"] else [])
    return out


def _exact_scan(case, s):
    """The recurrence itself, token by token, for all grids and channels at once."""
    size = s["lengths"]
    grids, c, states, dev = len(size), case["channels"], case["states"], s["x"].device
    per = c // case["groups"]
    a, d = s["a"].double(), s["d"].double()
    x = s["x"].double()
    raw = s["dt"].double() + s["dt_bias"].double()
    delta = torch.logaddexp(raw, torch.zeros((), dtype=torch.float64, device=dev))
    bs, cs = s["b"].double(), s["c"].double()
    back = case["backward"]
    value, slope = _silu_and_slope(s["z"].double()) if case["gate"] else (torch.ones_like(x), None)
    order = sorted(range(grids), key=lambda b: -size[b])  # the grids still running at step t come first
    rank = torch.tensor(order, device=dev)
    start, length = s["offsets"][:-1][rank], torch.tensor([size[b] for b in order], device=dev)
    alive = [sum(1 for b in order if size[b] > t) for t in range(max(size))]

    def spread(r, rows):  # [n, groups, states] as the channels see it
        return r[rows].repeat_interleave(per, 1)

    h = s["state"].double()[rank].clone() if case["state"] else torch.zeros(grids, c, states, dtype=torch.float64, device=dev)
    inner = torch.zeros_like(x)
    kept = torch.zeros(x.shape[0], c, states, dtype=torch.float64, device=dev) if back else None  # the states before the rows
    dc = torch.zeros_like(cs)
    ds = s["dy"].double() * value if back else None
    for t, n in enumerate(alive):
        rows = start[:n] + t
        live = h[:n]
        if back:
            kept[rows] = live
        live.mul_(torch.exp(delta[rows][..., None] * a)).add_((delta[rows] * x[rows])[..., None] * spread(bs, rows))
        inner[rows] = torch.einsum("bcn,bcn->bc", live, spread(cs, rows))
        if back:
            dc[rows] = (ds[rows][..., None] * live).unflatten(1, (case["groups"], per)).sum(2)
    inner += d * x
    out = [inner * value] + ([h[torch.argsort(rank)]] if case["state"] else [])
    if not back:
        return out
    g = s["dstate"].double()[rank].clone() if s["dstate"] is not None else torch.zeros_like(h)
    dx, ddelta, da, db = d * ds, torch.zeros_like(x), torch.zeros_like(a), torch.zeros_like(bs)
    for t, n in enumerate(alive):
        rows = start[:n] + length[:n] - 1 - t
        live = g[:n]
        live.add_(ds[rows][..., None] * spread(cs, rows))
        into = torch.einsum("bcn,bcn->bc", live, spread(bs, rows))
        dx[rows] += delta[rows] * into
        db[rows] = (live * (delta[rows] * x[rows])[..., None]).unflatten(1, (case["groups"], per)).sum(2)
        live.mul_(torch.exp(delta[rows][..., None] * a))
        q = live * kept[rows]
        ddelta[rows] = x[rows] * into + (q * a).sum(-1)
        da += (q * delta[rows][..., None]).sum(0)
    draw_ = ddelta / (1 + torch.exp(-raw))
    out += [dx, draw_, da, db, dc, (ds * x).sum(0), draw_.sum(0)]
    if case["gate"]:
        out.append(s["dy"].double() * inner * slope)
    return out + ([g[torch.argsort(rank)]] if case["state"] else [])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "conv":
        return _exact_conv(case, s)
    if case["op"] == "scan":
        return _exact_scan(case, s)
    if case["op"] == "conv_step":
        row = torch.cat([s["state"].double(), s["x"].double()[:, None]], 1)
        pre = torch.einsum("nkc,ck->nc", row, s["weight"].double()) + s["bias"].double()
        return [_silu_and_slope(pre)[0] if case["silu"] else pre, row[:, 1:]]
    if case["op"] == "scan_step":
        per = case["channels"] // case["groups"]
        x = s["x"].double()
        delta = torch.logaddexp(s["dt"].double() + s["dt_bias"].double(), torch.zeros_like(x))
        b, c = (s[r].double().repeat_interleave(per, 1) for r in "bc")
        h = torch.exp(delta[..., None] * s["a"].double()) * s["state"].double() + torch.einsum("nc,ncs->ncs", delta * x, b)
        y = torch.einsum("ncs,ncs->nc", h, c) + s["d"].double() * x
        return [y * _silu_and_slope(s["z"].double())[0] if case["gate"] else y, h]
    x, w = s["x"].double(), s["weight"].double()
    if case["residual"] and not case["backward"]:
        x = x + s["residual"].double()
    spread, middle = torch.var_mean(x, -1, correction=0, keepdim=True)
    r = (spread + 1e-5).sqrt()
    u = (x - middle) / r
    if not case["backward"]:
        return [torch.addcmul(s["bias"].double(), u, w)] + ([x] if case["residual"] else [])
    # through the norm's Jacobian: (I - 1 1^T / C - u u^T / C) / r
    d = s["dy"].double()
    v = d * w
    width = case["width"]
    dx = (v - v.sum(-1, keepdim=True) / width - u * (torch.einsum("tc,tc->t", u, v)[:, None] / width)) / r
    if case["residual"]:
        dx += s["residual"].double()
    return [dx, torch.einsum("tc,tc->c", d, u), d.sum(0)]
