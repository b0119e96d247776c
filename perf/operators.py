"""Performance cases of the LayerNorm, multi-axis rotary and Muon operators.

Each case names one operator with its sizes. ``prepare`` makes the inputs a
training step has on the GPU before the call, ``run`` makes one pass (the
operator's plain form, or the library's call when ``own`` is true), ``work``
counts the bytes and floating-point operations that the operator cannot do
without, and ``exact`` computes the same outputs from the definitions in
float64.

Operators
- ``ln_fwd``  y = (x - mean) rstd g + b over rows of H, with mean and rstd.
- ``ln_bwd``  dx (+ the residual branch's gradient), dg, db from dy and the saved statistics.
- ``mrope``   rotate-half rotary positions with one position per token and axis; ``inverse`` is its adjoint.
- ``muon``    momentum step and Newton-Schulz orthogonalisation of a weight matrix's gradient.
"""
import math

import torch

own = False

EPS = 1e-6
MOMENTUM, STEPS, MUON_EPS = 0.95, 5, 1e-7
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315

# Largest sizes of the drawn cases (those of the listed ones): elements of a norm's
# or a rotation's tensor, and multiply-adds of one pass over a matrix of the optimizer.
MAX_NORM = 98304 * 3584
MAX_ROPE = 98304 * 32 * 128
MAX_MUON = 3584 * 3584 * 18944


def listed():
    return [
        # the small parity layer of the tests: 2 x 128 tokens of width 256, where the launch is what counts
        dict(name="ln_fwd 256x256", op="ln_fwd", rows=256, H=256, ld=256, affine=True),
        # rows of an odd width inside wider rows (a slice of a fused buffer), no multiple of a vector
        dict(name="ln_fwd 4999x1153 in 1160", op="ln_fwd", rows=4999, H=1153, ld=1160, affine=True),
        # the default workload's batch: 96 x 1024 tokens of width 3584
        dict(name="ln_fwd 98304x3584", op="ln_fwd", rows=98304, H=3584, ld=3584, affine=True),
        dict(name="ln_bwd 256x256", op="ln_bwd", rows=256, H=256, ld=256, affine=True, dres=False),
        # 8 x 1024 tokens, with the residual branch's gradient added on the way
        dict(name="ln_bwd 8192x3584 +res", op="ln_bwd", rows=8192, H=3584, ld=3584, affine=True, dres=True),
        # 32 x 1024 tokens of width 5120
        dict(name="ln_bwd 32768x5120", op="ln_bwd", rows=32768, H=5120, ld=5120, affine=True, dres=False),
        # one short text sequence through the parity layer's heads
        dict(name="mrope 128 tok 6x64", op="mrope", rows=128, heads=6, d=64, ld=512, axes=3, s0=8, s1=12, s2=12,
             interleaved=False, per_axis=False, inverse=False, theta=1e6),
        # the patches of ragged images in a tower: heads of 80, a frequency ladder for each of height and width, backward
        dict(name="mrope 10003 tok 32x80 inv", op="mrope", rows=10003, heads=32, d=80, ld=3840, axes=2, s0=20, s1=20,
             s2=0, interleaved=False, per_axis=True, inverse=True, theta=1e4),
        # the default workload's tokens as video frames: 28 query and 4 key heads of 128 inside the fused qkv rows
        dict(name="mrope 98304 tok 32x128", op="mrope", rows=98304, heads=32, d=128, ld=4608, axes=3, s0=16, s1=24,
             s2=24, interleaved=False, per_axis=False, inverse=False, theta=1e6),
        # the parity layer's gate projection, taller than wide
        dict(name="muon 688x256", op="muon", rows=688, cols=256, nesterov=True),
        # a key projection of the 7B layer
        dict(name="muon 512x3584", op="muon", rows=512, cols=3584, nesterov=True),
        # the down projection of the 7B layer
        dict(name="muon 3584x18944", op="muon", rows=3584, cols=18944, nesterov=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "mrope", "muon"])
    if op in ("ln_fwd", "ln_bwd"):
        H = _log(rng, 16, 8192)
        if rng.random() < 0.5:
            H = max(8, H // 8 * 8)
        # the backward moves more an element: half the forward's largest size
        rows = _log(rng, 1, min(98304, MAX_NORM // (2 * H)))
        ld = H if rng.random() < 0.5 else H + rng.choice([1, 8, 40, 256])
        c = dict(op=op, rows=rows, H=H, ld=ld, affine=rng.random() < 0.8)
        if op == "ln_bwd":
            c["dres"] = rng.random() < 0.5
        return c
    if op == "mrope":
        d = rng.choice([32, 64, 72, 80, 96, 128, 128, 192, 256])
        axes = rng.choice([1, 2, 3, 3, 4])
        pairs = d // 2 if rng.random() < 0.7 else max(axes, d // 4)  # a quarter rotates a part of the head only
        cuts = sorted(rng.sample(range(1, pairs), axes - 1)) if axes > 1 else []
        s = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        heads = rng.randint(1, 40)
        rows = _log(rng, 1, min(98304, MAX_ROPE // (heads * d)))
        c = dict(op=op, rows=rows, heads=heads, d=d, ld=heads * d + rng.choice([0, 0, 3, 8, d, 2 * d]), axes=axes)
        c.update({"s%d" % i: v for i, v in enumerate(s)})
        c.update(interleaved=rng.random() < 0.3, per_axis=rng.random() < 0.3, inverse=rng.random() < 0.5,
                 theta=rng.choice([1e4, 1e6]))
        return c
    short = _log(rng, 2, 2048)
    long = _log(rng, short, max(short + 1, min(20000, MAX_MUON // (4 * short * short))))
    rows, cols = (short, long) if rng.random() < 0.5 else (long, short)
    return dict(op="muon", rows=rows, cols=cols, nesterov=rng.random() < 0.8)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _strided(rows, cols, ld):
    """An uninitialised [rows, cols] bf16 view of rows of ld elements."""
    return torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")[:, :cols]


def _normal(g, rows, cols, ld, std=1.0):
    t = _strided(rows, cols, ld)
    t.copy_(torch.randn(rows, cols, generator=g, device="cuda").mul_(std))
    return t


def _norm_inputs(case, g):
    rows, H, ld = case["rows"], case["H"], case["ld"]
    s = {"x": _normal(g, rows, H, ld)}
    # a residual stream: each row at a level and scale of its own
    s["x"].mul_(torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda")))
    s["x"].add_(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    if case["affine"]:
        s["g"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()
        s["b"] = (0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    else:
        s["g"] = s["b"] = None
    return s


def _sections(case):
    return [case["s%d" % i] for i in range(case["axes"])]


def _pair_axes(case):
    """(axis, index within the axis) of each rotated pair: runs of the sections, or dealt out in turn."""
    s = _sections(case)
    if not case["interleaved"]:
        return [(a, j) for a in range(len(s)) for j in range(s[a])]
    out, left = [], list(s)
    while any(left):
        for a in range(len(s)):
            if left[a]:
                out.append((a, s[a] - left[a]))
                left[a] -= 1
    return out


def _frequencies(case):
    """Per pair: its axis and, in float64, the angle of a position of one."""
    table, s = _pair_axes(case), _sections(case)
    if case["per_axis"]:
        freq = [case["theta"] ** (-j / s[a]) for a, j in table]
    else:
        freq = [case["theta"] ** (-i / len(table)) for i in range(len(table))]
    return [a for a, _ in table], freq


def _positions(case, g):
    """Axis 0 counts time or tokens, the others walk a grid of odd width, as a frame's patches do; text
    behind the images goes on far out, the same on every axis."""
    rows, axes = case["rows"], case["axes"]
    t = torch.arange(rows, device="cuda")
    width = int(torch.randint(23, 61, (1,), generator=g, device="cuda"))
    high = int(torch.randint(17, 41, (1,), generator=g, device="cuda"))
    far = int(torch.randint(0, 200000, (1,), generator=g, device="cuda"))
    walk = [t // (width * high), (t // width) % high, t % width, t % 7]
    if axes <= 2:  # no time axis: height and width, or a plain count
        walk = [t // width, t % width] if axes == 2 else [t]
    pos = torch.stack(walk[:axes])
    text = t >= rows - rows // 4
    return torch.where(text[None], far + t[None], pos).to(torch.int32).contiguous()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op in ("ln_fwd", "ln_bwd"):
        rows, H, ld = case["rows"], case["H"], case["ld"]
        s.update(_norm_inputs(case, g))
    if op == "ln_fwd":
        s["y"] = _strided(rows, H, ld)
        s["mean"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        s["rstd"] = torch.empty_like(s["mean"])
    elif op == "ln_bwd":
        xf = s["x"].float()
        var, mean = torch.var_mean(xf, dim=1, unbiased=False)
        s["mean"], s["rstd"] = mean, torch.rsqrt(var + EPS)
        s["dy"] = _normal(g, rows, H, ld, 0.1)
        s["dres"] = _normal(g, rows, H, ld, 0.1) if case["dres"] else None
        s["dx"] = _strided(rows, H, ld)
        s["dg"] = torch.empty(H, dtype=torch.float32, device="cuda")
        s["db"] = torch.empty_like(s["dg"])
    elif op == "mrope":
        rows, width = case["rows"], case["heads"] * case["d"]
        s["x"] = _normal(g, rows, width, case["ld"])
        s["y"] = _strided(rows, width, case["ld"])
        s["pos"] = _positions(case, g)
        axis, freq = _frequencies(case)
        s["axis"] = torch.tensor(axis, device="cuda")
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
    else:
        rows, cols = case["rows"], case["cols"]
        # a weight gradient: a few strong directions of falling strength over noise, in rows and columns of unlike scale
        rank = min(16, rows, cols)
        left = torch.randn(rows, rank, generator=g, device="cuda")
        right = torch.randn(rank, cols, generator=g, device="cuda")
        fall = 0.5 / torch.arange(1, rank + 1, device="cuda")
        row = torch.exp(0.3 * torch.randn(rows, 1, generator=g, device="cuda"))
        for name in ("g", "m"):
            noise = torch.randn(rows, cols, generator=g, device="cuda")
            s[name] = ((left * fall) @ right + 0.5 * noise) * row * 1e-3
        s["m"] *= 10.0
        s["m_out"] = torch.empty_like(s["m"])
        s["o"] = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    if own:
        from host_offloaded_layer_b200 import _lib as L

        s["stream"] = torch.cuda.current_stream()
        nbytes = 0
        if op == "ln_bwd":
            nbytes = L.mt_layernorm_bwd_workspace_bytes(case["rows"], case["H"])
        elif op == "muon":
            nbytes = L.mt_muon_workspace_bytes(case["rows"], case["cols"])
            s["cfg"] = L.make_muon_cfg(momentum=MOMENTUM, nesterov=case["nesterov"], steps=STEPS, eps=MUON_EPS, scale=1.0)
        elif op == "mrope":
            s["sections"] = _sections(case)
        s["ws_bytes"] = nbytes
        s["ws"] = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _plain_ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(dim=1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(dim=1) + EPS)
    y = c * rstd[:, None]
    if s["g"] is not None:
        y = y * s["g"].float() + s["b"].float()
    return {"y": y.bfloat16(), "mean": mean, "rstd": rstd}


def _plain_ln_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    w = dy if s["g"] is None else dy * s["g"].float()
    dx = rstd * (w - w.mean(dim=1, keepdim=True) - xh * (w * xh).mean(dim=1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.bfloat16(), "dg": (dy * xh).sum(dim=0), "db": dy.sum(dim=0)}


def _plain_mrope(s):
    case = s["case"]
    rows, heads, d, pairs = case["rows"], case["heads"], case["d"], s["freq"].numel()
    angle = s["pos"].index_select(0, s["axis"]).t().double() * s["freq"]  # [rows, pairs]
    cos = torch.cos(angle).float()[:, None]
    sin = torch.sin(angle).float()[:, None]
    if case["inverse"]:
        sin = -sin
    x = s["x"].reshape(rows, heads, d)
    a, b = x[..., :pairs].float(), x[..., pairs:2 * pairs].float()
    y = torch.cat([(a * cos - b * sin).bfloat16(), (b * cos + a * sin).bfloat16(), x[..., 2 * pairs:]], dim=-1)
    return {"y": y.reshape(rows, heads * d)}


def _plain_muon(s):
    m = MOMENTUM * s["m"] + s["g"]
    u = s["g"] + MOMENTUM * m if s["case"]["nesterov"] else m
    x = u / (torch.sqrt((u * u).sum()) + MUON_EPS)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    for _ in range(STEPS):
        a = x @ x.t()
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    if tall:
        x = x.t()
    return {"o": x.bfloat16(), "m": m}


def _own_ln_fwd(s):
    from host_offloaded_layer_b200 import _lib as L

    c = s["case"]
    L.mt_layernorm_fwd(s["x"], c["ld"], s["g"], s["b"], s["y"], c["ld"], s["mean"], s["rstd"], c["rows"], c["H"], EPS,
                       s["stream"])
    return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}


def _own_ln_bwd(s):
    from host_offloaded_layer_b200 import _lib as L

    c = s["case"]
    L.mt_layernorm_bwd(s["dy"], c["ld"], s["x"], c["ld"], s["g"], s["mean"], s["rstd"], s["dres"], c["ld"], s["dx"],
                       c["ld"], s["dg"], s["db"], c["rows"], c["H"], s["ws"], s["ws_bytes"], s["stream"])
    return {"dx": s["dx"], "dg": s["dg"], "db": s["db"]}


def _own_mrope(s):
    from host_offloaded_layer_b200 import _lib as L

    c = s["case"]
    L.mt_mrope(s["x"], c["ld"], s["y"], c["ld"], s["pos"], c["rows"], s["sections"], c["rows"], c["heads"], c["d"],
               c["theta"], c["interleaved"], c["per_axis"], c["inverse"], s["stream"])
    return {"y": s["y"]}


def _own_muon(s):
    from host_offloaded_layer_b200 import _lib as L

    c = s["case"]
    L.mt_muon_update(s["g"], c["cols"], s["m"], s["m_out"], c["cols"], s["o"], c["cols"], c["rows"], c["cols"], s["cfg"],
                     s["ws"], s["ws_bytes"], s["stream"])
    return {"o": s["o"], "m": s["m_out"]}


_plain = {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd, "mrope": _plain_mrope, "muon": _plain_muon}
_own = {"ln_fwd": _own_ln_fwd, "ln_bwd": _own_ln_bwd, "mrope": _own_mrope, "muon": _own_muon}


# ---------------------------------------------------------------- floors and the definitions in float64
def work(case):
    op = case["op"]
    if op == "muon":
        m, n = sorted((case["rows"], case["cols"]))
        # X X^T and A A are symmetric: half of each product is enough
        return {"bytes": 14.0 * m * n, "flops": STEPS * (3.0 * m * m * n + 1.0 * m * m * m)}
    if op == "mrope":
        n = case["rows"] * case["heads"] * case["d"]
        return {"bytes": 4.0 * n + 4.0 * case["rows"] * case["axes"], "flops": 3.0 * n}
    n, cols = case["rows"] * case["H"], (2 if case["affine"] else 0) * case["H"]
    if op == "ln_fwd":
        return {"bytes": 4.0 * n + 8.0 * case["rows"] + 2.0 * cols, "flops": 8.0 * n}
    return {"bytes": (8.0 if case["dres"] else 6.0) * n + 8.0 * case["rows"] + 8.0 * case["H"] + 1.0 * cols,
            "flops": 15.0 * n}


def exact(case, seed):
    s, op, f64 = prepare(case, seed), case["op"], torch.float64
    if op in ("ln_fwd", "ln_bwd"):
        parts = []
        g = torch.ones(case["H"], dtype=f64, device="cuda") if s["g"] is None else s["g"].to(f64)
        step = max(1, (1 << 26) // case["H"])  # in slices of rows: float64 copies of the whole would not leave room
        dg = torch.zeros(case["H"], dtype=f64, device="cuda")
        db = torch.zeros_like(dg)
        for r in range(0, case["rows"], step):
            at = slice(r, r + step)
            x = s["x"][at].to(f64)
            if op == "ln_fwd":
                var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
                y = (x - mean) / (var + EPS).sqrt() * g
                if s["b"] is not None:
                    y += s["b"].to(f64)
                parts.append((y, mean[:, 0], (var[:, 0] + EPS).rsqrt()))
            else:
                r1 = s["rstd"][at].to(f64)[:, None]
                xh = (x - s["mean"][at].to(f64)[:, None]) * r1
                dy = s["dy"][at].to(f64)
                dg += torch.einsum("rj,rj->j", dy, xh)
                db += dy.sum(0)
                dxh = dy * g
                dx = dxh - (dxh.sum(1, keepdim=True) + xh * torch.einsum("rj,rj->r", dxh, xh)[:, None]) / case["H"]
                dx *= r1
                if s["dres"] is not None:
                    dx += s["dres"][at].to(f64)
                parts.append((dx,))
        whole = [torch.cat([p[i] for p in parts]) for i in range(len(parts[0]))]
        return dict(zip(("y", "mean", "rstd"), whole)) if op == "ln_fwd" else {"dx": whole[0], "dg": dg, "db": db}
    if op == "mrope":
        axis, freq = _frequencies(case)
        d, n = case["d"], len(axis)
        y = s["x"].to(f64).reshape(case["rows"], case["heads"], d)
        sign = -1.0 if case["inverse"] else 1.0
        for i in range(n):  # each pair as a complex number, turned by its angle
            angle = s["pos"][axis[i]].to(f64) * (sign * freq[i])
            z = torch.complex(y[:, :, i], y[:, :, n + i]) * torch.polar(torch.ones_like(angle), angle)[:, None]
            y[:, :, i], y[:, :, n + i] = z.real, z.imag
        return {"y": y.reshape(case["rows"], -1)}
    # the wide side's Gram matrix, and the polynomial's steps on it alone
    g, m = s["g"].to(f64), s["m"].to(f64)
    m = m * MOMENTUM + g
    u = m * MOMENTUM + g if case["nesterov"] else m
    x = u / (torch.linalg.norm(u) + MUON_EPS)
    tall = case["rows"] > case["cols"]
    eye = torch.eye(min(x.shape), dtype=f64, device="cuda")
    for _ in range(STEPS):
        gram = x.mT @ x if tall else x @ x.mT
        poly = NS_A * eye + gram @ (NS_B * eye + NS_C * gram)
        x = x @ poly if tall else poly @ x
    return {"o": x, "m": m}
