"""Cases of the dense operators around the routed experts, for timing and comparing them.

Three operators: the gated feed-forward block (GatedFFN), the norms before and after a block with its
gate and residual scale (BlockNorm), and the AdamW step over many tensors (AdamW).  run() computes a case
with the framework's kernels where `own` is true, else in elementary torch operations in 32 bits, rounded
once where an output has fewer; exact() computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "f32": F32}
E4M3 = torch.float8_e4m3fn
QBLOCK = 256         # elements of a tensor that share a scale of its 8-bit states
QMAX = 448.0         # largest E4M3 value
QMIN = 2.0 ** -9     # smallest positive one
FLT_MIN = 2.0 ** -126

BETAS, EPS, DECAY, LR, MAX_NORM = (0.9, 0.999), 1e-8, 0.01, 1e-3, 1.0


# ---------------------------------------------------------------- cases

def _ffn(name, T, D, I, act="swiglu", out="bf16", train=False):
    return {"name": name, "op": "ffn", "T": T, "D": D, "I": I, "act": act, "out": out, "train": train}


def _norm(name, T, D, r, y, x, w, gate, train):
    return {"name": name, "op": "norm", "T": T, "D": D, "r": r, "y": y, "x": x, "w": w, "gate": gate, "train": train}


def _adamw(name, rows, cols, tensors, state, param, clip):
    return {"name": name, "op": "adamw", "rows": rows, "cols": cols, "tensors": tensors, "state": state, "param": param,
            "clip": clip}


def listed():
    return [
        # two shared experts of the K3 layer as one block of twice their width: a decode step of one token
        _ffn("ffn decode 1", 1, 3584, 6144),
        # the same block in a decode step of the 64-token batch
        _ffn("ffn decode 64", 64, 3584, 6144),
        # a short ragged batch on a layer of odd widths, SiTU, fp32 results (added onto the routed experts' y)
        _ffn("ffn ragged f32 train", 777, 1160, 2744, act="situ", out="f32", train=True),
        # a training step of the shared experts on the 4096-token batch: forward, input and weight gradients
        _ffn("ffn train 4096", 4096, 3584, 6144, train=True),
        # a dense layer in the model's width
        _ffn("ffn train wide", 8192, 7168, 14336, train=True),
        # between two blocks in a decode step of one token
        _norm("norm decode 1", 1, 7168, "f32", "f32", "bf16", "f32", "none", False),
        # the latent width's training step, residual stream and branch in fp32 as the routed experts return it
        _norm("norm mixed train", 1531, 3584, "f32", "f32", "bf16", "f32", "token", True),
        # the 4096-token training step in bf16 with a learned scale for each channel
        _norm("norm train 4096", 4096, 3584, "bf16", "bf16", "bf16", "bf16", "channel", True),
        # a long prefill's training step with a gate of the branch's own shape
        _norm("norm train wide", 16384, 7168, "bf16", "bf16", "bf16", "bf16", "full", True),
        # the rank-16 adapter of one layer: 6 small tensors
        _adamw("adamw adapter", 16, 3584, 6, "f32", "f32", True),
        # the adapters of many layers at once, 8-bit states
        _adamw("adamw adapters 8-bit", 16, 4999, 552, "e4m3", "f32", True),
        # the three matrices of the dense block and more of them: bf16 parameters with their fp32 masters
        _adamw("adamw dense", 6144, 3584, 9, "f32", "bf16", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "norm", "adamw"])
    if op == "ffn":
        D, I = 8 * rng.randint(16, 900), 8 * rng.randint(16, 1790)
        return {"op": "ffn", "T": _log(rng, 1, 8192), "D": D, "I": I, "act": rng.choice(["swiglu", "situ"]),
                "out": rng.choice(["bf16", "bf16", "f32"]), "train": rng.random() < 0.6}
    if op == "norm":
        r = rng.choice(["bf16", "f32"])
        return {"op": "norm", "T": _log(rng, 1, 16384), "D": rng.randint(1, 7168) if rng.random() < 0.25 else 8 * rng.randint(1, 896),
                "r": r, "y": rng.choice(["bf16", "f32"]), "x": "bf16" if r == "bf16" else rng.choice(["bf16", "f32"]), "w": r,
                "gate": rng.choice(["none", "channel", "token", "full"]), "train": rng.random() < 0.7}
    rows, cols = rng.randint(1, 64), rng.randint(1, 8000)
    return {"op": "adamw", "rows": rows, "cols": cols, "tensors": _log(rng, 1, min(600, max(2, 90_000_000 // (rows * cols)))),
            "state": rng.choice(["f32", "e4m3"]), "param": rng.choice(["f32", "bf16"]), "clip": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, sd=1.0, dt=F32):
    return (torch.randn(*shape, generator=g, device=DEV) * sd).to(dt)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "ffn":
        T, D, I = case["T"], case["D"], case["I"]
        s["x"] = _randn(g, T, D, dt=BF16)
        s["wg"], s["wu"] = _randn(g, I, D, sd=D ** -0.5, dt=BF16), _randn(g, I, D, sd=D ** -0.5, dt=BF16)
        s["wd"] = _randn(g, D, I, sd=I ** -0.5, dt=BF16)
        s["dy"] = _randn(g, T, D, sd=0.01, dt=BF16) if case["train"] else None
        if own:
            import quantized_moe_route_amd as q
            s["ffn"] = q.GatedFFN(s["wg"], s["wu"], s["wd"], max_tokens=T, act=q.ACTS[case["act"]], backward=case["train"])
    elif case["op"] == "norm":
        T, D = case["T"], case["D"]
        s["rr"], s["yy"] = _randn(g, T, D, sd=4.0, dt=DTYPES[case["r"]]), _randn(g, T, D, sd=2.0, dt=DTYPES[case["y"]])
        s["w1"], s["w2"] = ((1 + _randn(g, D, sd=0.2)).to(DTYPES[case["w"]]) for _ in range(2))
        shape = {"none": None, "channel": (D,), "token": (T,), "full": (T, D)}[case["gate"]]
        s["gg"] = None if shape is None else (0.5 + _randn(g, *shape, sd=0.3)).to(DTYPES[case["y"]] if case["gate"] == "full" else F32)
        if case["train"]:
            s["dr"], s["dx"] = _randn(g, T, D, sd=0.01, dt=DTYPES[case["r"]]), _randn(g, T, D, sd=0.01, dt=DTYPES[case["x"]])
        if own:
            import quantized_moe_route_amd as q
            s["norm"] = q.BlockNorm(D, max_tokens=T, w_post=s["w1"], w_next=s["w2"], gate=case["gate"], eps_post=1e-6, eps_next=1e-6,
                                    res_scale=1.0, branch_scale=0.7, r_dtype=DTYPES[case["r"]], y_dtype=DTYPES[case["y"]],
                                    x_dtype=DTYPES[case["x"]], backward=case["train"])
    else:
        n = case["rows"] * case["cols"]
        pad = -(-n // QBLOCK) * QBLOCK  # every tensor begins at a boundary of its own in the bank
        N = case["tensors"]

        def bank(sd, dt=F32):
            t = torch.zeros(N, pad, device=DEV)
            t[:, :n] = torch.randn(N, n, generator=g, device=DEV) * sd
            return t.to(dt)

        pdt = DTYPES[case["param"]]
        s["grad"] = bank(2e-3, pdt)
        w = bank(0.02)
        s["param"], s["master"] = (w.to(BF16), w) if pdt == BF16 else (w, None)
        m, v = bank(5e-4), bank(2e-3).square_()
        if case["state"] == "e4m3":
            s["m"], s["ms"] = _encode(m)
            s["v"], s["vs"] = _encode(v.sqrt())
        else:
            s["m"], s["v"], s["ms"], s["vs"] = m, v, None, None
        s["t"] = 100
        s["n"] = n
        if own:
            import quantized_moe_route_amd as q
            cut = lambda b: None if b is None else [b[i, :n].view(case["rows"], case["cols"]) for i in range(N)]  # noqa: E731
            per = pad // QBLOCK
            scales = lambda b: None if b is None else [b[i * per:(i + 1) * per] for i in range(N)]  # noqa: E731
            s["opt"] = q.AdamW(cut(s["param"]), cut(s["grad"]), m=cut(s["m"]), v=cut(s["v"]), m_scale=scales(s["ms"]),
                               v_scale=scales(s["vs"]), master=cut(s["master"]), betas=BETAS, eps=EPS, weight_decay=DECAY,
                               max_norm=MAX_NORM if case["clip"] else 0.0, step=s["t"])
    return s


# ---------------------------------------------------------------- plain forms, 32 bits

def _sig(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _act(act, g, u):
    if act == "situ":
        return 4.0 * torch.tanh(g / 4.0) * _sig(g) * (25.0 * torch.tanh(u / 25.0))
    return g * _sig(g) * u


def _act_grad(act, g, u):
    s = _sig(g)
    if act == "situ":
        tg, tu = torch.tanh(g / 4.0), torch.tanh(u / 25.0)
        a, b = 4.0 * tg * s, 25.0 * tu
        sech = lambda z: (1.0 / torch.cosh(z)).square()  # noqa: E731
        return (sech(g / 4.0) * s + a * (1.0 - s)) * b, a * sech(u / 25.0)
    return u * s * (1.0 + g * (1.0 - s)), g * s


def _run_ffn(s):
    out = DTYPES[s["out"]]
    x, wg, wu, wd = s["x"].float(), s["wg"].float(), s["wu"].float(), s["wd"].float()
    g, u = x @ wg.t(), x @ wu.t()
    h = _act(s["act"], g, u)
    y = (h @ wd.t()).to(out)
    if not s["train"]:
        return {"y": y}
    dy = s["dy"].float()
    dh = dy @ wd
    ag, au = _act_grad(s["act"], g, u)
    dg, du = dh * ag, dh * au
    return {"y": y, "dx": (dg @ wg + du @ wu).to(out), "dwg": (dg.t() @ x).to(out), "dwu": (du.t() @ x).to(out),
            "dwd": (dy.t() @ h).to(out)}


def _rms_back(d, z, rstd, w):
    """Gradient of z * rstd(z) * w in z, for the upstream d."""
    dw = d * w
    return rstd * (dw - z * (rstd.square() * (dw * z).mean(1, keepdim=True)))


def _run_norm(s):
    r, y, gate = s["rr"].float(), s["yy"].float(), s["gg"]
    w1, w2 = s["w1"].float(), s["w2"].float()
    gate = 1.0 if gate is None else gate.float()
    gate = gate[:, None] if s["gate"] == "token" else gate
    ry = torch.rsqrt(y.square().mean(1, keepdim=True) + 1e-6)
    n = y * ry * w1
    r2 = (r + 0.7 * gate * n).to(s["rr"].dtype)
    z = r2.float()
    rz = torch.rsqrt(z.square().mean(1, keepdim=True) + 1e-6)
    xdt = DTYPES[s["x"]]
    out = {"r": r2, "x": (z * rz * w2).to(xdt)}
    if not s["train"]:
        return out
    dx = s["dx"].float()
    d = s["dr"].float() + _rms_back(dx, z, rz, w2)
    dn = 0.7 * gate * d
    out |= {"dr": d.to(s["rr"].dtype), "dy": _rms_back(dn, y, ry, w1).to(s["yy"].dtype),
            "dw1": (dn * y * ry).sum(0).to(s["w1"].dtype), "dw2": (dx * z * rz).sum(0).to(s["w2"].dtype)}
    if s["gate"] != "none":
        dgate = 0.7 * d * n
        out["dgate"] = dgate.to(s["yy"].dtype) if s["gate"] == "full" else dgate.sum(1 if s["gate"] == "token" else 0)
    return out


def _encode(a):
    """E4M3 codes of `a` and the fp32 scale of each run of QBLOCK elements."""
    b = a.reshape(-1, QBLOCK)
    scale = b.abs().amax(1, keepdim=True) / QMAX
    scale = torch.where(scale < FLT_MIN, torch.zeros_like(scale), scale)
    q = torch.where(scale == 0, torch.zeros_like(b), b / torch.where(scale == 0, torch.ones_like(scale), scale))
    return q.to(E4M3).view(a.shape), scale.view(-1)


def _raise_zero(codes, a):
    """The second moment's root: a positive one whose code would be zero takes the smallest code."""
    low = torch.full_like(a, QMIN).to(E4M3).view(torch.uint8)
    c = codes.view(torch.uint8)
    return torch.where((c == 0) & (a > 0), low, c).view(E4M3)


def _decode(codes, scale):
    return (codes.float().view(-1, QBLOCK) * scale[:, None]).view(codes.shape)


def _run_adamw(s):
    s["t"] += 1
    b1, b2 = BETAS
    c1, c2 = 1 - b1 ** s["t"], math.sqrt(1 - b2 ** s["t"])
    g = s["grad"].float()
    if s["clip"]:
        g = g * (MAX_NORM / g.double().square().sum().sqrt().clamp(min=MAX_NORM)).float()
    small = s["state"] == "e4m3"
    m = _decode(s["m"], s["ms"]) if small else s["m"]
    v = _decode(s["v"], s["vs"]).square() if small else s["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g.square() * (1 - b2)
    root = v.sqrt()
    p = s["master"] if s["master"] is not None else s["param"]
    p.copy_(p * (1 - LR * DECAY) - (LR / c1) * (m / (root / c2 + EPS)))
    out = {"param": s["param"]}
    if s["master"] is not None:
        s["param"].copy_(p)
        out["master"] = p
    if small:
        mc, ms = _encode(m)
        vc, vs = _encode(root)
        s["m"].copy_(mc)
        s["v"].copy_(_raise_zero(vc, root))
        s["ms"].copy_(ms)
        s["vs"].copy_(vs)
        out |= {"ms": s["ms"], "vs": s["vs"]}
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return out | {"m": s["m"], "v": s["v"]}


# ---------------------------------------------------------------- one pass

def run(s):
    if not own:
        return {"ffn": _run_ffn, "norm": _run_norm, "adamw": _run_adamw}[s["op"]](s)
    if s["op"] == "ffn":
        out, f = DTYPES[s["out"]], s["ffn"]
        if not s["train"]:
            return {"y": f.forward(s["x"], out_dtype=out)}
        gu = f.new_saved_gu(s["T"])
        y = f.forward(s["x"], out_dtype=out, saved_gu=gu)
        dx, (dwg, dwu, dwd) = f.backward(s["x"], s["dy"], saved_gu=gu, dx_dtype=out, dw_dtype=out)
        return {"y": y, "dx": dx, "dwg": dwg, "dwu": dwu, "dwd": dwd}
    if s["op"] == "norm":
        f = s["norm"].forward(s["rr"], s["yy"], gate=s["gg"])
        out = {"r": f.r, "x": f.x}
        if s["train"]:
            b = s["norm"].backward(f, s["yy"], gate=s["gg"], dr_out=s["dr"], dx=s["dx"])
            out |= {"dr": b.dr, "dy": b.dy, "dw1": b.dw_post, "dw2": b.dw_next}
            if b.dgate is not None:
                out["dgate"] = b.dgate
        return out
    s["opt"].step(LR)
    names = ("param", "master", "m", "v", "ms", "vs")
    return {k: s[k] for k in names if s[k] is not None}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "ffn":
        T, D, I = case["T"], case["D"], case["I"]
        ob = 2 if case["out"] == "bf16" else 4
        if not case["train"]:
            return {"bytes": 2 * T * D + 6 * D * I + ob * T * D, "flops": 6 * T * D * I}
        return {"bytes": 4 * T * D + 6 * D * I + 2 * ob * T * D + 3 * ob * D * I, "flops": 18 * T * D * I}
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        size = lambda k: 2 if case[k] == "bf16" else 4  # noqa: E731
        rb, yb, xb, wb = size("r"), size("y"), size("x"), size("w")
        gate = {"none": 0, "channel": 4 * D, "token": 4 * T, "full": yb * T * D}[case["gate"]]
        b = T * D * (2 * rb + yb + xb) + gate + 2 * wb * D
        if case["train"]:
            b += T * D * (2 * rb + yb + xb) + gate + 2 * wb * D
        return {"bytes": b, "flops": T * D * (10 if not case["train"] else 40)}
    n = case["rows"] * case["cols"] * case["tensors"]
    pb = 2 if case["param"] == "bf16" else 4
    st = 16 if case["state"] == "f32" else 4 + 16 / QBLOCK
    return {"bytes": n * (3 * pb + (8 if pb == 2 else 0) + st), "flops": 20 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = lambda t: t.to(F64)  # noqa: E731
    if case["op"] == "ffn":
        x, wg, wu, wd = d(s["x"]), d(s["wg"]), d(s["wu"]), d(s["wd"])
        a, b = torch.matmul(x, wg.T), torch.matmul(x, wu.T)
        sg = torch.sigmoid(a)
        if case["act"] == "situ":
            ta, tb = torch.tanh(a / 4), torch.tanh(b / 25)
            left, right = 4 * ta * sg, 25 * tb
            dleft, dright = (1 - ta * ta) * sg + left * (1 - sg), 1 - tb * tb
        else:
            left, right = a * sg, b
            dleft, dright = sg + left * (1 - sg), torch.ones_like(b)
        out = {"y": torch.matmul(left * right, wd.T)}
        if case["train"]:
            dy = d(s["dy"])
            out["dwd"] = torch.matmul(dy.T, left * right)
            dh = torch.matmul(dy, wd)
            da, db = dh * dleft * right, dh * left * dright
            out["dx"] = torch.matmul(da, wg) + torch.matmul(db, wu)
            out["dwg"], out["dwu"] = torch.matmul(da.T, x), torch.matmul(db.T, x)
        return out
    if case["op"] == "norm":
        D = case["D"]
        w1, w2, y = d(s["w1"]), d(s["w2"]), d(s["yy"])
        gate = torch.ones((), dtype=F64, device=DEV) if s["gg"] is None else d(s["gg"])
        if case["gate"] == "token":
            gate = gate.unsqueeze(1)
        iy = ((y * y).sum(1, keepdim=True) / D + 1e-6) ** -0.5
        unit = y * iy
        r2 = d(s["rr"]) + 0.7 * gate * (unit * w1)
        z = d(r2.to(s["rr"].dtype))  # the norm reads the residual as it is stored
        iz = ((z * z).sum(1, keepdim=True) / D + 1e-6) ** -0.5
        zn = z * iz
        out = {"r": r2, "x": zn * w2}
        if case["train"]:
            back = lambda up, hat, inv: inv * (up - hat * (up * hat).sum(1, keepdim=True) / D)  # noqa: E731
            dx = d(s["dx"])
            dr = d(s["dr"]) + back(dx * w2, zn, iz)
            branch = 0.7 * dr
            dn = branch * gate
            out |= {"dr": dr, "dy": back(dn * w1, unit, iy), "dw1": (dn * unit).sum(0), "dw2": (dx * zn).sum(0)}
            if case["gate"] != "none":
                dgate = branch * (unit * w1)
                out["dgate"] = {"full": dgate, "token": dgate.sum(1), "channel": dgate.sum(0)}[case["gate"]]
        return out
    t, (b1, b2) = s["t"] + 1, BETAS
    g, w = d(s["grad"]), d(s["param"] if s["master"] is None else s["master"])
    if case["clip"]:
        g = g * min(1.0, MAX_NORM / float((g * g).sum().sqrt()))
    rep = lambda sc: d(sc).repeat_interleave(QBLOCK).view(g.shape)  # noqa: E731
    if case["state"] == "e4m3":
        m, v = d(s["m"]) * rep(s["ms"]), (d(s["v"]) * rep(s["vs"])) ** 2
    else:
        m, v = d(s["m"]), d(s["v"])
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    w = w - LR * (DECAY * w + (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)) ** 0.5 + EPS))
    out = {"param": w}
    if s["master"] is not None:
        out["master"] = w
    if case["state"] == "e4m3":
        top = lambda a: a.abs().view(-1, QBLOCK).amax(1) / 448  # noqa: E731
        return out | {"m": None, "v": None, "ms": top(m), "vs": top(v.sqrt())}
    return out | {"m": m, "v": v}
