"""BlockNorm against fp64: widths around the wave, the wide and the element-wise loads, every type,
gate and missing part, gradients against autograd of the definition and against differences.

Tolerances.  A bf16 result is off by half a step, 2^-8 of the value; where the residual is kept in
bf16 an element next to a border may round to the other side (one more step, 2^-7 of it, of the
residual and so of x).  fp32 sums over a row or a column of n elements: 4 sqrt(n) 2^-24 of the
result's largest magnitude, plus 8 ulp of the few products around them.  dr and dy are differences
rz (dx w2) - z rz^3 mean(...) of two terms that may cancel (at width 1 they are equal but for eps):
each term is rounded relative to itself, so their tolerance is relative to the terms' size."""
import math

import pytest
import torch

import block_ref as ref
import quantized_moe_route_amd as q

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def tol(dt, n, border=False):
    f = (4 * math.sqrt(n) + 8) * 2.0 ** -24
    return f if dt == F32 else f + 2.0 ** -8 + (2.0 ** -7 if border else 0.0)


def close(got, want, n, what, border=False, terms=0.0):
    assert got.shape == want.shape, what
    t = tol(got.dtype, n, border)
    top = max(terms, float(want.abs().max())) if want.numel() else 0.0
    e = float((got.to(F64) - want).abs().max()) if want.numel() else 0.0
    assert e <= t * max(top, 1e-30), f"{what}: {e:.3e} against {t:.2e} * {top:.3e}"


def make(T, D, rt, yt, xt, wt, gate, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * T + D)
    rnd = lambda *s, sd=1.0, dt=F32: (torch.randn(*s, generator=g) * sd).to(dt).cuda()  # noqa: E731
    shape = {"none": None, "channel": (D,), "token": (T,), "full": (T, D)}[gate]
    return dict(r=rnd(T, D, sd=3.0, dt=rt), y=rnd(T, D, sd=2.0, dt=yt), w1=rnd(D, dt=wt), w2=rnd(D, dt=wt),
                gate=None if shape is None else rnd(*shape, dt=yt if gate == "full" else F32),
                dr=rnd(T, D, dt=rt), dx=rnd(T, D, dt=xt))


def check(T, D, rt=F32, yt=F32, xt=BF16, wt=F32, gate="none", post=True, nxt=True, with_y=True, with_dr=True, alpha=0.9, beta=0.7):
    c = make(T, D, rt, yt, xt, wt, gate)
    w1, w2 = (c["w1"] if post else None), (c["w2"] if nxt else None)
    y, gt = (c["y"], c["gate"]) if with_y else (None, None)
    n = q.BlockNorm(D, max_tokens=T, w_post=w1, w_next=w2, gate=gate, eps_post=1e-5, eps_next=1e-6, res_scale=alpha,
                    branch_scale=beta, r_dtype=rt, y_dtype=yt, x_dtype=xt, device="cuda")
    f = n.forward(c["r"], y, gate=gt)
    leaf = lambda t: None if t is None else t.detach().to(F64).requires_grad_(True)  # noqa: E731
    r64, y64, g64, a64, b64 = leaf(c["r"]), leaf(y), leaf(gt), leaf(w1), leaf(w2)
    gv = g64 if g64 is None or gate != "token" else g64[:, None]
    r_out, x = ref.norm(r64, y64, gv, a64, b64, (1e-5, 1e-6), alpha, beta, stored=f.r)
    kept = rt == BF16
    close(f.r, r_out.detach(), D, "r_out", kept)
    if nxt:
        close(f.x, x.detach(), D, "x", kept)
    b = n.backward(f, y, gate=gt, dr_out=c["dr"] if with_dr else None, dx=c["dx"] if nxt else None)
    loss = ((c["dr"].to(F64) * r_out).sum() if with_dr else 0.0) + ((c["dx"].to(F64) * x).sum() if nxt else 0.0)
    loss.backward()
    big = lambda *f: float(math.prod(abs(t).detach().to(F64) if torch.is_tensor(t) else t for t in f if t is not None).max())  # noqa: E731
    terms = big(c["dx"], b64, f.rstd[1][:, None]) if nxt else 0.0
    close(b.dr, r64.grad, D, "dr", terms=alpha * terms if with_y else terms)
    if with_y:
        up = beta * (terms + (big(c["dr"]) if with_dr else 0.0)) * (big(gv) if gv is not None else 1.0)
        close(b.dy, y64.grad, D, "dy", terms=up * big(a64, f.rstd[0][:, None]) if post else up)
        if gate != "none":
            close(b.dgate, g64.grad, max(D, T), "dgate")
        if post:
            close(b.dw_post, a64.grad, max(D, T), "dw_post")
    if nxt:
        close(b.dw_next, b64.grad, max(D, T), "dw_next")
    again = n.backward(f, y, gate=gt, dr_out=c["dr"] if with_dr else None, dx=c["dx"] if nxt else None)
    for name in ("dr", "dy", "dgate", "dw_post", "dw_next"):
        p, s = getattr(b, name), getattr(again, name)
        assert (p is None and s is None) or torch.equal(p, s), name
    return c, n, f, b


@pytest.mark.parametrize("D", [1, 2, 7, 8, 63, 64, 65, 257, 512, 1000, 1023, 3584, 4099, 8192, 8200, 16383, 16384])
@pytest.mark.parametrize("T", [1, 3])
def test_widths(T, D):
    check(T, D)


@pytest.mark.parametrize("T", [2, 7, 8, 9, 511, 512, 513, 4097, 9000])
@pytest.mark.parametrize("D", [40, 33, 520, 515])
def test_row_counts_with_every_gradient(T, D):
    check(T, D, gate="channel")


@pytest.mark.parametrize("rt", [F32, BF16])
@pytest.mark.parametrize("yt", [F32, BF16])
@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("wt", [F32, BF16])
@pytest.mark.parametrize("gate,D", [("none", 136), ("channel", 136), ("token", 131), ("full", 136), ("full", 131)])
def test_types_and_gates(rt, yt, xt, wt, gate, D):
    check(9, D, rt, yt, xt, wt, gate)


@pytest.mark.parametrize("post,nxt,with_y,with_dr,gate", [
    (False, True, True, True, "token"), (True, False, True, True, "full"), (False, False, True, True, "channel"),
    (True, True, True, False, "none"), (False, True, False, True, "none"), (True, True, False, True, "channel"),
    (True, True, False, False, "none"), (False, True, True, False, "token")])
@pytest.mark.parametrize("D", [72, 69])
def test_missing_parts(post, nxt, with_y, with_dr, gate, D):
    check(6, D, post=post, nxt=nxt, with_y=with_y, with_dr=with_dr, gate=gate)


def test_in_place_and_unaligned_views_keep_their_values():
    T, D = 5, 264
    c, n, f, b = check(T, D, gate="full")
    r = c["r"].clone()
    g = n.forward(r, c["y"], gate=c["gate"], r_out=r)
    assert g.r is r and torch.equal(r, f.r) and torch.equal(g.x, f.x)
    odd = torch.empty(T * D + 1, device="cuda")[1:].view(T, D)  # element-wise loads
    odd.copy_(c["r"])
    g = n.forward(odd, c["y"], gate=c["gate"])
    torch.testing.assert_close(g.r, f.r, rtol=2 ** -20, atol=2 ** -20)


def test_zero_rows_and_zero_tokens():
    D = 136
    c = make(4, D, F32, F32, BF16, F32, "channel")
    n = q.BlockNorm(D, max_tokens=4, w_post=c["w1"], w_next=c["w2"], gate="channel")
    c["y"][1] = 0
    c["r"][2], c["y"][2] = 0, 0
    f = n.forward(c["r"], c["y"], gate=c["gate"])
    assert torch.equal(f.r[1], c["r"][1]) and not f.r[2].any() and not f.x[2].any()
    b = n.backward(f, c["y"], gate=c["gate"], dr_out=c["dr"], dx=c["dx"])
    assert all(torch.isfinite(t).all() for t in (b.dr, b.dy, b.dgate, b.dw_post, b.dw_next))
    e = n.forward(c["r"][:0], c["y"][:0], gate=c["gate"])
    b = n.backward(e, c["y"][:0], gate=c["gate"], dr_out=c["dr"][:0], dx=c["dx"][:0])
    assert not b.dgate.any() and not b.dw_post.any() and not b.dw_next.any()


def test_rows_keep_to_themselves():
    """A row that is not finite reaches no other row; rows behind the last stay as they were."""
    D = 520
    c = make(4, D, F32, F32, F32, F32, "none")
    n = q.BlockNorm(D, max_tokens=4, w_post=c["w1"], w_next=c["w2"], x_dtype=F32)
    clean = n.forward(c["r"], c["y"])
    y = c["y"].clone()
    y[1, 3] = float("nan")
    f = n.forward(c["r"], y)
    keep = [0, 2, 3]
    assert torch.equal(f.r[keep], clean.r[keep]) and torch.equal(f.x[keep], clean.x[keep]) and torch.isnan(f.x[1]).all()
    out = torch.full((4, D), 5.0, device="cuda")
    n.forward(c["r"][:2], c["y"][:2], r_out=out[:2])
    assert (out[2:] == 5).all()


def test_gradient_against_differences():
    """Directional derivative of sum(dr r_out) + sum(dx x) by central differences of the forward itself
    (fp32, step 2^-8: its truncation error is of the order of the step's square, 2^-16, and rounding
    2^-24 / 2^-8 = 2^-16 of the terms, against 2^-9 here)."""
    T, D, h = 6, 264, 2.0 ** -8
    c = make(T, D, F32, F32, F32, F32, "channel")
    n = q.BlockNorm(D, max_tokens=T, w_post=c["w1"], w_next=c["w2"], gate="channel", x_dtype=F32, branch_scale=0.7)
    f = n.forward(c["r"], c["y"], gate=c["gate"])
    b = n.backward(f, c["y"], gate=c["gate"], dr_out=c["dr"], dx=c["dx"])

    def loss(r, y, gate):
        g = n.forward(r, y, gate=gate)
        return float((c["dr"].to(F64) * g.r.to(F64)).sum() + (c["dx"].to(F64) * g.x.to(F64)).sum())

    args = [c["r"], c["y"], c["gate"]]
    for i, grad in enumerate((b.dr, b.dy, b.dgate)):
        v = torch.randn_like(args[i])
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * v, args[i] - h * v
        fd = (loss(*up) - loss(*dn)) / (2 * h)
        an = float((grad.to(F64) * v.to(F64)).sum())
        scale = float((grad.to(F64) * v.to(F64)).abs().sum())
        assert abs(fd - an) <= 2.0 ** -9 * scale, (i, fd, an)


def test_captured_and_replayed():
    T, D = 700, 72
    c, n, f, b = check(T, D, gate="channel")
    r, y = c["r"].clone(), c["y"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        n.backward(n.forward(r, y, gate=c["gate"]), y, gate=c["gate"], dr_out=c["dr"], dx=c["dx"])
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gf = n.forward(r, y, gate=c["gate"])
        gb = n.backward(gf, y, gate=c["gate"], dr_out=c["dr"], dx=c["dx"])
    for k in range(3):
        y.copy_(c["y"] * (k + 1))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (gf.r, gf.x, gb.dr, gb.dy, gb.dgate, gb.dw_post, gb.dw_next)]
        e = n.forward(r, y, gate=c["gate"])
        eb = n.backward(e, y, gate=c["gate"], dr_out=c["dr"], dx=c["dx"])
        assert all(torch.equal(p, w) for p, w in zip(got, (e.r, e.x, eb.dr, eb.dy, eb.dgate, eb.dw_post, eb.dw_next))), k


def test_python_refusals():
    c = make(4, 64, F32, F32, BF16, F32, "token")
    n = q.BlockNorm(64, max_tokens=4, w_post=c["w1"], w_next=c["w2"], gate="token")
    f = n.forward(c["r"], c["y"], gate=c["gate"])
    for kw in (dict(gate=None), dict(gate=c["gate"].cpu()), dict(gate=c["gate"][:2]), dict(gate=c["gate"].to(BF16))):
        with pytest.raises((ValueError, TypeError)):
            n.forward(c["r"], c["y"], **kw)
    with pytest.raises(TypeError):
        n.forward(c["r"].to(BF16), c["y"], gate=c["gate"])
    with pytest.raises(ValueError):
        n.forward(c["r"].t(), c["y"], gate=c["gate"])
    with pytest.raises(ValueError):
        n.backward(f, c["y"], gate=c["gate"], dr_out=c["dr"])  # dx is missing
    with pytest.raises(q.MoeError):
        n.forward(c["r"], c["y"], gate=c["gate"], r_out=c["y"])
    with pytest.raises(ValueError):
        q.BlockNorm(64, max_tokens=4, w_post=c["w1"], gate="row")
    with pytest.raises(q.MoeError):
        q.BlockNorm(64, max_tokens=4, w_post=c["w1"], eps_post=0.0)
    small = q.BlockNorm(64, max_tokens=2, w_next=c["w2"])
    with pytest.raises(q.MoeError):
        small.forward(c["r"])
