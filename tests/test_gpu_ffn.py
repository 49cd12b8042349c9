"""GatedFFN against fp64: sizes around every tile edge, both activations, both result types,
gradients, accumulation, missing outputs, streams, captured and replayed calls.

Tolerances.  A bf16 result is off by half a step, 2^-8 of the value, and by the rounding of the
operand before it (h, or dg and du), again 2^-8 of each term; the rounding errors of the terms of a
sum are independent, so relative to the norms 2 * 2^-8 holds both.  An fp32 result carries every
operand exactly: what is left is fp32 accumulation over at most K terms in three products one after
another, a random walk of sqrt(K) 2^-24 each, and the activation's own few ulp: 8 sqrt(K) 2^-24."""
import math

import pytest
import torch

import block_ref as ref
import quantized_moe_route_amd as q

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64

SIZES = [(1, 8, 8), (1, 512, 320), (2, 64, 48), (3, 72, 200), (15, 264, 136), (16, 256, 512), (17, 256, 512), (33, 1000, 72),
         (64, 520, 640), (65, 72, 200), (130, 520, 328), (300, 136, 264), (513, 1032, 776), (200, 8, 1024), (40, 1024, 8)]


def make(T, D, I, seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * T + D + I)
    rnd = lambda *s, sd: (torch.randn(*s, generator=g) * sd).to(BF16).cuda()  # noqa: E731
    return dict(x=rnd(T, D, sd=1.0), wg=rnd(I, D, sd=D ** -0.5), wu=rnd(I, D, sd=D ** -0.5), wd=rnd(D, I, sd=I ** -0.5),
                dy=rnd(T, D, sd=0.1))


def close(got, want, dt, K, what):
    assert got.dtype == dt and got.shape == want.shape, what
    tol = 2 * 2.0 ** -8 if dt == BF16 else 8 * math.sqrt(K) * 2.0 ** -24
    e = got.to(F64) - want
    l2, mx = float(e.norm() / want.norm()), float(e.abs().max() / want.abs().max())
    assert l2 <= tol and mx <= tol, f"{what}: rel {l2:.2e}, max {mx:.2e}, tolerance {tol:.2e}"


def layer(c, T, act="swiglu", **kw):
    return q.GatedFFN(c["wg"], c["wu"], c["wd"], max_tokens=T, act=q.ACTS[act], **kw)


@pytest.mark.parametrize("T,D,I", SIZES)
@pytest.mark.parametrize("act,dt", [("swiglu", BF16), ("situ", F32), ("swiglu", F32), ("situ", BF16)])
def test_forward_and_gradients(T, D, I, act, dt):
    c = make(T, D, I)
    f = layer(c, T, act)
    gu = f.new_saved_gu(T)
    y = f.forward(c["x"], out_dtype=dt, saved_gu=gu)
    assert torch.equal(y, f.forward(c["x"], out_dtype=dt))
    K = max(T, D, 2 * I)
    (dx, dwg, dwu, dwd), (g, u) = ref.ffn_grads(act, *(c[k] for k in ("x", "wg", "wu", "wd", "dy")))
    close(y, ref.ffn(act, c["x"], c["wg"], c["wu"], c["wd"]), dt, K, "y")
    close(gu, torch.stack([g, u], 1), F32, K, "g, u")
    for saved in (gu, None):
        got = f.backward(c["x"], c["dy"], saved_gu=saved, dx_dtype=dt, dw_dtype=dt)
        for a, b, n in zip((got[0], *got[1]), (dx, dwg, dwu, dwd), ("dx", "dw_gate", "dw_up", "dw_down")):
            close(a, b, dt, K, n)


# sizes at which the five products take, among them, every tile shape, whole and with the reduction in parts
@pytest.mark.parametrize("T,D,I", [(3300, 4104, 2056), (4096, 1024, 6144), (4000, 512, 3080), (1030, 520, 4104), (48, 2048, 3000)])
def test_every_tile_shape(T, D, I):
    c = make(T, D, I)
    f = layer(c, T)
    for dt in (BF16, F32):
        gu = f.new_saved_gu(T)
        y = f.forward(c["x"], out_dtype=dt, saved_gu=gu)
        want, _ = ref.ffn_grads("swiglu", *(c[k] for k in ("x", "wg", "wu", "wd", "dy")))
        K = max(T, D, 2 * I)
        close(y, ref.ffn("swiglu", c["x"], c["wg"], c["wu"], c["wd"]), dt, K, "y")
        got = f.backward(c["x"], c["dy"], saved_gu=gu, dx_dtype=dt, dw_dtype=dt)
        for a, b, n in zip((got[0], *got[1]), want, ("dx", "dw_gate", "dw_up", "dw_down")):
            close(a, b, dt, K, n)


# few tokens and much weight in fp32: the three terms of an operand are rows of their own, joined afterwards
@pytest.mark.parametrize("T,D,I", [(1, 4104, 2056), (4, 3336, 4008), (21, 2048, 3000), (22, 2048, 3000), (43, 1536, 5000), (64, 3000, 1504)])
def test_terms_as_rows(T, D, I):
    c = make(T, D, I)
    f = layer(c, T)
    K = 2 * max(D, I)
    (dx, *dw), _ = ref.ffn_grads("swiglu", *(c[k] for k in ("x", "wg", "wu", "wd", "dy")))
    want = ref.ffn("swiglu", c["x"], c["wg"], c["wu"], c["wd"])
    base = torch.randn(T, D, device="cuda")
    y = base.clone()
    close(f.forward(c["x"], out_dtype=F32), want, F32, K, "y")
    close(f.forward(c["x"], y, accumulate=True), want + base.to(F64), F32, K, "y added")
    got = f.backward(c["x"], c["dy"], dx_dtype=F32, dw_dtype=F32)
    for a, b, n in zip((got[0], *got[1]), (dx, *dw), ("dx", "dw_gate", "dw_up", "dw_down")):
        close(a, b, F32, K, n)
    g = torch.full((T + 1, D), 5.0, device="cuda")
    f.backward(c["x"], c["dy"], dx=g[:T], need_dw=False)
    assert torch.equal(g[:T], got[0]) and (g[T] == 5).all()


@pytest.mark.parametrize("T,D,I", [(1, 256, 128), (5, 264, 136), (100, 328, 264)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_accumulate_adds_onto_what_is_there(T, D, I, dt):
    c = make(T, D, I)
    f = layer(c, T)
    base = torch.randn(T, D, device="cuda").to(dt)
    want = ref.ffn("swiglu", c["x"], c["wg"], c["wu"], c["wd"]) + base.to(F64)
    y = base.clone()
    assert f.forward(c["x"], y, accumulate=True) is y
    close(y, want, dt, max(D, 2 * I), "y")
    (dx, *_), _ = ref.ffn_grads("swiglu", *(c[k] for k in ("x", "wg", "wu", "wd", "dy")))
    g = base.clone()
    f.backward(c["x"], c["dy"], dx=g, accumulate=True, need_dw=False)
    close(g, dx + base.to(F64), dt, max(D, 2 * I), "dx")


@pytest.mark.parametrize("T", [1, 7, 90])
def test_each_gradient_alone_has_the_same_bits(T):
    c = make(T, 264, 136)
    f = layer(c, T)
    dx, dw = f.backward(c["x"], c["dy"])
    one = f.backward(c["x"], c["dy"], need_dw=False)
    assert torch.equal(one[0], dx) and one[1] == (None, None, None)
    assert f.backward(c["x"], c["dy"], need_dx=False)[0] is None
    for i in range(3):
        part = [torch.full_like(w, 7.0) if j == i else None for j, w in enumerate(dw)]
        f.backward(c["x"], c["dy"], need_dx=False, dw=part)
        assert torch.equal(part[i], dw[i]), i
    # fp32 weight gradients beside a bf16 dx: each keeps its own precision
    mixed, dw32 = f.backward(c["x"], c["dy"], dw_dtype=F32)
    assert torch.equal(mixed, dx)
    assert torch.equal(dw32[0], f.backward(c["x"], c["dy"], dx_dtype=F32, dw_dtype=F32)[1][0])


def test_no_tokens_and_rows_behind_the_last():
    c = make(8, 64, 48)
    f = layer(c, 8)
    empty = c["x"][:0]
    assert f.forward(empty).shape == (0, 64)
    dx, dw = f.backward(empty, empty)
    assert dx.shape == (0, 64) and all(not w.any() for w in dw)
    for T in (1, 5):
        big = torch.full((8, 64), 3.0, device="cuda", dtype=BF16)
        f.forward(c["x"][:T], big[:T])
        assert (big[T:] == 3).all() and not (big[:T] == 3).all()
        d = torch.full((8, 64), 3.0, device="cuda", dtype=BF16)
        f.backward(c["x"][:T], c["dy"][:T], dx=d[:T])
        assert (d[T:] == 3).all()


@pytest.mark.parametrize("T", [1, 33])
def test_values_that_are_not_finite_stay_in_their_rows(T):
    c = make(T + 1, 264, 136)
    clean = {dt: layer(c, T + 1).forward(c["x"], out_dtype=dt) for dt in (BF16, F32)}
    x = c["x"].clone()
    x[0, 5] = float("inf")
    for dt in (BF16, F32):
        y = layer(c, T + 1).forward(x, out_dtype=dt)
        assert not torch.isfinite(y[0]).any() and torch.equal(y[1:], clean[dt][1:])


def test_two_calls_on_another_stream_and_their_bits():
    c = make(70, 520, 328)
    f = layer(c, 70)
    y = f.forward(c["x"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        z = [f.forward(c["x"]) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(y, t) for t in z)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_captured_and_replayed(T):
    c = make(T, 264, 520)
    f = layer(c, T)
    x, dy = c["x"].clone(), c["dy"].clone()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw = tuple(torch.empty_like(c[k]) for k in ("wg", "wu", "wd"))
    gu = f.new_saved_gu(T)

    def work():
        f.forward(x, y, saved_gu=gu)
        f.backward(x, dy, saved_gu=gu, dx=dx, dw=dw)

    work()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for k in range(3):
        n = make(T, 264, 520, seed=k + 1)
        x.copy_(n["x"])
        dy.copy_(n["dy"])
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, *dw)]
        work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, *dw))), k


def test_python_refusals():
    c = make(8, 64, 48)
    f = layer(c, 8, backward=False)
    with pytest.raises(q.MoeError):
        f.backward(c["x"], c["dy"])
    f = layer(c, 4)
    with pytest.raises(q.MoeError):
        f.forward(c["x"])  # more than max_tokens
    f = layer(c, 8)
    for bad in (c["x"].float(), c["x"].cpu(), c["x"][:, :32], torch.empty(64, 8, device="cuda", dtype=BF16).t()):
        with pytest.raises((TypeError, ValueError)):
            f.forward(bad)
    with pytest.raises(q.MoeError):
        f.forward(c["x"], c["x"])  # y overlaps x
    with pytest.raises(q.MoeError):
        f.backward(c["x"], c["dy"], dx=c["dy"])
    with pytest.raises(TypeError):
        f.forward(c["x"], torch.empty(8, 64, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        f.forward(c["x"], accumulate=True)
    odd = torch.empty(8 * 64 + 1, device="cuda", dtype=BF16)[1:].view(8, 64)
    with pytest.raises(q.MoeError):
        f.forward(odd)  # not 16-byte aligned
    f.close()
    with pytest.raises(RuntimeError):
        f.forward(c["x"])
