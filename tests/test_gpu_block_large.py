"""The dense block operators where element offsets pass 32 bits: rows at the far end against fp64."""
import pytest
import torch

import block_ref as ref
import quantized_moe_route_amd as q

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of free device memory")


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def rel(a, b):
    return float((a.to(F64) - b).abs().max() / b.abs().max())


def test_ffn():
    """2^32 < T 2 I: g and u, dg and du.  Tolerances as in the tests of ordinary sizes (two bf16 roundings)."""
    room(120)
    T, D, I = 70001, 64, 32768
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s, sd: (torch.randn(*s, generator=g, device="cuda") * sd).to(BF16)  # noqa: E731
    x, dy = rnd(T, D, sd=1.0), rnd(T, D, sd=0.1)
    wg, wu, wd = rnd(I, D, sd=D ** -0.5), rnd(I, D, sd=D ** -0.5), rnd(D, I, sd=I ** -0.5)
    f = q.GatedFFN(wg, wu, wd, max_tokens=T)
    gu = f.new_saved_gu(T)
    y = f.forward(x, saved_gu=gu)
    dx, _ = f.backward(x, dy, saved_gu=gu, need_dw=False)
    for rows in (slice(0, 3), slice(40000, 40003), slice(T - 3, T)):
        (want, *_), (gw, uw) = ref.ffn_grads("swiglu", x[rows], wg, wu, wd, dy[rows])
        assert rel(gu[rows], torch.stack([gw, uw], 1)) <= 1e-5
        assert rel(y[rows], ref.ffn("swiglu", x[rows], wg, wu, wd)) <= 2.0 ** -7
        assert rel(dx[rows], want) <= 2.0 ** -7


def test_norm():
    room(80)
    T, D = 262147, 16384
    g = torch.Generator(device="cuda").manual_seed(2)
    r = torch.randn(T, D, generator=g, device="cuda", dtype=BF16)
    y = torch.randn(T, D, generator=g, device="cuda", dtype=BF16)
    w1, w2 = (1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
    n = q.BlockNorm(D, max_tokens=T, w_post=w1, w_next=w2, r_dtype=BF16, y_dtype=BF16)
    f = n.forward(r, y)
    b = n.backward(f, y, dr_out=r, dx=f.x, need_dw=False)
    for rows in (slice(0, 2), slice(T - 2, T)):
        leaf = [t[rows].to(F64).requires_grad_(True) for t in (r, y)]
        ro, x = ref.norm(leaf[0], leaf[1], None, w1, w2, stored=f.r[rows])
        assert rel(f.r[rows], ro.detach()) <= 2.0 ** -7 and rel(f.x[rows], x.detach()) <= 2.0 ** -6
        ((r[rows].to(F64) * ro).sum() + (f.x[rows].to(F64) * x).sum()).backward()
        assert rel(b.dr[rows], leaf[0].grad) <= 2.0 ** -7 and rel(b.dy[rows], leaf[1].grad) <= 2.0 ** -7


@pytest.mark.parametrize("e4m3", [True, False])
def test_adamw(e4m3):
    """One tensor of more than 2^32 elements beside a small one."""
    room(110)
    n = (1 << 32) + 777
    p = [torch.zeros(n, device="cuda", dtype=BF16), torch.zeros(1000, device="cuda")]
    g = [torch.zeros(n, device="cuda", dtype=BF16), torch.ones(1000, device="cuda")]
    tail = torch.randn(777, device="cuda").to(BF16)
    g[0][-777:] = tail
    o = q.AdamW(p, g, **q.AdamW.new_state(p, e4m3=e4m3), weight_decay=0.0, max_norm=1e6)
    norm = torch.zeros((), device="cuda")
    o.step(1e-2, grad_norm=norm)
    total = float((tail.to(F64).square().sum() + 1000).sqrt())
    assert abs(float(norm) - total) <= 1e-6 * total
    zero = torch.zeros(777, device="cuda", dtype=F64)
    want = ref.adamw(zero, tail, zero, zero, 1, 1e-2, (0.9, 0.999), 1e-8, 0.0)[0]
    assert float((p[0][-777:].to(F64) - want).abs().max()) <= 2.0 ** -8 * 1.1e-2
    assert not p[0][:1 << 20].any() and not p[0][-5000:-777].any()
    assert float((p[1] + 1e-2).abs().max()) <= 1e-6
