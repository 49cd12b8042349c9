"""AdamW against fp64 and, for the 8-bit states, bit for bit against the definition in fp32.

Tolerances.  fp32 arithmetic of about ten roundings a step: 16 * 2^-24 of the value for m and v, and for the
parameter of the larger of its value and its update.  A bf16 parameter adds half a step, 2^-8.  An 8-bit state
holds half an E4M3 step, 2^-4 of the value (2^-10 of the run's scale below the normal codes)."""
import pytest
import torch

import block_ref as ref
import quantized_moe_route_amd as q

pytestmark = pytest.mark.gpu

BF16, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
U = 2.0 ** -24
SHAPES = [(1,), (3,), (4,), (255,), (256,), (257,), (1023,), (1024,), (1025,), (16, 264), (5, 1001), (4096,), (4097,), (70000,)]


def tensors(shapes, pt, gt, seed=0, sd=0.02):
    g = torch.Generator().manual_seed(seed)
    p = [(torch.randn(*s, generator=g) * sd).cuda() for s in shapes]
    gr = [(torch.randn(*s, generator=g) * 2e-3).to(gt).cuda() for s in shapes]
    return p, [t.to(pt) for t in p], gr


def encode(a):
    """(codes, scales, decoded) of one tensor by the definition, fp32."""
    n = a.numel()
    b = torch.zeros(-(-n // 256) * 256, device=a.device)
    b[:n] = a.reshape(-1)
    b = b.view(-1, 256)
    s = b.abs().amax(1) * (1.0 / 448.0)
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    c = torch.where(s[:, None] == 0, torch.zeros_like(b), b / torch.where(s == 0, torch.ones_like(s), s)[:, None]).to(E4M3)
    return c.view(torch.uint8).view(-1)[:n].view(a.shape), s


def decode(c, s):
    f = c.view(E4M3).float().reshape(-1)
    return (f * s.repeat_interleave(256)[:f.numel()]).view(c.shape)


def mirror32(p, g, m, v, t, lr, betas, eps, wd):
    """The new moments as the definition writes them, each operation rounded to fp32."""
    m = m * betas[0] + g * (1 - betas[0])
    v = v * betas[1] + g * g * (1 - betas[1])
    return m, v


@pytest.mark.parametrize("pt,gt,master", [(F32, F32, False), (F32, BF16, False), (BF16, BF16, True), (BF16, F32, False), (F32, F32, True)])
@pytest.mark.parametrize("clip", [0.0, 0.05])
def test_fp32_states(pt, gt, master, clip):
    w, p, g = tensors(SHAPES, pt, gt)
    mast = [t.clone() for t in w] if master else None
    wd = [0.01 * (i % 3) for i in range(len(p))]
    ls = [1.0 + 0.5 * (i % 2) for i in range(len(p))]
    st = q.AdamW.new_state(p)
    opt = q.AdamW(p, g, **st, master=mast, weight_decay=wd, lr_scale=ls, max_norm=clip, eps=1e-6)
    want = [(t.to(F64) if not master else mast[i].to(F64), torch.zeros_like(t, dtype=F64), torch.zeros_like(t, dtype=F64)) for i, t in enumerate(p)]
    norm = torch.zeros((), device="cuda")
    for step in range(1, 4):
        if step > 1:
            for i, t in enumerate(tensors(SHAPES, pt, gt, seed=step)[2]):
                g[i].copy_(t)
        total = float(torch.stack([t.to(F64).square().sum() for t in g]).sum().sqrt())
        c = clip / max(clip, total) if clip else 1.0
        before = [t.clone() for t in p]
        opt.step(1e-2, grad_norm=norm if clip else None)
        if clip:
            assert abs(float(norm) - total) <= 4 * U * total
        for i in range(len(p)):
            src = want[i][0] if master or pt == F32 else before[i].to(F64)  # a bf16 parameter starts from its rounding
            new = ref.adamw(src, g[i], want[i][1], want[i][2], step, 1e-2 * ls[i], (0.9, 0.999), 1e-6, wd[i], c)
            want[i] = new
            for got, x, k in ((st["m"][i], new[1], "m"), (st["v"][i], new[2], "v")):
                assert float((got.to(F64) - x).abs().max()) <= step * 16 * U * float(x.abs().max()) + 1e-44, (i, step, k)
            bound = step * 16 * U * (new[0].abs() + 2e-2 * ls[i])
            if master:
                assert ((mast[i].to(F64) - new[0]).abs() <= bound).all(), (i, step)
                assert torch.equal(p[i], mast[i].to(pt))
            else:
                if pt == BF16:
                    bound = bound + 2.0 ** -8 * new[0].abs()
                assert ((p[i].to(F64) - new[0]).abs() <= bound).all(), (i, step)


@pytest.mark.parametrize("pt,gt", [(F32, F32), (BF16, BF16), (F32, BF16)])
def test_8bit_states_are_the_definitions_bits(pt, gt):
    w, p, g = tensors(SHAPES, pt, gt)
    for t in g:  # runs of zeros, tiny and large gradients side by side
        f = t.view(-1)
        f[: f.numel() // 3] *= 1e-6
        if f.numel() > 600:
            f[256:512] = 0
    st = q.AdamW.new_state(p, e4m3=True)
    opt = q.AdamW(p, g, **st, eps=1e-6)
    m, v = [torch.zeros_like(t, dtype=F32) for t in p], [torch.zeros_like(t, dtype=F32) for t in p]
    for step in range(1, 5):
        before = [t.clone() for t in p]
        opt.step(1e-3)
        for i in range(len(p)):
            nm, nv = mirror32(None, g[i].float(), m[i], v[i].square(), step, 1e-3, (0.9, 0.999), 1e-6, 0.01)
            root = nv.sqrt()
            cm, sm = encode(nm)
            cv, sv = encode(root)
            cv = torch.where((cv == 0) & (root > 0) & (sv.repeat_interleave(256)[:root.numel()].view(root.shape) > 0), torch.ones_like(cv), cv)
            assert torch.equal(opt.m_scale[i], sm) and torch.equal(opt.v_scale[i], sv), (i, step)
            assert torch.equal(decode(st["m"][i], sm), decode(cm, sm)) and torch.equal(st["v"][i], cv), (i, step)
            m[i], v[i] = decode(st["m"][i], sm), decode(st["v"][i], sv)
            want = ref.adamw(before[i], torch.zeros_like(nm), nm / 0.9, nv / 0.999, step, 1e-3, (0.9, 0.999), 1e-6, 0.01)[0]
            bound = 32 * U * (before[i].to(F64).abs() + 2e-2) + (2.0 ** -8 * want.abs() if pt == BF16 else 0)
            assert ((p[i].to(F64) - want).abs() <= bound).all(), (i, step)


def test_a_lost_second_moment_does_not_blow_up_the_step():
    p = [torch.zeros(256, device="cuda")]
    g = [torch.full((256,), 1e-9, device="cuda")]
    g[0][0] = 1.0
    st = q.AdamW.new_state(p, e4m3=True)
    opt = q.AdamW(p, g, **st, weight_decay=0.0)
    for _ in range(20):
        opt.step(1e-3)
    assert (st["v"][0] > 0).all()
    assert float(p[0].abs().max()) <= 20 * 1e-3 * 1.01


def test_unaligned_views_and_many_tensors():
    n = 300
    sizes = [1 + (i * 37) % 900 for i in range(n)]
    bank = [torch.randn(sum(sizes) + 1, device="cuda") for _ in range(4)]
    cut = lambda b: [t for t in b[1:].split(sizes)]  # noqa: E731  (4-byte aligned only)
    p, g, m, v = (cut(b) for b in bank)
    for t in v:
        t.abs_()
    want = [ref.adamw(p[i], g[i], m[i], v[i], 8, 1e-2, (0.9, 0.999), 1e-8, 0.01) for i in range(n)]
    q.AdamW(p, g, m=m, v=v, step=7).step(1e-2)
    for i in range(n):
        for got, x in zip((p[i], m[i], v[i]), want[i]):
            assert ((got.to(F64) - x).abs() <= 16 * U * (x.abs() + 0.2) + 1e-12).all(), i


@pytest.mark.parametrize("pt", [F32, BF16])
@pytest.mark.parametrize("clip", [0.0, 0.3])
def test_8bit_states_at_any_alignment_have_the_same_bits(pt, clip):
    """Views that begin anywhere take the element-wise loads: the same arithmetic."""
    sizes = [1 + (i * 211) % 1900 for i in range(60)]
    n = sum(sizes)
    w, g = (torch.randn(n, device="cuda") * s for s in (0.02, 2e-3))

    def run(shift):
        bank = lambda t, dt: torch.cat([torch.zeros(shift, device="cuda"), t]).to(dt)[shift:].split(sizes)  # noqa: E731
        p, gr = bank(w, pt), bank(g, pt)
        if not shift:  # buffers of their own
            p, gr = [t.clone() for t in p], [t.clone() for t in gr]
        codes = [list(torch.zeros(n + shift, device="cuda", dtype=torch.uint8)[shift:].split(sizes)) for _ in range(2)]
        st = q.AdamW.new_state(p, e4m3=True) | (dict(m=codes[0], v=codes[1]) if shift else {})
        o = q.AdamW(p, gr, **st, max_norm=clip)
        for _ in range(3):
            o.step(1e-2)
        return p, o

    pa, a = run(0)
    pb, b = run(1)
    for x, y in ((pa, pb), (a.m, b.m), (a.v, b.v), (a.m_scale, b.m_scale), (a.v_scale, b.v_scale)):
        assert all(torch.equal(s, t) for s, t in zip(x, y))


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_norm_that_is_not_finite_skips_the_step(e4m3):
    w, p, g = tensors([(300,), (5, 100)], F32, F32)
    st = q.AdamW.new_state(p, e4m3=e4m3)
    opt = q.AdamW(p, g, **st, max_norm=1.0)
    opt.step(1e-2)
    keep = [t.clone() for t in (*p, *opt.m, *opt.v)]
    kept_scales = [t.clone() for t in (*opt.m_scale, *opt.v_scale) if t is not None]
    good = g[1].clone()
    norm = torch.zeros(1, device="cuda")
    for bad in (float("inf"), float("nan")):
        g[1][0, 0] = bad
        opt.step(1e-2, grad_norm=norm)
        assert not torch.isfinite(norm).any()
        assert all(torch.equal(a, b) for a, b in zip(keep, (*p, *opt.m, *opt.v)))
    g[1].copy_(good)
    opt.step(1e-2)
    twin = [t.clone() for t in keep[:2]]  # the same second step without the bad ones between
    scales = dict(m_scale=kept_scales[:2], v_scale=kept_scales[2:]) if e4m3 else {}
    q.AdamW(twin, g, m=keep[2:4], v=keep[4:6], max_norm=1.0, step=1, **scales).step(1e-2)
    assert all(torch.equal(a, b) for a, b in zip(p, twin))


@pytest.mark.parametrize("clip", [0.0, 0.01])
@pytest.mark.parametrize("e4m3", [False, True])
def test_captured_steps_count_their_replays(clip, e4m3):
    def fresh():
        w, p, g = tensors([(1000,), (33, 70)], F32, F32, sd=0.5)
        return p, g, q.AdamW(p, g, **q.AdamW.new_state(p, e4m3=e4m3), max_norm=clip, betas=(0.8, 0.9))

    p, g, opt = fresh()
    pe, ge, eager = fresh()
    lr = torch.tensor(1e-2, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        opt.step(lr)
    for k in range(4):
        lr.fill_(1e-2 / (k + 1))
        for a, b in zip(g, ge):
            a.mul_(-0.7)
            b.mul_(-0.7)
        graph.replay()
        eager.step(lr)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*p, *opt.m, *opt.v), (*pe, *eager.m, *eager.v))), k


def test_new_gradients_another_stream_and_no_tensors():
    w, p, g = tensors([(100,), (2000,)], F32, F32)
    pe = [t.clone() for t in p]
    o, e = q.AdamW(p, g, **q.AdamW.new_state(p)), q.AdamW(pe, g, **q.AdamW.new_state(pe))
    g2 = [t.to(BF16) * 2 for t in g]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o.step(1e-3)
        o.set_grads(g2)
        o.step(1e-3)
    torch.cuda.current_stream().wait_stream(s)
    e.step(1e-3)
    e.set_grads(g2)
    e.step(1e-3)
    assert all(torch.equal(a, b) for a, b in zip(p, pe))
    for clip in (0.0, 1.0):
        z = q.AdamW([], [], m=[], v=[], device="cuda", max_norm=clip)
        z.step(1e-3)
    t = torch.zeros(0, device="cuda")
    q.AdamW([t], [t.clone()], **q.AdamW.new_state([t])).step(1e-3)


def test_python_refusals():
    w, p, g = tensors([(100,), (200,)], F32, F32)
    st = q.AdamW.new_state(p)
    with pytest.raises(q.MoeError, match="overlaps"):
        q.AdamW([p[0], p[0]], [g[0], g[0]], m=[st["m"][0], st["m"][0]], v=[st["v"][0], st["v"][0]])
    with pytest.raises(q.MoeError, match="overlaps"):
        q.AdamW(p, p, **st)
    with pytest.raises(ValueError):
        q.AdamW(p, g[:1], **st)
    with pytest.raises((ValueError, TypeError)):
        q.AdamW(p, g, m=st["m"], v=st["v"], m_scale=[None, None], v_scale=[None, None])
    with pytest.raises(ValueError):
        q.AdamW(p, [g[0].cpu(), g[1]], **st)
    with pytest.raises(TypeError):
        q.AdamW([t.half() for t in p], g, **st)
    with pytest.raises(q.MoeError):
        q.AdamW(p, g, **st, betas=(1.0, 0.9))
    o = q.AdamW(p, g, **st)
    with pytest.raises(q.MoeError):
        o.step(float("nan"))
    with pytest.raises(q.MoeError):
        o.step(1e-3, grad_norm=torch.zeros(1, device="cuda"))  # without max_norm
    with pytest.raises(q.MoeError):
        o.set_step(-1)
    before = [t.clone() for t in p]
    o = q.AdamW(p, g, **st, max_norm=1.0)
    lr = torch.full((1,), 1e-3, device="cuda")
    for taken in (p[0].view(-1)[:1], g[1].view(-1)[-1:], o.m[0].view(-1)[1:2], lr):  # the norm where the step reads or writes
        with pytest.raises(q.MoeError):
            o.step(lr, grad_norm=taken)
    assert all(torch.equal(a, b) for a, b in zip(before, p))
