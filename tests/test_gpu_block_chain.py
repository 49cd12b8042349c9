"""One training step of a whole block through the public calls: norm, routed experts with an adapter, the
dense block added onto them, norm with residual and gate; all gradients back; AdamW on every parameter.
Against the fp64 definitions and the oracle, with the GPU's own stored bf16 values where a call hands them on."""
import numpy as np
import pytest
import torch

import block_ref as ref
import moe_synth as syn
import oracle
import quantized_moe_route_amd as q
from cases import device_layer, host_case

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def rel(a, b):
    b = torch.as_tensor(b)
    return float((a.detach().cpu().to(F64) - b.cpu()).abs().max() / b.cpu().abs().max())


@pytest.mark.parametrize("T", [1, 8, 45])
def test_block_training_step(T):
    w = syn.shrink(syn.WORKLOADS["tiny"], T=T, H=256, I=128, x_dtype="bf16", x_key=71)
    c = host_case(w)
    L = device_layer(c, max_tokens=T)
    D, I = w.H, 192
    g = torch.Generator().manual_seed(T)
    rnd = lambda *s, sd=1.0: torch.randn(*s, generator=g) * sd  # noqa: E731
    wg, wu, wd = (rnd(*s, sd=sd).to(BF16).cuda() for s, sd in (((I, D), D ** -0.5), ((I, D), D ** -0.5), ((D, I), I ** -0.5)))
    n0w, n1w, n2w = (1 + rnd(D, sd=0.1).cuda() for _ in range(3))
    gate = (0.5 + rnd(D, sd=0.1)).cuda()
    r0 = rnd(T, D).cuda()
    dr, dx2 = rnd(T, D, sd=0.1).cuda(), rnd(T, D, sd=0.1).to(BF16).cuda()
    pre = q.BlockNorm(D, max_tokens=T, w_next=n0w)
    out = q.BlockNorm(D, max_tokens=T, w_post=n1w, w_next=n2w, gate="channel", branch_scale=0.7)
    ffn = q.GatedFFN(wg, wu, wd, max_tokens=T)

    # forward
    f0 = pre.forward(r0)
    route = L.route(f0.x)
    sg = L.new_saved_gu(T)
    gu = ffn.new_saved_gu(T)
    y = L.forward(f0.x, route, saved_gu=sg)
    ffn.forward(f0.x, y, accumulate=True, saved_gu=gu)
    f1 = out.forward(r0, y, gate=gate)
    # backward
    b1 = out.backward(f1, y, gate=gate, dr_out=dr, dx=dx2)
    dyb = b1.dy.to(BF16)
    dxl = L.backward_input(f0.x, dyb, route, saved_gu=sg)
    dxl, dw = ffn.backward(f0.x, dyb, saved_gu=gu, dx=dxl, accumulate=True, dw_dtype=F32)
    b0 = pre.backward(f0, dr_out=b1.dr, dx=dxl.to(BF16))
    torch.cuda.synchronize()

    # the same in fp64, each step from what the call before it stored
    assert rel(f0.x, ref.norm(r0, None, None, None, n0w)[1]) <= 2.0 ** -8 * 1.01
    x64 = f0.x.cpu().to(F64).numpy()
    W = c.oracle_weights()
    ids, p, _ = oracle.route(x64, c.wr, None, w.k)
    assert np.array_equal(route.ids.cpu().numpy(), ids)
    yref = torch.as_tensor(oracle.forward(x64, ids, p, W)) + ref.ffn("swiglu", f0.x, wg, wu, wd).cpu()
    assert rel(y, yref) <= 1e-4
    leaf = [t.detach().to(F64).requires_grad_(True) for t in (r0, y, gate, n1w, n2w)]
    r1, x1 = ref.norm(leaf[0], leaf[1], leaf[2], leaf[3], leaf[4], beta=0.7)
    assert rel(f1.r, r1.detach()) <= 1e-6 and rel(f1.x, x1.detach()) <= 2.0 ** -8 * 1.01
    ((dr.to(F64) * r1).sum() + (dx2.to(F64) * x1).sum()).backward()
    for a, t in zip((b1.dr, b1.dy, b1.dgate, b1.dw_post, b1.dw_next), leaf):
        assert rel(a, t.grad) <= 1e-5
    (fx, *fw), _ = ref.ffn_grads("swiglu", f0.x, wg, wu, wd, dyb)
    want = torch.as_tensor(oracle.backward_input(x64, dyb.cpu().to(F64).numpy(), ids, p, c.wr, W)) + fx.cpu()
    assert rel(dxl, want) <= 1e-4
    for a, b in zip(dw, fw):
        assert rel(a, b) <= 1e-4
    leaf = [t.detach().to(F64).requires_grad_(True) for t in (r0, n0w)]
    r, x = ref.norm(leaf[0], None, None, None, leaf[1])
    ((b1.dr.to(F64) * r).sum() + (dxl.to(BF16).to(F64) * x).sum()).backward()
    assert rel(b0.dr, leaf[0].grad) <= 1e-5 and rel(b0.dw_next, leaf[1].grad) <= 1e-5

    # the optimizer over all of it, then the forward on the new weights
    params = [wg, wu, wd, n0w, n1w, n2w, gate]
    grads = [*dw, b0.dw_next, b1.dw_post, b1.dw_next, b1.dgate]
    master = [wg.float(), wu.float(), wd.float(), None, None, None, None]
    before = [t.clone() for t in params]
    zero = [torch.zeros_like(t, dtype=F64) for t in params]
    opt = q.AdamW(params, grads, **q.AdamW.new_state(params), master=master, max_norm=1.0, weight_decay=[0.1] * 3 + [0.0] * 4)
    opt.step(1e-2)
    norm = float(torch.stack([t.to(F64).square().sum() for t in grads]).sum().sqrt())
    for i, t in enumerate(params):
        new = ref.adamw(before[i], grads[i], zero[i], zero[i], 1, 1e-2, (0.9, 0.999), 1e-8, 0.1 if i < 3 else 0.0, 1.0 / max(1.0, norm))[0]
        assert float(((t if master[i] is None else master[i]).to(F64) - new).abs().max()) <= 1e-6
    y2 = ffn.forward(f0.x, out_dtype=F32)
    assert rel(y2, ref.ffn("swiglu", f0.x, wg, wu, wd)) <= 1e-5
    L.close()
