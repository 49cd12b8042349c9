"""Host-side checks of include/moe_block.h: defaults, sizes and refusals (no device is touched), and the
fp64 definitions against differences."""
import ctypes

import pytest
import torch

import block_ref as ref
from quantized_moe_route_amd import _lib as C

WS = 0x100000


def make(kind, **kw):
    d = {"ffn": C.MoeFfnDesc, "norm": C.MoeNormDesc, "adamw": C.MoeAdamwDesc}[kind]()
    getattr(C.lib(), f"moe_{kind}_desc_init")(ctypes.byref(d))
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def size(kind, d):
    n = ctypes.c_size_t()
    st = getattr(C.lib(), f"moe_{kind}_workspace_size")(ctypes.byref(d), ctypes.byref(n))
    return st, n.value


@pytest.mark.parametrize("kind,bad", [
    ("ffn", [dict(width=0), dict(width=12), dict(width=-8), dict(inter=0), dict(inter=20), dict(width=(1 << 20) + 8), dict(max_tokens=-1),
             dict(act=2), dict(act=-1), dict(flags=2)]),
    ("norm", [dict(width=0), dict(width=16385), dict(max_tokens=-1), dict(max_tokens=(1 << 30) + 1), dict(r_dtype=2), dict(y_dtype=-1), dict(x_dtype=9), dict(w_dtype=5),
              dict(gate=4), dict(gate=-1), dict(eps_post=0.0), dict(eps_next=-1.0), dict(eps_post=float("nan")),
              dict(res_scale=float("inf")), dict(branch_scale=float("nan")), dict(flags=8)]),
    ("adamw", [dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=float("nan")), dict(eps=0.0), dict(eps=1e-60), dict(max_norm=-1.0),
               dict(max_norm=float("inf")), dict(max_norm=1e-60), dict(state=2), dict(max_tensors=0), dict(max_elements=-1),
               dict(max_elements=1 << 41)])])
def test_descriptors(kind, bad):
    L = C.lib()
    st, n = size(kind, make(kind))
    assert st == C.MOE_OK and n > 0
    for kw in bad:
        st, _ = size(kind, make(kind, **kw))
        assert st in (C.MOE_ERR_INVALID_ARG, C.MOE_ERR_UNSUPPORTED), kw
        assert L.moe_last_error(), kw
    getattr(L, f"moe_{kind}_desc_init")(None)
    f = getattr(L, f"moe_{kind}_workspace_size")
    assert f(None, ctypes.byref(ctypes.c_size_t())) == C.MOE_ERR_INVALID_ARG
    assert f(ctypes.byref(make(kind)), None) == C.MOE_ERR_INVALID_ARG
    getattr(L, f"moe_{kind}_destroy")(None)


def ffn(ws_bytes=None, weights=(0x10000, 0x20000, 0x30000), ws=WS, **kw):
    L = C.lib()
    d = make("ffn", **{**dict(width=64, inter=48, max_tokens=8), **kw})
    h = ctypes.c_void_p()
    st = L.moe_ffn_create(ctypes.byref(d), *weights, ws, size("ffn", d)[1] if ws_bytes is None else ws_bytes, ctypes.byref(h))
    return st, h


def test_ffn_refusals():
    L = C.lib()
    BAD = C.MOE_ERR_INVALID_ARG
    assert ffn(weights=(0, 0x20000, 0x30000))[0] == BAD
    assert ffn(weights=(0x10008, 0x20000, 0x30000))[0] == BAD
    assert ffn(ws_bytes=16)[0] == C.MOE_ERR_WORKSPACE
    assert ffn(ws=WS + 16)[0] == C.MOE_ERR_WORKSPACE
    assert ffn(ws=0)[0] == C.MOE_ERR_WORKSPACE
    st, h = ffn()
    assert st == C.MOE_OK
    x, y, dy, gu, dx, w = 0x4000000, 0x5000000, 0x6000000, 0x7000000, 0x8000000, 0x9000000
    assert L.moe_ffn_forward(h, x, 0, y, 0, 0, None, None) == C.MOE_OK  # no tokens, nothing enqueued
    for args in [(None, x, 4, y, 0, 0, None), (h, x, 9, y, 0, 0, None), (h, x, -1, y, 0, 0, None), (h, None, 4, y, 0, 0, None),
                 (h, x, 4, None, 0, 0, None), (h, x, 4, y, 2, 0, None), (h, x + 8, 4, y, 0, 0, None), (h, x, 4, y + 4, 0, 0, None),
                 (h, x, 4, y, 0, 0, gu + 8), (h, x, 4, x, 0, 0, None), (h, x, 4, x + 4 * 64 * 2 - 16, 0, 0, None),
                 (h, x, 4, y, 0, 0, y + 16), (h, x, 4, 0x10000, 0, 0, None), (h, WS, 4, y, 0, 0, None)]:
        assert L.moe_ffn_forward(*args, None) == BAD, args
    for args in [(None, x, dy, 4, gu, dx, 0, 0, w, None, None, 0), (h, x, dy, 9, gu, dx, 0, 0, w, None, None, 0),
                 (h, None, dy, 4, gu, dx, 0, 0, w, None, None, 0), (h, x, None, 4, gu, dx, 0, 0, w, None, None, 0),
                 (h, x, dy, 4, gu, dx, 3, 0, w, None, None, 0), (h, x, dy, 4, gu, dx, 0, 0, w, None, None, 7),
                 (h, x, dy, 4, gu, dy, 0, 0, w, None, None, 0), (h, x, dy, 4, gu, dx, 0, 0, w, w, None, 0),
                 (h, x, dy, 4, gu, dx + 4, 0, 0, w, None, None, 0), (h, x, dy, 4, gu, dx, 0, 0, 0x20000, None, None, 0)]:
        assert L.moe_ffn_backward(*args, None) == BAD, args
    assert L.moe_ffn_backward(h, x, dy, 4, gu, None, 0, 0, None, None, None, 0, None) == C.MOE_OK  # nothing asked for
    L.moe_ffn_destroy(h)
    st, h = ffn(flags=0)
    assert L.moe_ffn_backward(h, x, dy, 4, gu, dx, 0, 0, None, None, None, 0, None) == BAD
    L.moe_ffn_destroy(h)


def norm(w=(0x10000, 0x20000), ws=WS, **kw):
    d = make("norm", **{**dict(width=64, max_tokens=8), **kw})
    h = ctypes.c_void_p()
    st = C.lib().moe_norm_create(ctypes.byref(d), *w, ws, size("norm", d)[1], ctypes.byref(h))
    return st, h


def test_norm_refusals():
    L = C.lib()
    BAD = C.MOE_ERR_INVALID_ARG
    assert norm(w=(None, 0x20000))[0] == BAD and norm(w=(0x10000, None))[0] == BAD
    assert norm(flags=C.MOE_NORM_POST)[0] == BAD  # w_next without its flag
    assert norm(w=(0x10002, 0x20000))[0] == BAD
    assert norm(ws=None)[0] == C.MOE_ERR_WORKSPACE
    assert norm(ws=None, flags=C.MOE_NORM_POST | C.MOE_NORM_NEXT)[0] == C.MOE_OK
    r, y, g, ro, x, rs, a, b, c = (0x1000000 * k for k in range(2, 11))
    st, h = norm(gate=C.MOE_GATE_TOKEN)
    assert st == C.MOE_OK
    fwd = dict(h=h, r=r, y=y, gate=g, T=4, r_out=ro, x=x, rstd=rs)
    for kw in [dict(h=None), dict(r=None), dict(gate=None), dict(T=9), dict(T=-1), dict(r_out=None), dict(x=None), dict(y=None),
               dict(y=None, r_out=None), dict(r=r + 2), dict(x=x + 1), dict(gate=g + 2), dict(rstd=rs + 1), dict(r_out=y), dict(r_out=r + 4),
               dict(x=ro), dict(x=0x10000)]:
        assert L.moe_norm_forward(*{**fwd, **kw}.values(), None) == BAD, kw
    bwd = dict(h=h, y=y, gate=g, r_out=ro, rstd=rs, dr_out=a, dx=x, T=4, dr=b, dy=c, dgate=None, dw_post=None, dw_next=None)
    for kw in [dict(h=None), dict(T=9), dict(dr=None), dict(dy=None), dict(dx=None), dict(r_out=None), dict(rstd=None), dict(gate=None),
               dict(y=None), dict(dr=y), dict(dy=y), dict(dr=a + 4), dict(dy=c + 2), dict(dgate=g), dict(dw_post=0x10000),
               dict(dw_post=0x3000001), dict(dw_next=WS)]:
        assert L.moe_norm_backward(*{**bwd, **kw}.values(), None) == BAD, kw
    L.moe_norm_destroy(h)
    st, h = norm(flags=C.MOE_NORM_NEXT, w=(None, 0x20000))
    assert st == C.MOE_OK
    assert L.moe_norm_backward(*{**bwd, "h": h, "gate": None}.values(), None) == BAD  # without MOE_NORM_BACKWARD
    L.moe_norm_destroy(h)
    st, h = norm(flags=C.MOE_NORM_POST, w=(0x10000, None))
    assert L.moe_norm_forward(h, r, None, None, 4, None, None, rs, None) == BAD  # nothing to compute
    assert L.moe_norm_forward(h, r, y, None, 4, ro, x, rs, None) == BAD  # x without MOE_NORM_NEXT
    L.moe_norm_destroy(h)


def test_adamw_refusals():
    L = C.lib()
    BAD = C.MOE_ERR_INVALID_ARG
    d = make("adamw", max_tensors=2, max_elements=2000)
    h = ctypes.c_void_p()
    n = size("adamw", d)[1]
    assert L.moe_adamw_create(ctypes.byref(d), WS, n - 1, ctypes.byref(h)) == C.MOE_ERR_WORKSPACE
    assert L.moe_adamw_create(ctypes.byref(d), WS, n, None) == BAD
    assert L.moe_adamw_create(ctypes.byref(d), WS, n, ctypes.byref(h)) == C.MOE_OK
    assert L.moe_adamw_step(h, 1e-3, None, None, None) == BAD and b"bound" in L.moe_last_error()
    assert L.moe_adamw_set_step(h, -1, None) == BAD and L.moe_adamw_set_step(None, 0, None) == BAD

    def tensor(i=0, **kw):
        e = C.MoeAdamwTensor()
        base = 0x10000000 * (i + 1)
        e.param, e.grad, e.m, e.v, e.n, e.lr_scale = base, base + 0x100000, base + 0x200000, base + 0x300000, 1000, 1.0
        for k, v in kw.items():
            setattr(e, k, v)
        return e

    def bind(*es):
        return L.moe_adamw_bind(h, (C.MoeAdamwTensor * max(1, len(es)))(*es), len(es), None)

    ok = tensor()
    for kw in [dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(n=-1), dict(n=2001), dict(param_dtype=2), dict(grad_dtype=-1),
               dict(m_scale=0x5000), dict(param=0x10000002), dict(m=0x10200001), dict(weight_decay=float("nan")), dict(lr_scale=float("inf")),
               dict(grad=ok.param), dict(grad=ok.param + 3996), dict(v=ok.m), dict(master=ok.param), dict(master=0x10000000 + 2)]:
        assert bind(tensor(**kw)) == BAD, kw
    assert bind(ok, ok) == BAD and b"overlaps" in L.moe_last_error()
    assert bind(ok, tensor(1, m=ok.m)) == BAD and bind(ok, tensor(1, param=ok.grad)) == BAD
    for kw in (dict(grad=WS), dict(m=WS + size("adamw", d)[1] - 4)):
        assert bind(tensor(**kw)) == BAD and b"workspace" in L.moe_last_error(), kw
    assert bind(ok, tensor(1), tensor(2)) == BAD  # more than max_tensors
    assert bind(tensor(n=1001), tensor(1)) == BAD  # more than max_elements
    assert L.moe_adamw_bind(h, None, 1, None) == BAD and L.moe_adamw_bind(None, None, 0, None) == BAD
    L.moe_adamw_destroy(h)
    d = make("adamw", state=C.MOE_STATE_E4M3)
    assert L.moe_adamw_create(ctypes.byref(d), WS, size("adamw", d)[1], ctypes.byref(h)) == C.MOE_OK
    assert bind(ok) == BAD and b"scale" in L.moe_last_error()
    L.moe_adamw_destroy(h)


def test_workspace_covers_the_chunks_of_any_set():
    """Tensors of every size: the chunk map's room is counted from max_tensors and max_elements alone."""
    for tensors, elements in [(1, 1), (1, 1 << 22), (1000, 1000), (7, (1 << 22) - 1), (600, 1 << 28), (1, 5000)]:
        d = make("adamw", max_tensors=tensors, max_elements=elements)
        st, n = size("adamw", d)
        assert st == C.MOE_OK
        for total in {1, elements, min(elements, (1 << 22) - 1), min(elements, 1 << 22)}:
            chunk = 1024 if total < 1 << 22 else 4096
            most = total // chunk + min(tensors, total)  # each tensor's last chunk may be partial
            assert n >= 4 * most + 80 * tensors


@pytest.mark.parametrize("act", ["swiglu", "situ"])
def test_ffn_definition_against_differences(act):
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, wg, wu, wd, dy = rnd(3, 16), rnd(24, 16), rnd(24, 16) * 3, rnd(16, 24), rnd(3, 16)
    grads, _ = ref.ffn_grads(act, x, wg, wu, wd, dy)
    args, h = [x, wg, wu, wd], 1e-6
    for i, grad in enumerate(grads):
        v = rnd(*args[i].shape)
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * v, args[i] - h * v
        fd = float((dy * (ref.ffn(act, *up) - ref.ffn(act, *dn))).sum()) / (2 * h)
        assert abs(fd - float((grad * v).sum())) <= 1e-7 * float((grad * v).abs().sum()) + 1e-8
