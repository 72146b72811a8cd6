"""Refusals of the row operators: host checks of the C ABI and of the binding. No call
here reaches a kernel, so none needs a GPU."""
import ctypes

import pytest
import torch

import expert_routing_grouped_layer_b200 as moe
from expert_routing_grouped_layer_b200 import build as moe_build
from expert_routing_grouped_layer_b200 import workloads as W

BAD, UNS, WS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE, moe.MOE_OK
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


def test_norm(lib):
    def f(kind=0, dt=0, x=256, ldx=64, T=4, H=64, w=256, b=256, eps=1e-6, y=256, ldy=64, mean=256, rstd=256):
        return lib.moe_norm(kind, dt, x, ldx, T, H, w, b, ctypes.c_float(eps), y, ldy, mean, rstd, None)
    for bad in (dict(kind=2), dict(kind=-1), dict(dt=3), dict(dt=-1), dict(x=None), dict(y=None), dict(T=-1),
                dict(H=0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(ldx=63), dict(ldy=63),
                dict(x=257), dict(y=257), dict(w=258), dict(b=258), dict(mean=258), dict(rstd=258),
                dict(dt=2, x=258)):
        assert f(**bad) == BAD, bad
    assert f(H=16385, ldx=16385, ldy=16385) == UNS
    assert f(T=0, x=None, y=None) == OK


def test_norm_backward(lib):
    need = lib.moe_norm_backward_workspace_bytes(4, 64)
    assert need == 4 * 2 * 64 * 4  # a pair of rows per CTA, one CTA per row
    assert lib.moe_norm_backward_workspace_bytes(-1, 64) == 0
    assert lib.moe_norm_backward_workspace_bytes(4, 0) == 0
    assert lib.moe_norm_backward_workspace_bytes(4, 16385) == 0

    def f(kind=0, dt=0, dy=256, lddy=64, x=256, ldx=64, T=4, H=64, w=256, mean=256, rstd=256, dx=256, lddx=64,
          dw=256, db=256, ws=256, n=need):
        return lib.moe_norm_backward(kind, dt, dy, lddy, x, ldx, T, H, w, mean, rstd, dx, lddx, dw, db, ws, n,
                                     None)
    for bad in (dict(kind=3), dict(dt=7), dict(dy=None), dict(x=None), dict(T=-1), dict(H=0), dict(lddy=1),
                dict(ldx=1), dict(lddx=1), dict(mean=None), dict(rstd=None), dict(ws=None), dict(ws=264),
                dict(dw=257), dict(db=257), dict(dx=257), dict(dy=257), dict(w=257)):
        assert f(**bad) == BAD, bad
    assert f(n=need - 1) == WS
    assert f(H=16385, ldx=16385, lddy=16385, lddx=16385) == UNS
    assert f(dx=None, dw=None, db=None) == OK  # nothing wanted
    assert f(kind=1, dx=None, dw=None) == OK   # the RMS norm has no bias gradient


def _cfg(**kw):
    return moe.make_config(W.CONFIGS["tiny_bf16"].replace(**kw))


def test_route(lib):
    def f(c, dt=2, l=256, ld=16, T=4, b=256, i=256, w=256):
        return lib.moe_route(ctypes.byref(c), dt, l, ld, T, b, i, w, None)

    def g(c, dt=2, l=256, ld=16, T=4, i=256, w=256, d=256, ldd=16):
        return lib.moe_route_backward(ctypes.byref(c), dt, l, ld, T, i, w, d, ldd, None)
    c = _cfg()
    for bad in (dict(dt=3), dict(l=None), dict(ld=15), dict(T=-1), dict(b=257), dict(i=None), dict(w=None),
                dict(i=258), dict(w=258), dict(l=258)):
        assert f(c, **bad) == BAD, bad
    for bad in (dict(dt=-1), dict(l=None), dict(ld=15), dict(T=-1), dict(i=None), dict(w=None), dict(d=None),
                dict(ldd=15), dict(d=258), dict(i=257), dict(w=257)):
        assert g(c, **bad) == BAD, bad
    assert f(c, T=0, l=None) == OK and g(c, T=0, l=None) == OK
    broken = _cfg()
    broken.n_group = 3
    assert f(broken) == BAD and g(broken) == BAD


def test_combine_backward(lib):
    def f(c, dout=256, y=256, row=256, w=256, T=4, dy=256, dw=256):
        return lib.moe_combine_backward(ctypes.byref(c), dout, y, row, w, T, dy, dw, None)
    c = _cfg()
    for bad in (dict(dout=None), dict(y=None), dict(row=None), dict(w=None), dict(dy=None), dict(T=-1),
                dict(dout=264), dict(y=264), dict(dy=264), dict(row=257), dict(w=257), dict(dw=257),
                dict(T=0x20000000)):
        assert f(c, **bad) == BAD, bad
    assert f(c, T=0, dout=None) == OK


def test_linear(lib):
    def f(dt=0, x=256, ldx=64, w=256, ldw=64, b=256, r=256, ldr=32, act=0, M=4, N=32, K=64, y=256, ldy=32, p=256,
          ldp=32, st=None):
        return lib.moe_linear(dt, x, ldx, w, ldw, b, r, ldr, act, M, N, K, y, ldy, p, ldp, st, None)
    for bad in (dict(dt=3), dict(x=None), dict(w=None), dict(y=None), dict(M=-1), dict(N=0), dict(K=0),
                dict(act=5), dict(act=-1), dict(ldx=60), dict(ldw=68), dict(ldx=56), dict(x=264), dict(w=264),
                dict(ldy=31), dict(ldr=31), dict(ldp=31), dict(y=257), dict(r=257), dict(p=257), dict(b=258),
                dict(st=257), dict(M=0x7fffffff)):
        assert f(**bad) == BAD, bad
    assert f(dt=2) == UNS  # fp32 operands
    assert f(M=0, x=None) == OK


def test_linear_backward(lib):
    need = lib.moe_linear_backward_workspace_bytes(4, 32, 64, 0)
    assert need >= 4 * 32 * 2 + 32 * 4
    assert lib.moe_linear_backward_workspace_bytes(4, 0, 64, 0) == 0
    assert lib.moe_linear_backward_workspace_bytes(4, 32, 64, 9) == 0

    def f(dt=0, dy=256, lddy=32, x=256, ldx=64, w=256, ldw=64, p=256, ldp=32, act=2, M=4, N=32, K=64, dx=256,
          lddx=64, dw=256, lddw=64, db=256, ws=256, n=need, st=None):
        return lib.moe_linear_backward(dt, dy, lddy, x, ldx, w, ldw, p, ldp, act, M, N, K, dx, lddx, dw, lddw, db,
                                       ws, n, st, None)
    for bad in (dict(dt=9), dict(dy=None), dict(x=None), dict(w=None), dict(p=None), dict(act=7), dict(M=-1),
                dict(N=0), dict(K=0), dict(lddy=31), dict(ldx=60), dict(ldw=60), dict(ldp=31), dict(lddx=63),
                dict(lddw=63), dict(x=264), dict(w=264), dict(dx=257), dict(dw=257), dict(db=257), dict(ws=None),
                dict(ws=264), dict(st=258), dict(p=257)):
        assert f(**bad) == BAD, bad
    assert f(n=need - 1) == WS
    assert f(dt=2) == UNS
    assert f(dx=None, dw=None, db=None) == OK


F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32


def _refused(why, fn, *args, **kw):
    with pytest.raises(ValueError, match=why):
        fn(*args, **kw)


def test_binding_refuses_before_the_library(lib):
    """The native module checks type, shape and layout, then the device: tensors on the CPU
    pass every check but the last and never reach the library."""
    z = torch.zeros
    cfg = W.CONFIGS["tiny_bf16"]
    E, k, H = cfg.n_routed_experts, cfg.num_experts_per_tok, cfg.hidden
    x, w, t = z(4, 64, dtype=BF), z(64), z(4)
    ws = z(64)
    dev = "not on a CUDA device"
    _refused(dev, moe.moe_norm, x, w, w, 1e-6, x, t, t)
    _refused(dev, moe.moe_norm_backward, x, x, w, t, t, x, w, w, ws)
    l, idx, tw = z(4, E), z(4, k, dtype=I32), z(4, k)
    _refused(dev, moe.moe_route, cfg, l, z(E), idx, tw)
    _refused(dev, moe.moe_route_backward, cfg, l, idx, tw, l)
    d, y, ro = z(4, H, dtype=BF), z(4 * k, H, dtype=BF), z(4 * k, dtype=I32)
    _refused(dev, moe.moe_combine_backward, cfg, d, y, ro, tw, y, tw)
    wt, o = z(8, 64, dtype=BF), z(4, 8, dtype=BF)
    _refused(dev, moe.moe_linear, x, wt, z(8), o, o, o)
    _refused(dev, moe.moe_linear_backward, o, x, wt, o, x, wt, z(8), ws, act="relu")


def test_binding_checks_layout(lib):
    z = torch.zeros
    x, w, t = z(4, 64, dtype=BF), z(64), z(4)
    n = lambda x_=x, w_=w, b_=None, y_=x, m_=None, eps=1e-6, **kw: moe.moe_norm(x_, w_, b_, eps, y_, m_, t, **kw)
    _refused("x is missing", n, x_=None)
    _refused("not a tensor", n, x_=[1, 2])
    _refused("a matrix", n, x_=z(64, dtype=BF))
    _refused("float32 is wanted", n, x_=z(4, 64, dtype=torch.float64))
    _refused("adjacent", n, x_=z(4, 128, dtype=BF)[:, ::2])
    _refused("overlap", n, x_=z(64, dtype=BF).expand(4, 64))
    _refused("overlap", n, y_=z(200, dtype=BF).as_strided((4, 64), (32, 1)))
    _refused("y is missing", n, y_=None)
    _refused(r"shape \(4, 65\), not \(4, 64\)", n, y_=z(4, 65, dtype=BF))
    _refused("torch.float16, not torch.bfloat16", n, y_=z(4, 64, dtype=torch.float16))
    _refused("w has shape", n, w_=z(63))
    _refused("not torch.float32", n, w_=z(64, dtype=BF))
    _refused("contiguous", n, w_=z(128)[::2])
    _refused("mean has shape", n, m_=z(5))
    _refused("strided", n, x_=x.to_sparse())
    with pytest.raises(KeyError):
        n(kind="batch")
    with pytest.raises((ValueError, TypeError)):
        n(eps="a")
    with pytest.raises((ValueError, TypeError)):
        n(eps=None)
    # a single row's stride is not looked at
    _refused("not on a CUDA device", moe.moe_norm, z(64, dtype=BF).as_strided((1, 64), (1, 1)), None, None, 1e-6,
             z(1, 64, dtype=BF))
    cfg = W.CONFIGS["tiny_bf16"]
    E, k, H = cfg.n_routed_experts, cfg.num_experts_per_tok, cfg.hidden
    idx, tw = z(4, k, dtype=I32), z(4, k)
    _refused("logits has 17 columns", moe.moe_route, cfg, z(4, 17), None, idx, tw)
    _refused("topk_idx is torch.float32", moe.moe_route, cfg, z(4, E), None, tw, tw)
    _refused("topk_w has shape", moe.moe_route, cfg, z(4, E), None, idx, z(4, k + 1))
    _refused("dlogits is torch.float32", moe.moe_route_backward, cfg, z(4, E, dtype=BF), idx, tw, z(4, E))
    d, y, ro = z(4, H, dtype=BF), z(4 * k, H, dtype=BF), z(4 * k, dtype=I32)
    _refused("dout has shape", moe.moe_combine_backward, cfg, z(4, H + 1, dtype=BF), y, ro, tw, y, tw)
    _refused("y has shape", moe.moe_combine_backward, cfg, d, z(4, H, dtype=BF), ro, tw, y, tw)
    _refused("contiguous", moe.moe_combine_backward, cfg, z(4, 2 * H, dtype=BF)[:, :H], y, ro, tw, y, tw)
    xl, wt, o = z(4, 64, dtype=BF), z(8, 64, dtype=BF), z(4, 8, dtype=BF)
    _refused("w has shape", moe.moe_linear, xl, z(8, 65, dtype=BF), None, None, o)
    _refused("w is torch.float16", moe.moe_linear, xl, wt.half(), None, None, o)
    _refused("residual has shape", moe.moe_linear, xl, wt, None, z(4, 9, dtype=BF), o)
    _refused("bias is torch.bfloat16", moe.moe_linear, xl, wt, z(8, dtype=BF), None, o)
    _refused("dw has shape", moe.moe_linear_backward, o, xl, wt, None, None, z(8, 63, dtype=BF), None, None)
    with pytest.raises(KeyError):
        moe.moe_linear(xl, wt, None, None, o, act="swish")


def test_missing_binding_fails_loudly(lib, monkeypatch, tmp_path):
    monkeypatch.setattr(moe, "BINDING_PATH", str(tmp_path / "nope.so"))
    monkeypatch.setattr(moe, "_binding", None)
    with pytest.raises(RuntimeError, match="not built"):
        moe.moe_norm(torch.zeros(4, 64), None, None, 1e-6, torch.zeros(4, 64))


def _seven():
    """Every operator with small CPU tensors (refused at the latest for their device), as (call,
    arguments that are tensors)."""
    z = torch.zeros
    cfg = W.CONFIGS["tiny_bf16"]
    E, k, H = cfg.n_routed_experts, cfg.num_experts_per_tok, cfg.hidden
    m = lambda *s: z(*s, dtype=BF)
    return [(moe.moe_norm, (m(4, 64), z(64), z(64), 1e-6, m(4, 64), z(4), z(4))),
            (moe.moe_norm_backward, (m(4, 64), m(4, 64), z(64), z(4), z(4), m(4, 64), z(64), z(64), z(64))),
            (moe.moe_route, (cfg, z(4, E), z(E), z(4, k, dtype=I32), z(4, k))),
            (moe.moe_route_backward, (cfg, z(4, E), z(4, k, dtype=I32), z(4, k), z(4, E))),
            (moe.moe_combine_backward, (cfg, m(4, H), m(4 * k, H), z(4 * k, dtype=I32), z(4, k), m(4 * k, H), z(4, k))),
            (moe.moe_linear, (m(4, 64), m(8, 64), z(8), m(4, 8), m(4, 8), m(4, 8))),
            (moe.moe_linear_backward, (m(4, 8), m(4, 64), m(8, 64), m(4, 8), m(4, 64), m(8, 64), z(8), z(64)))]


def test_binding_refuses_tensors_that_require_a_gradient(lib):
    """No graph is recorded, so nothing that torch would record passes unnoticed."""
    for fn, args in _seven():
        for i, a in enumerate(args):
            if not (isinstance(a, torch.Tensor) and a.is_floating_point()):
                continue
            given = list(args)
            given[i] = a.clone().requires_grad_()
            _refused("requires a gradient", fn, *given)
            with torch.no_grad():
                _refused("not on a CUDA device", fn, *given)
            given[i] = given[i].detach()
            _refused("not on a CUDA device", fn, *given)
