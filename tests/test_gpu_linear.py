"""moe_linear and moe_linear_backward against the 64-bit formulas.

Tolerances. The tensor cores add K products in steps of 16, each step off by at most one
unit of 2^-23 of the sum of magnitudes, plus a tree of partial sums: (K / 16 + 16) 2^-23
sum |x w|. The activations' slopes are below 1.13, their own evaluation is off by at most
2^-21 (1 + |z|). Rounding to the output's type: half a step. In the backward pass g is
rounded to the type before the products."""
import pytest
import torch

import expert_routing_grouped_layer_b200 as moe
import ops_reference as ref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
TINY = {HF: 2.0 ** -25, BF: 1e-38}  # half of fp16's smallest step


def acc_unit(K):
    return (K / 16 + 16) * 2.0 ** -23


def _mat(g, rows, cols, dt, pad=True, scale=1.0):
    ld = (cols + 7) // 8 * 8 if pad else cols
    return (torch.randn(rows, ld, generator=g, device="cuda") * scale).to(dt)[:, :cols]


def _forward(M, N, K, dt, act="none", bias=True, residual=False, pre=False, seed=0, check=True, out_ld=None):
    g = torch.Generator(device="cuda").manual_seed(seed + M + N + K)
    x, w = _mat(g, M, K, dt), _mat(g, N, K, dt, scale=K ** -0.5)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    r = _mat(g, M, N, dt, pad=out_ld is None) if residual else None
    y = torch.full((M, out_ld or N), 77.0, dtype=dt, device="cuda")
    z = torch.full((M, out_ld or N), 77.0, dtype=dt, device="cuda") if pre else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_linear(x, w, b, r, y[:, :N], z[:, :N] if pre else None, act=act, dev_status=st)
    assert st.item() == 0
    if check:
        zd, yd = ref.linear(x, w, b, r, act)
        mag = x.double().abs() @ w.double().abs().t() + (b.double().abs() if bias else 0)
        err = acc_unit(K) * mag
        if pre:
            assert ((z[:, :N].double() - zd).abs() <= ref.U[dt] * zd.abs() + err * 1.01 + TINY[dt]).all()
        ev = 1.13 * err + 2.0 ** -21 * (1 + zd.abs()) + 2.0 ** -23 * (r.double().abs() if residual else 0)
        bad = (y[:, :N].double() - yd).abs() > ref.U[dt] * yd.abs() + 1.01 * ev + TINY[dt]
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())
        assert (y[:, N:] == 77).all()
    return x, w, b, r, y, z


SIZES = [(1, 1, 1), (1, 128, 64), (1, 2048, 7168), (1, 300, 515), (2, 7168, 2048), (3, 5, 7), (15, 130, 100),
         (16, 384, 7168), (17, 257, 66), (64, 640, 1024), (80, 1000, 72), (96, 2048, 512), (127, 129, 65),
         (128, 7168, 2048), (129, 256, 192), (200, 96, 4097), (256, 4096, 256), (257, 300, 700),
         (512, 2048, 1024), (700, 512, 2048), (1037, 2051, 1111), (2048, 2048, 2048), (5000, 100, 40),
         (4096, 16, 128), (9, 20000, 64), (3000, 1500, 1000), (1111, 7168, 64)]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(M, N, K, dt):
    _forward(M, N, K, dt)


@pytest.mark.parametrize("M,N,K", [(5, 200, 333), (300, 515, 128), (2048, 1024, 512)])
@pytest.mark.parametrize("act", list(moe.ACT))
def test_epilogue(M, N, K, act):
    _forward(M, N, K, BF, act, residual=True, pre=True)
    _forward(M, N, K, HF, act, bias=False, pre=True)
    _forward(M, N, K, BF, act, bias=False, residual=True)


@pytest.mark.parametrize("M,N,out_ld", [(33, 100, 101), (33, 101, 101), (600, 514, 517), (600, 512, 516)])
def test_output_strides(M, N, out_ld):
    """Outputs and residuals whose rows allow no wide accesses; what lies between stays."""
    _forward(M, N, 96, BF, "silu", residual=True, pre=True, out_ld=out_ld)


def test_residual_in_place_and_equal_bits():
    for M, N, K in [(4, 512, 2048), (3000, 1024, 512)]:
        x, w, b, r, y, _ = _forward(M, N, K, BF, "none", residual=True, seed=1)
        h = r.clone()
        moe.moe_linear(x, w, b, h, h)
        assert torch.equal(h, y)
        for _ in range(3):
            again = torch.empty_like(y)
            moe.moe_linear(x, w, b, r, again)
            assert torch.equal(again, y)


def test_values_outside_the_matrices_stay_outside():
    """NaN in the padding of x's and w's rows and behind their last rows reaches nothing;
    NaN and infinities inside reach their own rows and columns."""
    for M, N, K in [(20, 140, 70), (300, 600, 70)]:
        g = torch.Generator(device="cuda").manual_seed(2)
        xa = torch.full((M + 5, 80), float("nan"), dtype=BF, device="cuda")
        wa = torch.full((N + 5, 80), float("nan"), dtype=BF, device="cuda")
        xa[:M, :K] = torch.randn(M, K, generator=g, device="cuda").to(BF)
        wa[:N, :K] = torch.randn(N, K, generator=g, device="cuda").to(BF)
        x, w = xa[:M, :K], wa[:N, :K]
        y = torch.empty(M, N, dtype=BF, device="cuda")
        moe.moe_linear(x, w, None, None, y)
        assert torch.isfinite(y).all()
        x[3, 5] = float("nan")
        w[7, 0] = float("inf")
        for act in ("none", "relu"):
            moe.moe_linear(x, w, None, None, y, act=act)
            assert torch.isnan(y[3]).all()
            keep = torch.ones(M, dtype=torch.bool, device="cuda")
            keep[3] = False
            z = x[keep].double() @ w.double().t()
            want = z[:, 7].clamp(min=0) if act == "relu" else z[:, 7]
            assert torch.equal(y[keep][:, 7].double(), want)
            cols = torch.ones(N, dtype=torch.bool, device="cuda")
            cols[7] = False
            assert torch.isfinite(y[keep][:, cols]).all()


def _backward(M, N, K, dt, act, seed=0, dy_pad=True, want=(True, True, True)):
    g = torch.Generator(device="cuda").manual_seed(seed + M + N + K)
    x, w = _mat(g, M, K, dt), _mat(g, N, K, dt, scale=K ** -0.5)
    dy, pre = _mat(g, M, N, dt, pad=dy_pad), _mat(g, M, N, dt, pad=dy_pad)
    dx = torch.full((M, K), 7.0, dtype=dt, device="cuda") if want[0] else None
    dw = torch.full((N, K), 7.0, dtype=dt, device="cuda") if want[1] else None
    db = torch.full((N,), 7.0, device="cuda") if want[2] else None
    ws = torch.empty(moe.moe_linear_backward_workspace_bytes(M, N, K, act), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = pre if act != "none" else None
    moe.moe_linear_backward(dy, x, w, p, dx, dw, db, ws, act=act, dev_status=st)
    assert st.item() == 0
    gd, rdx, rdw, rdb = ref.linear_backward(dy, x, w, p, act)
    slope = 2.0 ** -21 * dy.double().abs() * (1 + pre.double().abs()) if act != "none" else 0 * gd
    dg = slope + ref.U[dt] * gd.abs() + TINY[dt]
    ga, wa, xa = gd.abs(), w.double().abs(), x.double().abs()
    if want[0]:
        tol = dg @ wa + acc_unit(N) * 1.01 * (ga @ wa) + ref.U[dt] * rdx.abs() * 1.01 + TINY[dt]
        assert ((dx.double() - rdx).abs() <= tol).all()
    if want[1]:
        tol = dg.t() @ xa + acc_unit(M) * 1.01 * (ga.t() @ xa) + ref.U[dt] * rdw.abs() * 1.01 + TINY[dt]
        assert ((dw.double() - rdw).abs() <= tol).all()
    if want[2]:  # at most 64 rows a warp (M <= 32768), 8 warps, 8 x 8 chunks
        assert ((db.double() - rdb).abs() <= slope.sum(0) + 96 * 2.0 ** -24 * ga.sum(0)).all()
    return x, w, dy, pre, dx, dw, db


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 200, 300), (3, 5, 7), (16, 128, 128), (33, 100, 515),
                                   (65, 64, 7168), (128, 2048, 512), (200, 1000, 129), (300, 515, 700),
                                   (1037, 300, 411), (5000, 100, 40), (777, 2048, 1024), (2048, 2048, 2048),
                                   (4100, 64, 64)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_backward(M, N, K, dt):
    _backward(M, N, K, dt, "silu")
    _backward(M, N, K, dt, "none", seed=1)


@pytest.mark.parametrize("act", list(moe.ACT))
def test_backward_activations_and_strides(act):
    _backward(100, 101, 96, BF, act, dy_pad=False)
    _backward(515, 264, 130, HF, act)
    for want in ((True, False, False), (False, True, False), (False, False, True)):
        _backward(70, 90, 50, BF, act, want=want)


def test_gradients_against_differences():
    """The forward's own formula, evaluated either side of a value."""
    for act in moe.ACT:
        x, w, dy, pre, dx, dw, db = _backward(4, 6, 8, BF, act, seed=3)
        b = pre.double() - x.double() @ w.double().t()  # a bias per element that gives this pre
        f = lambda x_, w_: (ref.act(x_ @ w_.t() + b, act) * dy.double()).sum().item()
        h = 1e-6
        for t, i, j in [(0, 1, 2), (3, 5, 7)]:
            d = torch.zeros(4, 8, dtype=torch.float64, device="cuda")
            d[t, j] = h
            num = (f(x.double() + d, w.double()) - f(x.double() - d, w.double())) / (2 * h)
            # bf16: g and the result are rounded, 2^-8 of the terms each
            terms = (dy[t].double().abs() * w[:, j].double().abs()).sum().item()
            assert abs(num - dx[t, j].item()) <= 2.5 * 2.0 ** -8 * terms + 1e-4
            e = torch.zeros(6, 8, dtype=torch.float64, device="cuda")
            e[i, j] = h
            num = (f(x.double(), w.double() + e) - f(x.double(), w.double() - e)) / (2 * h)
            terms = (dy[:, i].double().abs() * x[:, j].double().abs()).sum().item()
            assert abs(num - dw[i, j].item()) <= 2.5 * 2.0 ** -8 * terms + 1e-4


def test_no_rows():
    w = torch.ones(6, 16, dtype=BF, device="cuda")
    x = torch.empty(0, 16, dtype=BF, device="cuda")
    y = torch.empty(0, 6, dtype=BF, device="cuda")
    moe.moe_linear(x, w, None, None, y)
    wide = torch.full((6, 20), 3.0, dtype=BF, device="cuda")
    db = torch.ones(6, device="cuda")
    moe.moe_linear_backward(y, x, w, None, x, wide[:, :16], db, None)
    assert (wide[:, :16] == 0).all() and (wide[:, 16:] == 3).all() and (db == 0).all()


def test_two_streams_and_graphs():
    """The same layer on two streams at once, and captured graphs replayed on new inputs."""
    M, N, K = 96, 1024, 2048
    runs = []
    for seed in (5, 6):
        s = torch.cuda.Stream()
        x, w, b, r, y, z = _forward(M, N, K, BF, "gelu", residual=True, pre=True, seed=seed)
        dy = torch.randn(M, N, device="cuda").to(BF)
        out = [torch.empty_like(y), torch.empty_like(z), torch.empty_like(x), torch.empty_like(w),
               torch.empty(N, device="cuda")]
        ws = torch.empty(moe.moe_linear_backward_workspace_bytes(M, N, K, "gelu"), dtype=torch.uint8,
                         device="cuda")

        def step(stream=None, x=x, w=w, b=b, r=r, out=out, dy=dy, ws=ws):
            moe.moe_linear(x, w, b, r, out[0], out[1], act="gelu", stream=stream)
            moe.moe_linear_backward(dy, x, w, out[1], out[2], out[3], out[4], ws, act="gelu", stream=stream)
        step()
        torch.cuda.synchronize()
        runs.append((s, step, out, [o.clone() for o in out], x))
    for _ in range(20):
        for s, step, *_ in runs:
            step(s)
    torch.cuda.synchronize()
    for s, step, out, want, x in runs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    graphs = []
    for s, step, out, want, x in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        x.neg_()
        graphs.append(g)
    torch.cuda.synchronize()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for s, step, out, want, x in runs:
        got = [o.clone() for o in out]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, out))


def _tail(z, act):
    """The activation in double precision without differences of close numbers."""
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    return ref.act(z, act)


def _tail_case(act, dt, lo, hi, rel, n=4000):
    """act and its slope on n values of z in [lo, hi], each off by `rel` of itself and the rounding."""
    z = torch.linspace(lo, hi, n, dtype=torch.float64, device="cuda").to(dt)
    want = _tail(z.double(), act)
    one = torch.ones(1, 8, dtype=dt, device="cuda")  # rows of 16 bytes; the product has one term
    x = torch.zeros(n, 8, dtype=dt, device="cuda")
    x[:, 0] = z
    for cols in (1, 128):  # a split and a pair kernel's tile
        w = torch.zeros(cols, 8, dtype=dt, device="cuda")
        w[:, 0] = 1
        y = torch.empty(n, cols, dtype=dt, device="cuda")
        moe.moe_linear(x[:, :1], w[:, :1], None, None, y, act=act)
        off = (y.double() - want[:, None]).abs()
        assert (off <= (ref.U[dt] + rel) * want.abs()[:, None] + TINY[dt]).all()
    # one row of n columns: db is the slope in fp32
    zd = z.double().requires_grad_(True)
    slope = torch.autograd.grad(_tail(zd, act).sum(), zd)[0]
    for cols in (n, n - 1):  # wide and element accesses
        db = torch.empty(cols, device="cuda")
        ws = torch.empty(moe.moe_linear_backward_workspace_bytes(1, cols, 1, act), dtype=torch.uint8, device="cuda")
        dy = torch.ones(1, cols, dtype=dt, device="cuda")
        w = torch.zeros(cols, 8, dtype=dt, device="cuda")
        moe.moe_linear_backward(dy, one[:, :1], w[:, :1], z[None, :cols], None, None, db, ws, act=act)
        assert ((db.double() - slope[:cols]).abs() <= rel * slope[:cols].abs() + 1e-38).all()


@pytest.mark.parametrize("dt", [BF, HF])
def test_gelu_tanh_far_below_zero(dt):
    """Relative to the value, which is down to 1e-26 here. The exponential's argument is at most 70
    and off by four roundings and the instruction's 2^-23 of it, 70 * 6 * 2^-24 = 2.5e-5 relative;
    the slope's factor of it, z (1 - s) u' ~ 30, multiplies no error of s: 2^-14 holds both."""
    _tail_case("gelu_tanh", dt, -9.0, -3.0, 2.0 ** -14)


@pytest.mark.parametrize("dt", [BF, HF])
def test_gelu_far_below_zero(dt):
    """Relative to the value, which is down to 1e-36 here. exp(-z^2 / 2) has an argument of at most 82,
    off by two roundings and the instruction's 2^-23 of it: 82 * 4 * 2^-24 = 2.0e-5 relative; the fit
    5e-7; the slope is -z^2 times that and more: 2^-14 holds both."""
    _tail_case("gelu", dt, -12.8, -3.0, 2.0 ** -14)


def test_gelu_near_zero():
    """The slope in fp32 where it is of order one: fit 2e-7 and a dozen roundings of terms below 1.2."""
    z = torch.linspace(-3, 3, 4096, dtype=torch.float64, device="cuda").to(HF)
    zd = z.double().requires_grad_(True)
    for act in ("gelu", "gelu_tanh", "silu"):
        slope = torch.autograd.grad(_tail(zd, act).sum(), zd)[0]
        db = torch.empty(4096, device="cuda")
        ws = torch.empty(moe.moe_linear_backward_workspace_bytes(1, 4096, 1, act), dtype=torch.uint8, device="cuda")
        one = torch.ones(1, 1, dtype=HF, device="cuda")
        moe.moe_linear_backward(torch.ones(1, 4096, dtype=HF, device="cuda"), one, torch.empty(4096, 8, dtype=HF,
                                device="cuda")[:, :1], z[None], None, None, db, ws, act=act)
        assert ((db.double() - slope).abs() <= 2.0 ** -20).all()


@pytest.mark.parametrize("act,lo", [("silu", -95.0), ("gelu_tanh", -10.3)])
def test_sigmoid_forms_to_the_end_of_the_range(act, lo):
    """Down to where the value itself leaves the fp32 range (1e-38, which the tolerance allows): the
    argument, at most 98, is off by five units of 2^-24 of it, 2.9e-5 relative."""
    _tail_case(act, BF, lo, -3.0, 2.0 ** -14)


@pytest.mark.parametrize("act", [a for a in moe.ACT if a != "none"])
@pytest.mark.parametrize("dt", [BF, HF])
def test_gradient_at_infinite_and_huge_pre(act, dt):
    """z beyond the f16 range is kept as an infinite pre; its slope is still 0 or 1."""
    big = [1e20, 3e38] if dt == BF else [5e4, 65504.0]
    pre = torch.tensor([[float("inf"), *big, 300.0, -float("inf"), *(-b for b in big), -300.0, float("nan")]],
                       device="cuda").to(dt)
    N = pre.shape[1]
    db, g = torch.empty(N, device="cuda"), torch.empty(N, 1, dtype=dt, device="cuda")
    ws = torch.empty(moe.moe_linear_backward_workspace_bytes(1, N, 1, act), dtype=torch.uint8, device="cuda")
    dy = torch.full((1, N), 2.0, dtype=dt, device="cuda")
    one, w = torch.ones(1, 1, dtype=dt, device="cuda"), torch.ones(N, 8, dtype=dt, device="cuda")[:, :1]
    moe.moe_linear_backward(dy, one, w, pre, None, g, db, ws, act=act)
    want = torch.tensor([2.0] * 4 + [0.0] * 4, device="cuda")
    assert torch.equal(db[:8], want) and torch.isnan(db[8])
    assert torch.equal(g[:8, 0].float(), want) and torch.isnan(g[8, 0])


def _between(rows, cols, extra, dt):
    """A matrix inside a wider one of sevens, rows a multiple of 16 bytes apart; the wider one."""
    wide = torch.full((rows, (cols + 7) // 8 * 8 + extra), 7.0, dtype=dt, device="cuda")
    return wide[:, :cols], wide


@pytest.mark.parametrize("extra", [0, 8, 40])
@pytest.mark.parametrize("M,N,K", [(4, 23, 5), (17, 2791, 79), (149, 15, 4), (666, 7, 155), (3000, 1500, 64),
                                   (2500, 1503, 65), (2500, 1505, 130), (1037, 2051, 1111), (300, 4097, 33)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_what_lies_behind_ragged_rows_stays(M, N, K, extra, dt):
    """Outputs whose rows start on 16-byte boundaries and end inside one: y, pre, dx and dw leave the
    elements behind their rows as they are, and are right up to the last one."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x, w = _mat(g, M, K, dt), _mat(g, N, K, dt, scale=K ** -0.5)
    b = torch.randn(N, generator=g, device="cuda")
    for res in (None, _mat(g, M, N, dt), "y"):
        for with_pre in (False, True):
            (y, wide), (z, zwide) = _between(M, N, extra, dt), _between(M, N, extra, dt)
            r = res
            if res == "y":  # in place
                y.copy_(_mat(g, M, N, dt))
                r = y.clone()
            moe.moe_linear(x, w, b, y if res == "y" else res, y, z if with_pre else None, act="silu")
            zd, yd = ref.linear(x, w, b, r, "silu")
            err = acc_unit(K) * (x.double().abs() @ w.double().abs().t() + b.double().abs())
            ev = 1.13 * err + 2.0 ** -21 * (1 + zd.abs()) + 2.0 ** -23 * (r.double().abs() if r is not None else 0)
            assert ((y.double() - yd).abs() <= ref.U[dt] * yd.abs() + 1.01 * ev + TINY[dt]).all()
            assert (wide[:, N:] == 7).all()
            if with_pre:
                assert ((z.double() - zd).abs() <= ref.U[dt] * zd.abs() + err * 1.01 + TINY[dt]).all()
            assert (zwide[:, N:] == 7).all()
    dy = _mat(g, M, N, dt)
    (dx, xwide), (dw, wwide) = _between(M, K, extra, dt), _between(N, K, extra, dt)
    ws = torch.empty(moe.moe_linear_backward_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    moe.moe_linear_backward(dy, x, w, None, dx, dw, None, ws)
    assert (xwide[:, K:] == 7).all() and (wwide[:, K:] == 7).all()
    gd, rdx, rdw, _ = ref.linear_backward(dy, x, w, None, "none")
    tol = acc_unit(N) * 1.01 * (gd.abs() @ w.double().abs()) + ref.U[dt] * rdx.abs() * 1.01 + TINY[dt]
    assert ((dx.double() - rdx).abs() <= tol).all()
    tol = acc_unit(M) * 1.01 * (gd.abs().t() @ x.double().abs()) + ref.U[dt] * rdw.abs() * 1.01 + TINY[dt]
    assert ((dw.double() - rdw).abs() <= tol).all()
