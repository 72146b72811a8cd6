"""moe_norm and moe_norm_backward against the 64-bit formulas.

Tolerances. An output rounded once to its type is off by half a step of its value. The
fp32 arithmetic before it: sums of H terms by at most 16 per thread and trees of 10
levels, and a handful of operations per element, together below 64 units of 2^-24 of the
terms' magnitudes (for a centred element those of x and the mean). Column sums add up to
T / grid rows one after the other; T is chosen so that this stays below 64 as well."""
import pytest
import torch

import expert_routing_grouped_layer_b200 as moe
import ops_reference as ref

pytestmark = pytest.mark.gpu
E32 = 64 * 2.0 ** -24
# below 2^-14 fp16's steps stay at 2^-24, so half a step there is 2^-25, not 2^-11 of the value
# (a 16383-wide row holds values of 1e-5); bf16 and fp32 have fp32's range
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38, torch.float32: 1e-38}


def _case(T, H, dt, seed, ld=None, scale=1.0, off=0.0, w=True, b=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = torch.randn(T, ld or H, generator=g, device="cuda") * scale + off
    x = full.to(dt)[:, :H]
    dy = torch.randn(T, ld or H, generator=g, device="cuda").to(dt)[:, :H]
    return (x, dy, 1 + 0.3 * torch.randn(H, generator=g, device="cuda") if w else None,
            0.2 * torch.randn(H, generator=g, device="cuda") if b else None)


def _check(x, dy, w, b, eps, kind):
    T, H = x.shape
    dt = x.dtype
    y, dx = torch.full_like(x, 7), torch.full_like(x, 7)
    mean = torch.full((T,), 7.0, device="cuda") if kind == "layer" else None
    rstd = torch.full((T,), 7.0, device="cuda")
    moe.moe_norm(x, w, b, eps, y, mean, rstd, kind=kind)
    want, m, r = ref.norm(x, w, b, eps, kind)
    aw = torch.ones(H, device="cuda") if w is None else w.abs()
    ab = torch.zeros(H, device="cuda") if b is None else b.abs()
    size = (x.double().abs() + m.abs()[:, None]) * r[:, None]
    assert ((y.double() - want).abs() <= ref.U[dt] * want.abs() + E32 * (size * aw + ab) + TINY[dt]).all()
    assert ((rstd.double() - r).abs() <= E32 * r * (1 + (m * r) ** 2)).all()
    if kind == "layer":
        assert ((mean.double() - m).abs() <= E32 * x.double().abs().mean(1)).all()

    dw, db = torch.full((H,), 7.0, device="cuda"), torch.full((H,), 7.0, device="cuda")
    ws = torch.empty(moe.moe_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    moe.moe_norm_backward(dy, x, w, mean, rstd, dx, dw, db if kind == "layer" else None, ws, kind=kind)
    wdx, wdw, wdb = ref.norm_backward(dy, x, w, mean, rstd, kind)
    mm = mean.double().abs()[:, None] if kind == "layer" else 0.0
    n = (x.double().abs() + mm) * rstd.double()[:, None]
    g = dy.double().abs() * aw
    terms = rstd.double()[:, None] * (g + g.mean(1, keepdim=True) + n * (g * n).mean(1, keepdim=True))
    assert ((dx.double() - wdx).abs() <= ref.U[dt] * wdx.abs() + E32 * terms + TINY[dt]).all()
    assert ((dw.double() - wdw).abs() <= E32 * (dy.double().abs() * n).sum(0)).all()
    if kind == "layer":
        assert ((db.double() - wdb).abs() <= E32 * dy.double().abs().sum(0)).all()
    # equal calls give equal bits
    dw2, dx2 = torch.empty_like(dw), torch.empty_like(dx)
    moe.moe_norm_backward(dy, x, w, mean, rstd, dx2, dw2, None, ws, kind=kind)
    assert torch.equal(dw, dw2) and torch.equal(dx, dx2)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 2), (5, 7), (2, 8), (33, 31), (700, 64), (64, 1000),
                                 (40, 4095), (9, 4097), (300, 7168), (12, 8200), (17, 16384), (6, 16383)])
def test_sizes(kind, dt, T, H):
    _check(*_case(T, H, dt, T + H), 1e-6, kind)


# Rows of one warp (up to 512 elements): whole and partial vectors of a lane, rows one by one and in
# pairs, warps without a row, and partial sums that need many rounds of the second kernel.
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 512), (9, 64), (37, 512), (591, 256), (593, 504), (1500, 512), (4737, 8),
                                 (20003, 64), (20003, 63)])
def test_short_rows(kind, dt, T, H):
    _check(*_case(T, H, dt, T + H), 1e-6, kind)


@pytest.mark.parametrize("T,H", [(37, 512), (1501, 256)])
def test_short_rows_in_place(T, H):
    x, dy, w, b = _case(T, H, torch.bfloat16, 3)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_norm(x, w, b, 1e-6, torch.empty_like(x), mean, rstd)
    ws = torch.empty(moe.moe_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    want = torch.empty_like(x)
    moe.moe_norm_backward(dy, x, w, mean, rstd, want, dw, db, ws)
    for into_dy in (False, True):
        a, g = x.clone(), dy.clone()
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        moe.moe_norm_backward(g, a, w, mean, rstd, g if into_dy else a, dw2, db2, ws)
        assert torch.equal(g if into_dy else a, want) and torch.equal(dw, dw2) and torch.equal(db, db2)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_many_rows(dt):
    _check(*_case(4000, 1024, dt, 1), 1e-5, "layer")


@pytest.mark.parametrize("ld,off", [(136, 0), (129, 0), (136, 1), (136, 8)])
def test_strides_and_offsets(ld, off):
    """Rows inside wider rows, 16-byte aligned or not; what lies between the rows stays."""
    x, dy, w, b = _case(50, 120, torch.bfloat16, 5, ld=ld)
    wide = torch.zeros(50, 2 * ld, dtype=torch.bfloat16, device="cuda")
    xs = wide[:, off:off + 120]
    xs.copy_(x)
    _check(xs, dy, w, b, 1e-6, "layer")
    assert (wide[:, off + 120:] == 0).all() and (wide[:, :off] == 0).all()
    y = torch.full((50, ld), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_norm(xs, w, b, 1e-6, y[:, :120])
    assert (y[:, 120:] == 3).all() and not (y[:, :120] == 3).all()


@pytest.mark.parametrize("w,b", [(False, True), (True, False), (False, False)])
def test_without_weight_or_bias(w, b):
    _check(*_case(30, 512, torch.bfloat16, 6, w=w, b=b), 1e-6, "layer")


def test_values():
    """Rows far off centre, tiny, constant and zero."""
    x, dy, w, b = _case(64, 640, torch.float32, 7)
    x[0:8] = x[0:8] + 1000.0
    x[8:16] *= 1e-18
    x[16] = 3.0
    x[17] = 0.0
    _check(x, dy, w, b, 1e-6, "layer")
    _check(x, dy, w, None, 1e-6, "rms")
    y = torch.empty_like(x)
    moe.moe_norm(x, w, b, 1e-6, y)
    assert torch.allclose(y[16], b, atol=1e-6) and torch.equal(y[17], b)
    x[3, 5] = float("nan")
    moe.moe_norm(x, w, b, 1e-6, y)
    assert torch.isnan(y[3]).all() and torch.isfinite(y[4]).all()


def test_in_place_and_partial_outputs():
    x, dy, w, b = _case(300, 7168, torch.bfloat16, 8)
    T, H = x.shape
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_norm(x, w, b, 1e-6, y, mean, rstd)
    z = x.clone()
    moe.moe_norm(z, w, b, 1e-6, z)
    assert torch.equal(z, y)
    ws = torch.empty(moe.moe_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
    only = torch.empty_like(x)
    moe.moe_norm_backward(dy, x, w, mean, rstd, only, None, None, None)
    assert torch.equal(only, dx)
    for which in (0, 1):
        got = [None, None]
        got[which] = torch.empty(H, device="cuda")
        moe.moe_norm_backward(dy, x, w, mean, rstd, None, got[0], got[1], ws)
        assert torch.equal(got[which], (dw, db)[which])
    gx = dy.clone()
    moe.moe_norm_backward(gx, x, w, mean, rstd, gx, None, None, None)
    assert torch.equal(gx, dx)
    none = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_norm(none, w, b, 1e-6, none)
    moe.moe_norm_backward(none, none, w, mean[:0], rstd[:0], none, dw, db, None)
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("T,H", [(400, 1023), (30, 515), (64, 4097)])
def test_in_place_off_the_16_byte_grid(T, H):
    x, dy, w, b = _case(T, H, torch.bfloat16, 9)
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_norm(x, w, b, 1e-6, y, mean, rstd)
    dx = torch.empty_like(x)
    moe.moe_norm_backward(dy, x, w, mean, rstd, dx, None, None, None)
    for _ in range(5):
        z = x.clone()
        moe.moe_norm(z, w, b, 1e-6, z)
        assert torch.equal(z, y)
        for keep in (dy, x):
            g = keep.clone()
            moe.moe_norm_backward(g if keep is dy else dy, g if keep is x else x, w, mean, rstd, g, None, None, None)
            assert torch.equal(g, dx)


def test_rows_between_other_data():
    """NaN before, between and behind the rows reaches nothing, on and off the 16-byte grid."""
    for off, H, ld in [(0, 120, 128), (1, 120, 131), (3, 119, 129)]:
        T = 700
        g = torch.Generator(device="cuda").manual_seed(H)
        flat = torch.full((T * ld + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
        x = flat[off:off + T * ld].view(T, ld)[:, :H]
        x.copy_(torch.randn(T, H, generator=g, device="cuda"))
        _check(x, x.clone(), None, None, 1e-6, "layer")
        y = torch.full_like(flat, 5.0)
        moe.moe_norm(x, None, None, 1e-6, y[off:off + T * ld].view(T, ld)[:, :H])
        mask = torch.ones_like(flat, dtype=torch.bool)
        mask[off:off + T * ld].view(T, ld)[:, :H] = False
        assert (y[mask] == 5).all() and torch.isfinite(y).all()


def test_gradient_against_differences():
    x, _, w, b = _case(4, 96, torch.float32, 9)
    T, H = x.shape
    c = torch.randn(T, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_norm(x, w, b, 1e-6, y, mean, rstd)
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = torch.empty(moe.moe_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    moe.moe_norm_backward(c, x, w, mean, rstd, dx, dw, None, ws)
    f = lambda x_, w_: (ref.norm(x_, w_, b, 1e-6, "layer")[0] * c).sum().item()
    h = 1e-4
    for t, e in [(0, 0), (2, 95), (3, 40)]:
        d = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        d[t, e] = h
        # central differences: off by h^2 times the third derivative (order 1) and 1e-16 / h
        assert abs((f(x.double() + d, w) - f(x.double() - d, w)) / (2 * h) - dx[t, e].item()) < 1e-5
        dd = d[t]
        assert abs((f(x, w.double() + dd) - f(x, w.double() - dd)) / (2 * h) - dw[e].item()) < 1e-4


def test_two_captured_graphs_on_another_stream():
    """A forward and a backward captured on a side stream, with a workspace each, and
    replayed on new inputs."""
    s = torch.cuda.Stream()

    def capture(seed):
        x, dy, w, b = _case(128, 1024, torch.bfloat16, seed)
        out = [torch.empty_like(x), torch.empty(128, device="cuda"), torch.empty(128, device="cuda"),
               torch.empty_like(x), torch.empty(1024, device="cuda"), torch.empty(1024, device="cuda")]
        ws = torch.empty(moe.moe_norm_backward_workspace_bytes(128, 1024), dtype=torch.uint8, device="cuda")

        def step():
            moe.moe_norm(x, w, b, 1e-6, out[0], out[1], out[2])
            moe.moe_norm_backward(dy, x, w, out[1], out[2], out[3], out[4], out[5], ws)
        step()
        g = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            step()
        return g, x, out, step

    with torch.cuda.stream(s):
        graphs = [capture(1), capture(2)]
        for g, x, out, step in graphs:
            x.mul_(0.5).add_(0.25)
        for g, *_ in graphs:
            g.replay()
        s.synchronize()
        for g, x, out, step in graphs:
            got = [o.clone() for o in out]
            for o in out:
                o.zero_()
            step()
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, out))


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [1024, 1023])
def test_large_rows_have_one_outcome(H, dt, kind):
    """Rows whose squares add up to more than fp32 holds get rstd 0 and y = b, those just below it are
    right, whichever kernel the batch size and the alignment choose."""
    g = torch.Generator(device="cuda").manual_seed(H)
    w, b = 1 + 0.3 * torch.randn(H, generator=g, device="cuda"), 0.2 * torch.randn(H, generator=g, device="cuda")
    rows = torch.randn(3, H, generator=g, device="cuda")
    rows = (rows / rows.abs().max() * torch.tensor([[1e20], [4e17], [1e18]], device="cuda")).to(dt)
    for T in (3, 64, 700):
        x = torch.randn(T, H, generator=g, device="cuda").to(dt)
        x[:3] = rows
        y, mean, rstd = torch.empty_like(x), torch.zeros(T, device="cuda"), torch.empty(T, device="cuda")
        moe.moe_norm(x, w, b, 1e-6, y, mean if kind == "layer" else None, rstd, kind=kind)
        assert rstd[0] == 0 and torch.equal(y[0], b.to(dt)) and torch.isfinite(y).all()
        _, m, r = ref.norm(x[1:3], w, b, 1e-6, kind)
        assert ((rstd[1:3].double() - r).abs() <= E32 * r * (1 + (m * r) ** 2)).all()
        dx, dw, db = torch.empty_like(x), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
        ws = torch.empty(moe.moe_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
        moe.moe_norm_backward(torch.ones_like(x), x, w, mean if kind == "layer" else None, rstd, dx, dw, db, ws,
                              kind=kind)
        assert (dx[0] == 0).all() and torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("H,ld", [(1, 1), (1, 2), (2, 2), (3, 3), (3, 5), (5, 7), (7, 7), (7, 9)])
def test_rows_of_few_bytes_between_other_data(H, ld):
    """NaN in front of, between and behind rows of fewer than 16 bytes reaches nothing."""
    for T in (1, 2, 3, 9, 700):
        for off in (0, 1, 3, 7):
            flat = torch.full((T * ld + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
            x = flat[off:off + T * ld].view(T, ld)[:, :H]
            x.copy_(torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda"))
            before = flat.clone()
            _check(x, x.clone(), None, None, 1e-6, "rms")
            assert torch.equal(flat.view(torch.int16), before.view(torch.int16))
