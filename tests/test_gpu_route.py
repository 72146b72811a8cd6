"""moe_route, moe_route_backward and moe_combine_backward against 64-bit references.

The chosen experts have to be those of the double-precision order exactly. Weights: at
most 70 additions in fp32 and a few operations before and after, below 1e-5 relative.
Gradients: the same relative to the sum of their terms' magnitudes, plus half a step of
the output's type."""
import math

import pytest
import torch

import expert_routing_grouped_layer_b200 as moe
import ops_reference as ref
from expert_routing_grouped_layer_b200 import workloads as W

pytestmark = pytest.mark.gpu
BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
REL = 1e-5


def _cfg(E, k, groups=1, kept=1, score="sigmoid", renorm=True, hidden=128):
    return W.CONFIGS["tiny_bf16"].replace(hidden=hidden, n_routed_experts=E, num_experts_per_tok=k,
                                          n_group=groups, topk_group=kept, score_fn=score,
                                          norm_topk_prob=renorm, routed_scaling_factor=2.5)


def _route(cfg, logits, bias):
    T, k = logits.shape[0], cfg.num_experts_per_tok
    idx = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 77.0, device="cuda")
    moe.moe_route(cfg, logits, bias, idx, w)
    return idx, w


def _check(cfg, logits, bias):
    idx, w = _route(cfg, logits, bias)
    ri, rw = ref.route(cfg, logits, bias)
    assert torch.equal(idx.cpu(), ri)
    gw = w.double().cpu()
    assert torch.equal(torch.isnan(gw), torch.isnan(rw))
    ok = ~torch.isnan(rw)
    # 1e-38: products below the normal range
    assert ((gw - rw)[ok].abs() <= REL * rw[ok].abs() + 1e-38).all()
    return idx


def _logits(T, E, dt, seed, scale=1.7):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, E, generator=g, device="cuda") * scale).to(dt), \
        0.2 * torch.rand(E, generator=g, device="cuda") - 0.1


SHAPES = [(1, 1, 1, 1), (2, 1, 1, 1), (16, 4, 1, 1), (33, 32, 1, 1), (60, 6, 5, 3), (72, 8, 9, 4),
          (128, 8, 1, 1), (256, 8, 8, 4), (384, 8, 8, 4), (384, 8, 1, 1), (320, 32, 32, 32),
          (510, 3, 17, 2), (640, 6, 1, 1), (896, 16, 1, 1), (896, 16, 16, 5), (1000, 7, 1, 1),
          (1020, 9, 17, 9), (1008, 5, 24, 3), (1024, 32, 1, 1), (1024, 2, 32, 1), (904, 4, 8, 8)]


@pytest.mark.parametrize("score", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("E,k,groups,kept", SHAPES)
def test_shapes(E, k, groups, kept, score):
    """Every layout of experts over lanes, biased and not, all three types."""
    for i, dt in enumerate((FL, BF, HF)):
        l, bias = _logits(60, E, dt, E + k + i)
        _check(_cfg(E, k, groups, kept, score, renorm=i != 1), l, bias)
        _check(_cfg(E, k, groups, kept, score), l, None)


@pytest.mark.parametrize("T", [1, 2, 7, 2400])
def test_batch_sizes(T):
    l, bias = _logits(T, 64, FL, T)
    _check(_cfg(64, 6, 4, 2), l, bias)


@pytest.mark.parametrize("score", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
def test_near_ties(score, groups, kept):
    """Scores that fp32 cannot tell apart: a few distinct logits and biases one to three
    units of the last place from each other, exact ties among them."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, E = 300, 128
    base = torch.randint(0, 6, (T, E), generator=g, device="cuda").float() * 0.37 - 1.0
    l = base * (1 + 2.0 ** -23 * torch.randint(0, 3, (T, E), generator=g, device="cuda"))
    bias = 0.01 + 2.0 ** -30 * torch.randint(0, 4, (E,), generator=g, device="cuda")
    for b in (bias, torch.zeros(E, device="cuda"), None):
        _check(_cfg(E, 8, groups, kept, score), l, b)
    # all scores within the bound of one another
    one = 0.3 + 2.0 ** -25 * torch.randint(0, 50, (20, E), generator=g, device="cuda").float()
    _check(_cfg(E, 8, groups, kept, score), one, bias)
    _check(_cfg(E, 8, groups, kept, score), torch.zeros(9, E, device="cuda"), torch.zeros(E, device="cuda"))


def test_a_left_out_expert_that_fp32_would_rank_behind():
    """Two equal experts at the last place and a third a little better than both in
    double precision, at every position."""
    E, k = 64, 2
    cfg = _cfg(E, k)
    for at in (0, 20, 63):
        l = torch.full((1, E), -3.0, device="cuda")
        l[0, 5], l[0, 30], l[0, 40] = 1.0, 0.5, 0.5
        b = torch.zeros(E, device="cuda")
        l[0, at], b[at] = 0.25, float(1 / (1 + math.exp(-0.5)) - 1 / (1 + math.exp(-0.25)))
        for step in (-2.0 ** -27, 2.0 ** -27, 0.0):
            b2 = b.clone()
            b2[at] += step
            _check(cfg, l, b2)


@pytest.mark.parametrize("E", [64, 256, 1024])
def test_near_ties_inside_kept_groups(E):
    """Two of four groups are clearly the best, with more nearly equal scores than lanes; the
    others hold the best single expert, which no tie may bring back."""
    l = torch.full((12, 4, E // 4), -5.0, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(E)
    l[:, 0::2] = 1.0 + 2.0 ** -23 * torch.randint(0, 9, (12, 2, E // 4), generator=g, device="cuda")
    l[:, 1::2, 3] = 2.0
    l[6:, 0, 5:] = -5.0  # and fewer near ties than lanes
    l[6:, 2, 5:] = -4.0
    bias = 0.01 + 2.0 ** -30 * torch.randint(0, 4, (E,), generator=g, device="cuda")
    for score in ("sigmoid", "sqrtsoftplus"):
        idx = _check(_cfg(E, 8, 4, 2, score), l.view(12, E), bias)
        assert (idx // (E // 4) % 2 == 0).all()
        _check(_cfg(E, 8, 4, 2, score), l.view(12, E), None)


def test_equal_logits():
    """An untrained router: all logits equal, with and without a bias of zeros."""
    for E, k, groups, kept in [(16, 4, 1, 1), (384, 8, 1, 1), (384, 8, 8, 4), (1024, 32, 16, 1)]:
        for dt in (FL, BF):
            l = torch.full((9, E), 0.25, dtype=dt, device="cuda")
            for b in (None, torch.zeros(E, device="cuda")):
                _check(_cfg(E, k, groups, kept), l, b)


@pytest.mark.parametrize("groups,kept,E,k", [(16, 1, 1024, 30), (8, 1, 512, 8), (2, 1, 600, 32), (32, 2, 1024, 17)])
def test_few_lanes_hold_all_candidates(groups, kept, E, k):
    l, bias = _logits(40, E, FL, E + groups)
    _check(_cfg(E, k, groups, kept), l, bias)
    _check(_cfg(E, k, groups, kept, "softmax"), l, None)


@pytest.mark.parametrize("score", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 2)])
def test_masks(score, groups, kept):
    """Masked experts, whole groups, rows with fewer than k experts, empty rows; NaN and
    +inf rows; a masked expert by its bias."""
    T, E, k = 64, 64, 8
    l, bias = _logits(T, E, FL, 4)
    l[0] = -math.inf
    l[1, 3:] = -math.inf
    l[2, :-1] = -math.inf
    l[3, ::2] = -math.inf
    l[4, 8:56] = -math.inf
    l[5, 7] = math.nan
    l[6, 9] = math.inf
    l[7] = torch.finfo(FL).min
    l[8, 1:] = torch.finfo(FL).min
    l[9] = math.inf
    l[10] = math.nan
    idx = _check(_cfg(E, k, groups, kept, score), l, bias)
    assert (idx[[0, 5, 6, 9, 10]] == -1).all() and (idx[1, 3:] == -1).all() and idx[2, 0] == 63
    _check(_cfg(E, k, groups, kept, score, renorm=False), l, None)
    bias[10:20] = -math.inf
    _check(_cfg(E, k, groups, kept, score), l, bias)
    bias[0] = math.nan
    idx, w = _route(_cfg(E, k, groups, kept, score), l, bias)
    assert (idx == -1).all() and torch.isnan(w).all()


@pytest.mark.parametrize("score", ["sigmoid", "sqrtsoftplus", "softmax"])
def test_scores_below_the_fp32_range(score):
    """Renormalised weights of logits far below zero keep their proportions; saturated
    scores are ordered by their logits."""
    l = torch.full((3, 32), -300.0, device="cuda")
    l[0, :4] = torch.tensor([-200.0, -201.0, -199.5, -250.0])
    l[1, :4] = torch.tensor([60.0, 70.0, 65.0, 80.0])
    l[2, :4] = torch.tensor([-100.0, -100.5, -104.0, -110.0])
    for b in (None, torch.zeros(32, device="cuda")):
        _check(_cfg(32, 4, score=score), l, b)
    big = torch.zeros(32, device="cuda")
    big[20:] = 5.0  # the bias chooses experts whose softmax share is nothing
    l[1, 20:] = -150.0 - torch.arange(12, device="cuda")
    _check(_cfg(32, 4, score=score), l, big)


def test_strides():
    l, bias = _logits(40, 100, BF, 8)
    wide = torch.full((40, 219), 9.0, dtype=BF, device="cuda")
    wide[:, 5:105] = l
    cfg = _cfg(100, 6)
    a = _route(cfg, l, bias)
    b = _route(cfg, wide[:, 5:105], bias)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dw = torch.randn(40, 6, device="cuda")
    d1 = torch.empty_like(l)
    moe.moe_route_backward(cfg, l, a[0], dw, d1)
    out = torch.full((40, 131), 5.0, dtype=BF, device="cuda")
    moe.moe_route_backward(cfg, wide[:, 5:105], a[0], dw, out[:, 3:103])
    assert torch.equal(out[:, 3:103], d1)
    assert (out[:, :3] == 5).all() and (out[:, 103:] == 5).all()


def _check_backward(cfg, logits, idx, dw):
    T, E = logits.shape
    dl = torch.full_like(logits, 9)
    moe.moe_route_backward(cfg, logits, idx, dw, dl)
    x = logits.double().requires_grad_(True)
    valid = (idx >= 0) & (idx < E)
    w = ref.route_weights(cfg, x, idx)
    up = torch.where(valid, dw, 0.0).double()
    want = torch.autograd.grad((w * up).sum(), x)[0] if valid.any() else torch.zeros_like(x)
    want = torch.where(valid.any(1, keepdim=True), want, 0.0).detach()
    # terms of one element: its own weight times (its gradient and the row's mean of them)
    p = ref.scores(logits.double(), cfg.score_fn)
    at = torch.where(valid, idx, 0).long()
    aw = torch.where(valid, w.detach().abs(), 0.0)
    own = torch.zeros_like(want).scatter_add_(1, at, aw * up.abs())
    share = torch.zeros_like(want).scatter_add_(1, at, aw) if cfg.norm_topk_prob else \
        (p if cfg.score_fn == "softmax" else torch.zeros_like(p))
    mean = (aw * up.abs()).sum(1, keepdim=True)
    tol = REL * (own + share * mean * (1.0 if cfg.norm_topk_prob else 2.5)) + ref.U[logits.dtype] * want.abs()
    tol = tol + (2.0 ** -25 if logits.dtype == HF else 1e-38)  # fp16's smallest step; the fp32 range
    bad = (dl.double() - want).abs() > tol
    assert not bad.any(), ((dl.double() - want)[bad][:4], want[bad][:4])


@pytest.mark.parametrize("score", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(1, 1), (16, 4), (33, 32), (100, 7), (384, 8), (896, 16), (1021, 5), (1024, 32)])
def test_backward(E, k, score, renorm):
    for i, dt in enumerate((FL, BF, HF)):
        l, bias = _logits(50, E, dt, E + i)
        cfg = _cfg(E, k, score=score, renorm=renorm)
        idx, _ = _route(cfg, l, bias)
        dw = torch.randn(50, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i))
        idx[0] = -1           # a token that chose nothing
        idx[1, k // 2:] = -1  # some slots empty
        idx[2, 0] = E + 3     # no such expert
        dw[0] = math.nan      # ... whose gradient is never read
        dw[1, k // 2:] = math.nan
        dw[2, 0] = math.inf
        _check_backward(cfg, l, idx, dw)


def test_backward_masked_and_far_logits():
    l, bias = _logits(6, 64, FL, 5)
    l[0, 10:] = -math.inf
    l[1] = -200.0 - torch.arange(64, device="cuda")
    l[2] = 50.0 + torch.arange(64, device="cuda")
    for score in ("sigmoid", "sqrtsoftplus", "softmax"):
        cfg = _cfg(64, 4, score=score)
        idx, _ = _route(cfg, l, bias)
        dw = torch.randn(6, 4, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
        dl = torch.empty_like(l)
        moe.moe_route_backward(cfg, l, idx, dw, dl)
        assert torch.isfinite(dl).all() and (dl[0, 10:] == 0).all()
        _check_backward(cfg, l[2:], idx[2:].contiguous(), dw[2:].contiguous())
    # renormalised sigmoids far below zero go over into a softmax of the chosen
    cfg = _cfg(64, 4)
    idx, w = _route(cfg, l[1:2], None)
    dl = torch.empty_like(l[1:2])
    up = torch.tensor([[1.0, -2.0, 0.5, 3.0]], device="cuda")
    moe.moe_route_backward(cfg, l[1:2], idx, up, dl)
    s = torch.softmax(l[1, :4].double(), 0)
    want = 2.5 * s * (up[0].double() - (s * up[0].double()).sum())
    assert torch.allclose(dl[0, :4].double(), want, rtol=1e-5, atol=0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_same_expert_twice(score, renorm):
    """An expert in several slots gets the sum of their gradients."""
    l, _ = _logits(8, 40, FL, 6)
    idx = torch.randint(0, 5, (8, 6), device="cuda", dtype=torch.int32)
    dw = torch.randn(8, 6, device="cuda")
    _check_backward(_cfg(40, 6, score=score, renorm=renorm), l, idx, dw)


def test_backward_against_differences():
    """moe_route itself, evaluated either side of a logit."""
    for score in ("sigmoid", "sqrtsoftplus", "softmax"):
        for renorm in (True, False):
            cfg = _cfg(32, 4, score=score, renorm=renorm)
            l = torch.linspace(-2, 2, 32, device="cuda").view(1, 32)  # steps far above h
            idx, _ = _route(cfg, l, None)
            dw = torch.tensor([[0.3, -1.0, 2.0, 0.7]], device="cuda")
            dl = torch.empty_like(l)
            moe.moe_route_backward(cfg, l, idx, dw, dl)
            h = 2.0 ** -7
            for e in idx[0].tolist():
                f = []
                for s in (h, -h):
                    x = l.clone()
                    x[0, e] += s
                    i, w = _route(cfg, x, None)
                    by = dict(zip(i[0].tolist(), w[0].tolist()))
                    assert set(by) == set(idx[0].tolist())
                    f.append(sum(by[j] * g for j, g in zip(idx[0].tolist(), dw[0].tolist())))
                # h^2 times a third derivative of order 1, and fp32 weights over h
                assert abs((f[0] - f[1]) / (2 * h) - dl[0, e].item()) < 1e-3


@pytest.mark.parametrize("T,k,H", [(1, 1, 128), (5, 3, 128), (33, 8, 1152), (7, 32, 256), (40, 6, 7168)])
@pytest.mark.parametrize("dropped", [0.0, 0.4])
def test_combine_backward(T, k, H, dropped):
    g = torch.Generator(device="cuda").manual_seed(T)
    N = T * k
    dout = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    y = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    w = torch.rand(T, k, generator=g, device="cuda")
    row_of = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    drop = torch.rand(N, generator=g, device="cuda") < dropped
    row_of[drop] = torch.where(torch.arange(N, device="cuda") % 2 == 0, -1, N + 5).to(torch.int32)[drop]
    dy = torch.full((N, H), 3.0, dtype=BF, device="cuda")
    dw = torch.full((T, k), 3.0, device="cuda")
    cfg = _cfg(64, k, hidden=H)
    want_dy, want_dw = ref.combine_backward(dout, y, row_of, w, dy)
    moe.moe_combine_backward(cfg, dout, y, row_of, w, dy, dw)
    # one product in fp32, one rounding
    assert ((dy.double() - want_dy).abs() <= (2.0 ** -8 + 2.0 ** -24) * want_dy.abs()).all()
    size = torch.zeros(T * k, dtype=torch.float64)
    for p, row in enumerate(row_of.tolist()):
        if 0 <= row < N:
            size[p] = (dout[p // k].double() * y[row].double()).abs().sum()
    # at most H / 32 + 5 additions in a row (28 * 8 + 5 at 7168)
    assert ((dw.double().cpu() - want_dw).abs() <= 256 * 2.0 ** -24 * size.view(T, k)).all()
    only = torch.full((N, H), 3.0, dtype=BF, device="cuda")
    moe.moe_combine_backward(cfg, dout, None, row_of, w, only, None)
    assert torch.equal(only, dy)


def test_on_another_stream_and_in_a_graph():
    cfg = _cfg(384, 8, 8, 4)
    l, bias = _logits(128, 384, BF, 1)
    idx, w = _route(cfg, l, bias)
    dw = torch.randn(128, 8, device="cuda")
    dl = torch.empty_like(l)
    moe.moe_route_backward(cfg, l, idx, dw, dl)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    i2, w2, d2 = torch.empty_like(idx), torch.empty_like(w), torch.empty_like(dl)

    def step(stream=None):
        moe.moe_route(cfg, l, bias, i2, w2, stream=stream)
        moe.moe_route_backward(cfg, l, i2, dw, d2, stream=stream)
    step(s)
    s.synchronize()
    assert torch.equal(i2, idx) and torch.equal(w2, w) and torch.equal(d2, dl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    i2.zero_(), w2.zero_(), d2.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(i2, idx) and torch.equal(w2, w) and torch.equal(d2, dl)


@pytest.mark.parametrize("renorm", [True, False])
def test_sqrtsoftplus_far_below_zero(renorm):
    """e^l leaves the fp32 range at -88, sqrt(log(1 + e^l)) only at -174: weights and gradients of
    rows whose chosen logits all lie between, and around where the formula changes (-20, -80)."""
    l = torch.full((6, 32), -300.0, device="cuda")
    l[0, :4] = torch.tensor([-98.0, -100.3, -102.0, -103.5])
    l[1, :4] = torch.tensor([-102.0, -103.0, -102.5, -103.4])
    l[2, :4] = torch.tensor([-104.0, -110.0, -130.0, -150.0])
    l[3, :4] = torch.tensor([-19.9, -20.1, -19.0, -21.0])
    l[4, :4] = torch.tensor([-79.9, -80.1, -87.0, -89.0])
    l[5, :4] = torch.tensor([-800.0, -801.0, -803.0, -800.5]) if renorm else torch.tensor([-30.0, -5.0, -95.0, 2.0])
    l[5, 4:] = -1000.0
    cfg = _cfg(32, 4, score="sqrtsoftplus", renorm=renorm)
    idx, w = _route(cfg, l, None)
    x = torch.where(l.double() < -40, l.double(), 0.0)
    s = torch.where(l.double() < -40, torch.exp(x / 2), ref.scores(l.double(), "sqrtsoftplus"))
    want, order = torch.sort(s, dim=1, descending=True, stable=True)
    want = want[:, :4]
    if renorm:
        want = want / want.sum(1, keepdim=True)
    want = 2.5 * want
    assert torch.equal(idx.long(), order[:, :4])
    assert ((w.double() - want).abs() <= REL * want).all()
    # d s / d l = sig(l) / (2 s): s / 2 far below zero
    dw = torch.tensor([[0.5, -1.0, 2.0, 0.25]], device="cuda").expand(6, 4).contiguous()
    dl = torch.empty_like(l)
    moe.moe_route_backward(cfg, l, idx, dw, dl)
    at = idx.long()
    lk, p = l.double().gather(1, at), s.gather(1, at)
    slope = torch.where(lk < -40, 0.5, torch.sigmoid(lk) / (2 * p * p))  # over s
    up = dw.double()
    grad = want * slope * (up - (up * want / 2.5).sum(1, keepdim=True) if renorm else up)
    got = dl.double().gather(1, at)
    assert ((got - grad).abs() <= REL * want * (up.abs() + (3.75 if renorm else 0))).all()


@pytest.mark.parametrize("score", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3), (32, 5)])
def test_biases_of_the_lowest_value(groups, kept, score):
    """The type's lowest value as a bias is a number: such experts come last, by their logits, but
    before those that -inf masks, and a group of them before a group without any."""
    E, k = 64, 8
    lowest = torch.finfo(FL).min
    l, bias = _logits(60, E, FL, 11)
    g = torch.Generator(device="cuda").manual_seed(5)
    l[:40][torch.rand(40, E, generator=g, device="cuda") < 0.5] = -math.inf
    l[20:30, :48] = -math.inf
    l[30:34] = 0.5  # equal logits
    for many in (4, 10, 58, 64):
        b = bias.clone()
        b[torch.randperm(E, generator=g, device="cuda")[:many]] = lowest
        _check(_cfg(E, k, groups, kept, score), l, b)
        b[:8] = -math.inf  # whole groups without an expert
        _check(_cfg(E, k, groups, kept, score), l, b)
    b = torch.full((E,), lowest, device="cuda")
    b[3], b[40] = 0.5 * lowest, -lowest
    _check(_cfg(E, k, groups, kept, score), l, b)


@pytest.mark.parametrize("score", ["sigmoid", "sqrtsoftplus", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [64, 61])
def test_backward_of_masked_experts_in_slots(E, renorm, score):
    """Slots that name masked experts, some of a row's or all of them, in rows with and without others."""
    l, _ = _logits(5, E, FL, 21)
    l[0] = -math.inf
    l[1, :4] = -math.inf
    l[2, :2] = -math.inf
    l[3, 1:] = -math.inf
    idx = torch.arange(4, device="cuda", dtype=torch.int32).expand(5, 4).contiguous()
    dw = torch.randn(5, 4, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    cfg = _cfg(E, 4, score=score, renorm=renorm)
    dl = torch.full_like(l, 9)
    moe.moe_route_backward(cfg, l, idx, dw, dl)
    assert torch.isfinite(dl).all() and (dl[l == -math.inf] == 0).all()
    assert (dl[1] == 0).all() if renorm or score != "softmax" else True
    _check_backward(cfg, l[4:], idx[4:].contiguous(), dw[4:].contiguous())
    # the row whose other slots are unmasked: as if those alone had been chosen
    two = torch.full_like(dl[2:3], 9)
    only = torch.tensor([[-1, -1, 2, 3]], dtype=torch.int32, device="cuda")
    moe.moe_route_backward(cfg, l[2:3], only, dw[2:3].contiguous(), two)
    assert ((dl[2:3] - two).abs() <= REL * two.abs() + REL * 2.5 * dw[2].abs().max()).all()
