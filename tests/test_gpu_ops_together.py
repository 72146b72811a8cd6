"""The operators around the experts in one training step of a block, as a program uses them:
norm -> router product -> routing -> permutation -> experts -> combine, then back through
the combine, the routing, the router product and the norm (the experts frozen), and a
dense layer with its residual beside them. Checked against 64-bit autograd over the same
inputs, with the experts' output rows and the chosen experts taken from the run.

Tolerance: relative L2. The run rounds to bf16 the normalised rows, the logits, the combined
output's gradient into rows, dlogits, and each matrix product's output: at most 7 roundings
on the way to any gradient, each at most 2^-8 of its value, and a logit's rounding error
(2^-8 of about 2) reaches a weight undiminished: 9 * 2^-8 = 3.5e-2 in all."""
import pytest
import torch

import expert_routing_grouped_layer_b200 as moe
import ops_reference as ref
from expert_routing_grouped_layer_b200 import workloads as W

pytestmark = pytest.mark.gpu
TOL = 9 * 2.0 ** -8
BF = torch.bfloat16


class Block:
    """A block's parameters, workspaces and gradients, allocated once."""

    def __init__(self, T, seed):
        self.cfg = W.CONFIGS["tiny_bf16"].replace(T=T, n_group=4, topk_group=2)
        c = self.cfg
        H, E, k, I, S = (c.hidden, c.n_routed_experts, c.num_experts_per_tok, c.moe_intermediate_size,
                         c.n_shared_experts)
        N = T * k
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
        e = lambda *s, t=BF: torch.empty(*s, dtype=t, device="cuda")
        self.x, self.dout, self.ddense = rand(T, H).to(BF), rand(T, H).to(BF), rand(T, H).to(BF)
        self.nw, self.nb = 1 + 0.2 * rand(H), 0.1 * rand(H)
        self.wr = (1.7 * rand(E, H) * H ** -0.5).to(BF)
        self.bias = 0.1 * rand(E)
        self.wd, self.bd = (rand(H, H) * H ** -0.5).to(BF), 0.1 * rand(H)
        self.experts = W.make_weights(c, "cuda")
        f, i = torch.float32, torch.int32
        self.ws = e(moe.moe_workspace_bytes(c, T), t=torch.uint8)
        self.status = torch.zeros(1, dtype=i, device="cuda")
        self.h, self.mean, self.rstd = e(T, H), e(T, t=f), e(T, t=f)
        self.logits, self.idx, self.w = e(T, E), e(T, k, t=i), e(T, k, t=f)
        self.off, self.pairs, self.row_of = e(E + 1, t=i), e(N, t=i), e(N, t=i)
        self.y, self.sy, self.out = e(N, H), e(S, T, H), e(T, H)
        self.dense, self.pre = e(T, H), e(T, H)
        self.dy, self.dw, self.dlogits = torch.zeros(N, H, dtype=BF, device="cuda"), e(T, k, t=f), e(T, E)
        self.dh, self.dwr = e(T, H), e(E, H)
        self.dx, self.dnw, self.dnb = e(T, H), e(H, t=f), e(H, t=f)
        self.dhd, self.dwd, self.dbd = e(T, H), e(H, H), e(H, t=f)
        need = max(moe.moe_norm_backward_workspace_bytes(T, H),
                   moe.moe_linear_backward_workspace_bytes(T, H, H, "gelu"))
        self.ops_ws = e(need, t=torch.uint8)

    def step(self):
        c, T = self.cfg, self.cfg.T
        moe.moe_norm(self.x, self.nw, self.nb, 1e-6, self.h, self.mean, self.rstd)
        moe.moe_linear(self.h, self.wr, None, None, self.logits, dev_status=self.status)
        moe.moe_route(c, self.logits, self.bias, self.idx, self.w)
        moe.moe_permute(c, self.idx, T, self.off, self.pairs, self.row_of, self.status, self.ws)
        moe.moe_grouped_swiglu(c, self.h, T, self.pairs, self.off, self.experts, self.y, self.sy, self.ws,
                               self.status)
        moe.moe_combine(c, self.y, self.sy, self.row_of, self.w, T, self.out)
        moe.moe_linear(self.h, self.wd, self.bd, self.x, self.dense, self.pre, act="gelu",
                       dev_status=self.status)
        # and back
        moe.moe_combine_backward(c, self.dout, self.y, self.row_of, self.w, self.dy, self.dw)
        moe.moe_route_backward(c, self.logits, self.idx, self.dw, self.dlogits)
        moe.moe_linear_backward(self.dlogits, self.h, self.wr, None, self.dh, self.dwr, None, self.ops_ws,
                                dev_status=self.status)
        moe.moe_norm_backward(self.dh, self.x, self.nw, self.mean, self.rstd, self.dx, self.dnw, self.dnb,
                              self.ops_ws)
        moe.moe_linear_backward(self.ddense, self.h, self.wd, self.pre, self.dhd, self.dwd, self.dbd,
                                self.ops_ws, act="gelu", dev_status=self.status)

    def results(self):
        return [self.out, self.dense, self.idx, self.w, self.dy, self.dw, self.dlogits, self.dwr, self.dx,
                self.dnw, self.dnb, self.dhd, self.dwd, self.dbd]


def _rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("T", [1, 50, 700])
def test_block_step(T):
    b = Block(T, T)
    b.step()
    torch.cuda.synchronize()
    assert b.status.item() == 0
    x, nw, nb, wr, wd, bd = (t.double().requires_grad_(True) for t in (b.x, b.nw, b.nb, b.wr, b.wd, b.bd))
    mean = x.mean(1, keepdim=True)
    h = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + 1e-6) * nw + nb
    w = ref.route_weights(b.cfg, h @ wr.t(), b.idx)
    k = b.cfg.num_experts_per_tok
    rows = b.y.double()[b.row_of.long()].view(T, k, -1)
    out = (w[:, :, None] * rows).sum(1)
    assert _rel(b.out.float(), (out + b.sy.double().sum(0)).detach()) < TOL
    assert _rel(b.w, w.detach()) < TOL
    gx, gnw, gnb, gwr = torch.autograd.grad((out * b.dout.double()).sum(), (x, nw, nb, wr), retain_graph=True)
    for got, want in ((b.dx, gx), (b.dnw, gnw), (b.dnb, gnb), (b.dwr, gwr)):
        assert _rel(got, want) < TOL
    dense = ref.act(h @ wd.t() + bd, "gelu") + x
    assert _rel(b.dense, dense.detach()) < TOL
    gh, gwd, gbd = torch.autograd.grad((dense * b.ddense.double()).sum(), (h, wd, bd))
    for got, want in ((b.dhd, gh), (b.dwd, gwd), (b.dbd, gbd)):
        assert _rel(got, want) < TOL


def test_block_step_captured():
    """The whole step in a graph, replayed on new inputs, gives the bits of direct calls."""
    s = torch.cuda.Stream()
    b = Block(130, 7)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b.step()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            b.step()
        b.x.neg_()
        b.dout.mul_(2)
        g.replay()
        s.synchronize()
        got = [r.clone() for r in b.results()]
        for r in b.results():
            r.zero_()
        b.step()
        s.synchronize()
    assert all(torch.equal(a, r) for a, r in zip(got, b.results()))
    assert b.status.item() == 0


def test_two_blocks_at_once():
    """Two steps with their own workspaces on two streams do not disturb one another."""
    blocks = [Block(300, 11), Block(300, 12)]
    want = []
    for b in blocks:
        b.step()
        torch.cuda.synchronize()
        want.append([r.clone() for r in b.results()])
        for r in b.results():
            r.zero_()
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.step()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        assert all(torch.equal(a, r) for a, r in zip(w, b.results()))


@pytest.mark.parametrize("T", [6, 3000])
def test_nan_weight_of_a_pair_without_a_row_reaches_the_output(T):
    """On both sides of the combine's small-batch path; finite weights of such pairs add nothing."""
    cfg = W.CONFIGS["tiny_bf16"]
    H, k = cfg.hidden, cfg.num_experts_per_tok
    S = cfg.n_shared_experts
    g = torch.Generator(device="cuda").manual_seed(T)
    y, sy = torch.randn(T * k, H, generator=g, device="cuda").to(BF), torch.randn(S, T, H, generator=g, device="cuda").to(BF)
    row_of = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda")
    row_of.view(T, k)[1:4] = -1
    row_of.view(T, k)[4, 1:] = -1
    out, want = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")
    moe.moe_combine(cfg, y, sy, row_of, w, T, want)
    w[2], w[4, 1] = float("nan"), float("nan")
    moe.moe_combine(cfg, y, sy, row_of, w, T, out)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[2, 4]] = False
    assert torch.isnan(out[[2, 4]]).all()
    assert torch.equal(out[keep], want[keep]) and torch.isfinite(want).all()
    w[2], w[4, 1] = 3.0, 5.0
    moe.moe_combine(cfg, y, sy, row_of, w, T, out)
    assert torch.equal(out, want)


def _permute(cfg, idx, T):
    N, E = T * cfg.num_experts_per_tok, cfg.n_routed_experts
    e = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")
    off, pairs, row_of, st = e(E + 1), e(N), e(N), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    moe.moe_permute(cfg, idx, T, off, pairs, row_of, st, ws)
    return off, pairs, row_of, st.item()


@pytest.mark.parametrize("T", [9, 3000])  # one CTA, and several chunks of pairs
def test_permute_takes_minus_one_as_no_expert(T):
    cfg = W.CONFIGS["tiny_bf16"]
    k, E = cfg.num_experts_per_tok, cfg.n_routed_experts
    idx = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T))
    idx[2], idx[5, 1:], idx[T - 1] = -1, -1, -1
    off, pairs, row_of, st = _permute(cfg, idx, T)
    flat = idx.view(-1)
    has = flat >= 0
    n = int(has.sum())
    order = torch.sort(torch.where(has, flat, E), stable=True)[1][:n]
    assert st == 0 and off[E].item() == n
    assert torch.equal(pairs[:n].long(), order) and (pairs[n:] == -7).all()
    assert (row_of[~has] == -1).all() and torch.equal(row_of[order].long(), torch.arange(n, device="cuda"))
    for bad in (-2, E):  # any other id outside the range is an error
        idx[3, 0] = bad
        assert _permute(cfg, idx, T)[3] == moe.MOE_DEV_BAD_EXPERT


@pytest.mark.parametrize("T", [50, 2500])
def test_padded_and_nan_tokens(T):
    """Masked (padded) tokens, tokens with fewer experts than k and a token with a NaN logit through the
    routing, the permutation, the experts, the combine and back. Tolerance: the combine's one rounding
    (2^-8 of the result) and fp32 sums of at most 16 terms."""
    b = Block(T, T + 1)
    c, k, E = b.cfg, b.cfg.num_experts_per_tok, b.cfg.n_routed_experts
    pad = torch.arange(T, device="cuda") % 7 == 3
    moe.moe_norm(b.x, b.nw, b.nb, 1e-6, b.h, b.mean, b.rstd)
    moe.moe_linear(b.h, b.wr, None, None, b.logits, dev_status=b.status)
    b.logits[pad] = -float("inf")
    b.logits[1, 2:] = -float("inf")
    b.logits[2, 5] = float("nan")
    moe.moe_route(c, b.logits, b.bias, b.idx, b.w)
    moe.moe_permute(c, b.idx, T, b.off, b.pairs, b.row_of, b.status, b.ws)
    assert (b.idx[pad] == -1).all() and (b.idx[2] == -1).all() and (b.idx[1] >= 0).sum() == 2
    b.y.fill_(float("nan"))  # rows that no pair has stay so, and reach nothing
    moe.moe_grouped_swiglu(c, b.h, T, b.pairs, b.off, b.experts, b.y, b.sy, b.ws, b.status)
    moe.moe_combine(c, b.y, b.sy, b.row_of, b.w, T, b.out)
    assert b.status.item() == 0
    has = b.row_of.view(T, k) >= 0
    assert torch.equal(has, b.idx >= 0) and b.off[E].item() == has.sum().item()
    rows = b.y.double()[b.row_of.long().clamp(min=0)].view(T, k, -1)
    terms = torch.where(has[:, :, None], b.w.double()[:, :, None] * rows, 0.0)
    want = terms.sum(1) + b.sy.double().sum(0)
    size = terms.abs().sum(1) + b.sy.double().abs().sum(0)
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    good[2] = False
    assert torch.isnan(b.out[2]).all()
    assert ((b.out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size)[good].all()
    # and back: empty slots get no gradient, padded rows none at all
    moe.moe_combine_backward(c, b.dout, b.y, b.row_of, b.w, b.dy, b.dw)
    assert torch.isfinite(b.dy).all() and (b.dw[~has] == 0).all() and torch.isfinite(b.dw).all()
    b.dw[~has] = float("nan")
    moe.moe_route_backward(c, b.logits, b.idx, b.dw, b.dlogits)
    assert torch.isfinite(b.dlogits).all() and (b.dlogits[pad] == 0).all() and (b.dlogits[2] == 0).all()
    moe.moe_linear_backward(b.dlogits, b.h, b.wr, None, b.dh, b.dwr, None, b.ops_ws, dev_status=b.status)
    moe.moe_norm_backward(b.dh, b.x, b.nw, b.mean, b.rstd, b.dx, b.dnw, b.dnb, b.ops_ws)
    assert (b.dx[pad] == 0).all() and torch.isfinite(b.dnw).all() and b.status.item() == 0
