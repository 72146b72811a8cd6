"""The operators' outputs as torch sees them: version counters, so that autograd notices a saved
tensor that a call has overwritten, and parameters that require a gradient."""
import pytest
import torch

import expert_routing_grouped_layer_b200 as moe
from expert_routing_grouped_layer_b200 import workloads as W

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def _calls():
    """(call, arguments, positions that it writes)"""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s, t=torch.float32: torch.randn(*s, generator=g, device="cuda").to(t)
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")
    cfg = W.CONFIGS["tiny_bf16"]
    E, k, H = cfg.n_routed_experts, cfg.num_experts_per_tok, cfg.hidden
    ws = z(1 << 20, t=torch.uint8)
    idx = torch.arange(4 * k, device="cuda", dtype=I32).view(4, k) % E
    rows = torch.arange(4 * k, device="cuda", dtype=I32)
    return [(moe.moe_norm, (r(4, 64, t=BF), r(64), r(64), 1e-6, z(4, 64, t=BF), z(4), z(4)), (4, 5, 6)),
            (moe.moe_norm_backward, (r(4, 64, t=BF), r(4, 64, t=BF), r(64), z(4), z(4), z(4, 64, t=BF), z(64), z(64),
                                     ws), (5, 6, 7, 8)),
            (moe.moe_route, (cfg, r(4, E), r(E), z(4, k, t=I32), z(4, k)), (3, 4)),
            (moe.moe_route_backward, (cfg, r(4, E), idx, r(4, k), z(4, E)), (4,)),
            (moe.moe_combine_backward, (cfg, r(4, H, t=BF), r(4 * k, H, t=BF), rows, r(4, k), z(4 * k, H, t=BF),
                                        z(4, k)), (5, 6)),
            (moe.moe_linear, (r(4, 64, t=BF), r(8, 64, t=BF), r(8), r(4, 8, t=BF), z(4, 8, t=BF), z(4, 8, t=BF)),
             (4, 5)),
            (moe.moe_linear_backward, (r(4, 8, t=BF), r(4, 64, t=BF), r(8, 64, t=BF), None, z(4, 64, t=BF),
                                       z(8, 64, t=BF), z(8), ws), (4, 5, 6, 7))]


def test_outputs_raise_their_version():
    for fn, args, written in _calls():
        before = {i: a._version for i, a in enumerate(args) if isinstance(a, torch.Tensor)}
        fn(*args)
        for i, v in before.items():
            assert args[i]._version == v + (1 if i in written else 0), (fn.__name__, i)


def test_backward_notices_an_overwritten_tensor():
    fn, args, _ = _calls()[0]
    leaf = torch.ones(4, 64, dtype=BF, device="cuda", requires_grad=True)
    loss = (leaf * args[4]).sum()  # saves y
    fn(*args)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_parameters_under_no_grad_and_inference_mode():
    for fn, args, written in _calls():
        fn(*args)
        want = [args[i].clone() for i in written if args[i].dtype != torch.uint8]
        for mode in (torch.no_grad, torch.inference_mode):
            with mode():
                new = [a.clone() if isinstance(a, torch.Tensor) else a for a in args]
                if mode is torch.no_grad:
                    for a in new:
                        if isinstance(a, torch.Tensor) and a.is_floating_point():
                            a.requires_grad_()
                fn(*new)
                got = [new[i] for i in written if args[i].dtype != torch.uint8]
                assert all(torch.equal(a, b) for a, b in zip(want, got)), fn.__name__
