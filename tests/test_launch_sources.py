"""Launches in the sources: every kernel goes through one of the two helpers of sm100.cuh, both of which
set programmatic serialization, and every kernel that they launch waits for its predecessor first."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "expert_routing_grouped_layer_b200", "csrc")


def _text(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def _sources():
    return {os.path.basename(p): _text(p) for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*")))}


def _kernels():
    """(file, name, the body's first two statements)"""
    out = []
    for name, text in _sources().items():
        for m in re.finditer(r"__global__ void", text):
            body = text.index("{", m.end())
            sig = re.sub(r"__launch_bounds__\((?:[^()]|\([^()]*\))*\)", "", text[m.end():body])
            out.append((name, re.search(r"(\w+)\s*\(", sig).group(1),
                        [s.strip() for s in text[body + 1:].split(";")[:2]]))
    return out


def test_every_kernel_waits_first():
    kernels = [k for k in _kernels() if k[0] != "selftest.cu"]
    for f, name, first in kernels:
        assert first == ["pdl_wait()", "pdl_trigger()"], (f, name, first)
    names = {k[1] for k in kernels}
    rows = {"norm_fwd_kernel", "norm_fwd_ring_kernel", "norm_bwd_ring_kernel", "norm_fwd_ragged_kernel",
            "norm_bwd_ragged_kernel", "norm_param_kernel", "route_fwd_kernel", "route_bwd_kernel",
            "combine_bwd_kernel", "linear_pair_kernel", "linear_split_kernel", "linear_act_bwd_kernel",
            "linear_bias_kernel"}
    assert rows <= names and len(kernels) >= 31


def test_both_launch_helpers_set_programmatic_serialization():
    text = _sources()["sm100.cuh"]
    for helper in ("launch_pdl", "launch_cluster"):
        body = text[text.index("inline cudaError_t %s(" % helper):]
        body = body[:body.index("\n}\n")]
        assert "cudaLaunchAttributeProgrammaticStreamSerialization" in body, helper
        assert "programmaticStreamSerializationAllowed = 1" in body, helper
        attributes = int(re.search(r"cudaLaunchAttribute attr\[(\d)\]", body).group(1))
        assert "cfg.numAttrs = %d" % attributes in body, helper  # all of them are passed


def test_no_launch_past_the_helpers():
    for name, text in _sources().items():
        if name in ("sm100.cuh", "selftest.cu"):
            continue
        assert "<<<" not in text and "cudaLaunch" not in text, name
