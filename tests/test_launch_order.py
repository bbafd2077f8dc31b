"""When a kernel may come up behind the one before it in the stream (programmatic dependent launch).

A decode call with QGEMM_OPT_LAUNCH_OVERLAP reads its weight before its own wait; the contract only
forbids the kernel launched immediately before it to write that weight. So every kernel further back
must be complete by then, which holds if no kernel releases its dependents before its own wait. The
CPU part takes each kernel's order of release and wait from the sources and derives what is ordered
before what in a chain; the GPU part runs such chains."""
import glob
import itertools
import os
import re

import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests._util import ROOT, ensure_built

RELEASE = re.compile(r"grid_release\(\)|griddepcontrol\.launch_dependents")
WAIT = re.compile(r"grid_wait\(\)|griddepcontrol\.wait")


def kernels():
    """{kernel: its releases and waits in source order} of every kernel that has any."""
    out = {}
    for path in sorted(glob.glob(os.path.join(ROOT, "weight_quantized_gemm_gb300", "csrc", "*.cu*"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for body in src.split("__global__")[1:]:
            name = re.search(r"void\s+(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\s*\(", body).group(1)
            body = body[: body.find("\n}")]
            found = sorted([(m.start(), "release") for m in RELEASE.finditer(body)] + [(m.start(), "wait") for m in WAIT.finditer(body)])
            if found:
                out[name] = [what for _, what in found]
    return out


def complete_before_start(chain):
    """For each kernel of the chain (its order of 'release' and 'wait'), the kernels known to be
    complete when it comes up, if all are launched with the attribute."""
    known, at_wait = [], []
    for i, order in enumerate(chain):
        if i == 0:
            start = set()
        else:
            # it comes up once its predecessor has released it; without a release, once that is complete
            before = chain[i - 1]
            if "release" not in before:
                start = at_wait[i - 1] | {i - 1}
            elif before.index("release") > before.index("wait"):
                start = at_wait[i - 1]
            else:
                start = known[i - 1]
        known.append(start)
        # its wait ends when its predecessor is complete, which itself has waited
        at_wait.append(start | (at_wait[i - 1] | {i - 1} if i else set()))
    return known


def test_sources_have_the_kernels():
    assert {"mx_quant_kernel", "nv_quant_kernel", "fp4_dequant_kernel", "group_gemm_kernel", "combine_kernel", "route_small_kernel",
            "stream_kernel"} <= set(kernels())


def test_only_the_kernel_just_before_may_still_run():
    found = kernels()
    for names in itertools.product(found, repeat=3):
        chain = [found[n] for n in names] + [["wait", "release"]]
        for i, known in enumerate(complete_before_start(chain)):
            assert known >= set(range(i - 1)), f"a kernel after {names[:i]} comes up before one two back is complete"


@pytest.mark.gpu
@pytest.mark.parametrize("between", ["quant", "combine", "decode"])
def test_weight_written_two_kernels_back(between):
    """fp4_dequant writes a FLOAT weight, another call follows, then a decode call reads the weight
    with the overlap option on: the bits of the same chain without the option."""
    ensure_built()
    dev, M, K, N, rounds = "cuda", 8, 4096, 4096, 12
    x = torch.randn(M, K, device=dev).bfloat16()
    weights = []
    for i in range(3):
        w = torch.randn(N, K, device=dev) * 0.02
        codes = torch.empty(qg.qgemm_fp4_codes_bytes(N, K), dtype=torch.uint8, device=dev)
        scales = torch.empty(qg.qgemm_fp4_scales_bytes(N, K, qg.FMT_MXFP4, 0), dtype=torch.uint8, device=dev)
        qg.qgemm_fp4_quant(N, K, w, qg.F32, K, N, None, qg.FMT_MXFP4, 0, codes, scales)
        weights.append((codes, scales))
    Bp, other = torch.zeros(N, K, dtype=torch.bfloat16, device=dev), torch.randn(128, K, device=dev).bfloat16()
    side, slot = torch.empty(M, 128, dtype=torch.bfloat16, device=dev), torch.arange(M, dtype=torch.int32, device=dev).view(M, 1)
    one, summed = torch.ones(M, 1, device=dev), torch.empty_like(x)
    a = (torch.empty(M, K // 2, dtype=torch.uint8, device=dev),
         torch.empty(qg.qgemm_fp4_scales_bytes(M, K, qg.FMT_MXFP4, 0), dtype=torch.uint8, device=dev))
    wsb = max(qg.qgemm_workspace_bytes(M, K, n, qg.MODE_FLOAT, 0, qg.BF16, qg.BF16) for n in (N, 128))
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)

    def chain():
        outs = []
        for i in range(rounds):
            C = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
            qg.qgemm_fp4_dequant(N, K, qg.FMT_MXFP4, 0, *weights[i % 3], None, Bp, qg.BF16)
            if between == "quant":
                qg.qgemm_fp4_quant(M, K, x, qg.BF16, K, M, None, qg.FMT_MXFP4, 0, *a)
            elif between == "combine":
                qg.qgemm_moe_combine(M, 1, K, M, x, qg.BF16, slot, one, None, summed, qg.BF16)
            else:
                qg.qgemm_run(M, K, 128, qg.MODE_FLOAT, 0, x, qg.BF16, other, None, side, qg.BF16, ws, wsb)
            qg.qgemm_run(M, K, N, qg.MODE_FLOAT, 0, x, qg.BF16, Bp, None, C, qg.BF16, ws, wsb)
            outs.append(C)
        torch.cuda.synchronize()
        return outs

    want = chain()
    full = torch.empty(N, K, dtype=torch.bfloat16, device=dev)
    for i in range(3):
        qg.qgemm_fp4_dequant(N, K, qg.FMT_MXFP4, 0, *weights[i], None, full, qg.BF16)
        ref = x.double() @ full.double().T
        assert float((want[i].double() - ref).norm() / ref.norm()) < 4e-3        # bf16 output
    prev = qg.qgemm_set_option(qg.OPT_LAUNCH_OVERLAP, 1)
    try:
        for _ in range(5):
            for got, ref in zip(chain(), want):
                assert torch.equal(got, ref)
    finally:
        qg.qgemm_set_option(qg.OPT_LAUNCH_OVERLAP, prev)
    assert qg.qgemm_status() == 0
