"""The bounded waits of every form of the product kernel run out on purpose (GPU), as in
test_gpu_experts_timeout.py, at shapes whose form is asserted: pairs of blocks in the 4-bit formats, and
clusters that share the K of 128-row tiles."""
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests._util import ensure_built
from tests.test_gpu_fp4 import operands
from tests.test_gpu_group_tiles import plan

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("fmt", [2, 3, 4])
# (the grouped call's 16-bit operands take smaller tiles at two of these shapes)
@pytest.mark.parametrize("M,K,N,form,form16", [
    (513, 4096, 4000, (256, 1), (128, 1)), (2048, 1024, 14336, (256, 1), (256, 1)), (128, 9728, 2500, (128, 4), (128, 2)),
    (120, 9728, 1200, (128, 8), (128, 8)), (300, 4096, 4096, (128, 1), (128, 1)), (40, 8192, 300, (32, 8), (32, 8))])
def test_wait_runs_out_then_next_call_is_exact(M, K, N, form, form16, fmt):
    assert plan(M, 1, fmt == 2, K, N, fmt) == (form16 if fmt == 2 else form)
    if fmt == 2:
        A, B = (torch.randn(M, K, device=DEV).bfloat16(), None, None), (torch.randn(N, K, device=DEV).bfloat16(), None, None)
    else:
        A, B, _, _ = operands(M, N, K, fmt, 5)
    offsets = torch.tensor([0, M], dtype=torch.int32, device=DEV)

    def run():
        C = torch.full((M, N), float("nan"), device=DEV)
        if fmt == 2:
            qg.qgemm_grouped_run(M, 1, K, N, fmt, offsets, A[0], None, None, B[0], None, None, None, 0, C, 0)
        else:
            qg.qgemm_fp4_run(M, K, N, fmt, A[0], A[1], A[2], B[0], B[1], B[2], None, 0, None, C, 0)
        return C

    ref = run()
    assert qg.qgemm_status() == 0 and torch.isfinite(ref).all()
    prev = qg.qgemm_set_option(qg.OPT_WAIT_LIMIT_US, 2000), qg.qgemm_set_option(qg.OPT_DEBUG_STALL, 1)
    try:
        run()
        assert qg.qgemm_status() == -6
        assert qg.qgemm_status() == 0
    finally:
        qg.qgemm_set_option(qg.OPT_WAIT_LIMIT_US, prev[0])
        qg.qgemm_set_option(qg.OPT_DEBUG_STALL, prev[1])
    for _ in range(2):
        assert torch.equal(run(), ref)
    assert qg.qgemm_status() == 0
