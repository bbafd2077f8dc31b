"""The bounded waits of the 4-bit and grouped products, made to run out on purpose (GPU).

As in test_gpu_timeout.py, QGEMM_OPT_DEBUG_STALL has the role that issues the MMAs wait first on a
barrier that nothing arrives at. The call must end by itself within the lowered bound, alone (one
block a tile), in a cluster that shares a tile's K and in pairs of blocks; qgemm_status reports the
timeout and clears it, and the next call gives the bits of an undisturbed one."""
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests._util import ensure_built
from tests.test_gpu_fp4 import operands

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("fmt", [2, 3, 4])
@pytest.mark.parametrize("M,N,K", [(1, 24000, 512), (9, 512, 4096), (100, 300, 2048), (120, 20000, 512), (400, 1000, 1024), (2000, 4000, 512)])
def test_wait_runs_out_then_next_call_is_exact(M, N, K, fmt):
    if fmt == 2:
        a, b = torch.randn(M, K, device=DEV).bfloat16(), torch.randn(N, K, device=DEV).bfloat16()
        A, B = (a, None, None), (b, None, None)
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
