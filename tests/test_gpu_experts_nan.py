"""NaN through the activations of the 4-bit and grouped products (GPU): what an operand's NaN scale or
value reaches stays NaN behind every activation, and nothing else does."""
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests._util import ensure_built, torch_dtype
from tests.test_gpu_fp4 import gpu_quant

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


# by the number of rows: K shared by a cluster, one block a tile, pairs of blocks
@pytest.mark.parametrize("M,N,K", [(9, 512, 4096), (40, 300, 512), (520, 2000, 1024), (2100, 2560, 1024)])
@pytest.mark.parametrize("act", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("fmt", [1, 2, 3, 4])
def test_nan_stays_behind_activations(M, N, K, act, fmt):
    g = torch.Generator(device=DEV).manual_seed(M + act)
    a, w = torch.randn(M, K, generator=g, device=DEV), torch.randn(N, K, generator=g, device=DEV) * 0.05
    row, channel = M - 2, 211
    a[row, 100], w[channel, 3] = float("nan"), float("nan")
    if fmt >= 3:
        A, B = gpu_quant(a, M, K, fmt), gpu_quant(w, N, K, fmt, 1)
    else:
        A, B = (a.to(torch_dtype(fmt)), None, None), (w.to(torch_dtype(fmt)), None, None)
    for dt in (0, 1, 2):
        C = torch.zeros(M, N // 2 if act == 4 else N, dtype=torch_dtype(dt), device=DEV)
        if fmt >= 3:
            qg.qgemm_fp4_run(M, K, N, fmt, A[0], A[1], A[2], B[0], B[1], B[2], None, act, None, C, dt)
        else:
            offsets = torch.tensor([0, M], dtype=torch.int32, device=DEV)
            qg.qgemm_grouped_run(M, 1, K, N, fmt, offsets, A[0], None, None, B[0], None, None, None, act, C, dt)
        assert qg.qgemm_status() == 0
        want = torch.zeros(C.shape, dtype=torch.bool)
        want[row], want[:, channel // 2 if act == 4 else channel] = True, True
        assert torch.equal(torch.isnan(C).cpu(), want)
