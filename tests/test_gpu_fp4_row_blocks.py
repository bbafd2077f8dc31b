"""NVFP4 quantization at every number of warps a row (GPU): one to eight, hence eight rows to one in a thread
block, with a last block that is part full, and rows longer than a block keeps in registers."""
import pytest
import torch

from tests._util import ensure_built, torch_dtype
from tests.test_gpu_fp4 import NV, check_quant, gpu_quant, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("warps", [1, 2, 3, 4, 5, 6, 7, 8, 9])
@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("layout", [0, 1])
def test_warps_of_a_row(warps, dt, layout):
    per = 1024 if dt == 0 else 2048                 # values that a warp keeps
    K, M = per * warps - 512, 11
    g = torch.Generator(device="cuda").manual_seed(K)
    x = (torch.randn(M, K, generator=g, device="cuda") * torch.exp2(torch.arange(M, device="cuda").float() - 5)[:, None]).to(torch_dtype(dt))
    x[3, K - 1] = 500.0                             # the row's largest value in its last warp
    check_quant(host(x), *gpu_quant(x, M, K, NV, layout), NV, layout, K)
