"""The order of rows by adapter in batches that take the kernel several turns of its blocks (16384 rows each)."""
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests._util import ensure_built

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("kind", ["any", "outside", "runs", "late"])
@pytest.mark.parametrize("L", [1, 3, 1024])
@pytest.mark.parametrize("M", [16383, 16384, 16385, 32768, 32769, 49153, 70001])
def test_turns(M, L, kind):
    g = torch.Generator().manual_seed(M + L)
    ids = {"any": lambda: torch.randint(L, (M,), generator=g), "outside": lambda: torch.randint(-L, 2 * L, (M,), generator=g),
           "runs": lambda: torch.arange(M) // 9001 % L, "late": lambda: torch.where(torch.arange(M) < M - 5, -1, L - 1)}[kind]()
    none = (ids < 0) | (ids >= L)
    order = torch.sort(torch.where(none, L, ids), stable=True).indices.int()
    count = int((~none).sum())
    order[count:] = -1
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64), torch.cumsum(torch.bincount(ids[~none], minlength=L), 0))).int()
    guard = 64
    row = torch.full((M + guard,), 77, dtype=torch.int32, device=DEV)
    got = torch.full((L + 1 + guard,), 77, dtype=torch.int32, device=DEV)
    for _ in range(2):
        qg.qgemm_lora_group(M, L, ids.int().to(DEV), row, got)
        assert torch.equal(row[:M].cpu(), order) and torch.equal(got[: L + 1].cpu(), offsets)
        assert bool((row[M:] == 77).all()) and bool((got[L + 1:] == 77).all())
