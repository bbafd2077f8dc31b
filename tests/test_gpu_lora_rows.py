"""Adapters beside rows of Y that start at any value (odd widths, parts of joined projections): what is there is added, and what lies
between the rows stays."""
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests import _serve_ref as ref
from tests._util import ensure_built
from tests.test_gpu_lora import check, grouped, make, mixed, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


# (N, pad): rows 2, 4, 6, 8, 10 and 14 bytes past a 16-byte boundary in turn, or always at one but the last column cut
ROWS = [(1, 0), (1, 2), (2, 1), (7, 0), (31, 0), (33, 2), (63, 2), (64, 1), (65, 0), (66, 0), (95, 3), (129, 1), (130, 0), (200, 2), (519, 0), (1030, 5)]


@pytest.mark.parametrize("N,pad", ROWS)
@pytest.mark.parametrize("dtype,y_dtype", [(qg.F16, qg.F32), (qg.BF16, qg.BF16), (qg.BF16, qg.F32), (qg.F16, qg.F16), (qg.BF16, qg.F16)])
@pytest.mark.parametrize("M,R", [(21, 16), (150, 40), (37, 136), (2310, 16), (1300, 40), (900, 104), (300, 256)])
def test_rows_anywhere(M, R, dtype, y_dtype, N, pad):
    """Few rows and many, each form of both kernels; the last value of Y's memory is the last row's last."""
    c = make(M, 128, N, 2, R, dtype, y_dtype, mixed(M, 2, N), seed=N, pad_y=pad, ragged=N % 2 == 1)
    check(c)
    if pad:
        d = make(M, 128, N, 2, R, dtype, y_dtype, mixed(M, 2, N), seed=N, pad_y=pad)
        memory = torch.empty(M * (N + pad) - pad, dtype=d["Y"].dtype, device=d["Y"].device)     # the last row without its padding
        memory.copy_(d["Y"].flatten()[: memory.numel()])
        before = memory.clone()
        view = torch.as_strided(memory, (M, N), (N + pad, 1))
        want, allow = ref.lora(view.clone(), d["X"], d["A"], d["B"], d["adapter"], None, d["scale"])
        row, offsets = grouped(d["adapter"], 2)
        qg.qgemm_lora_run(M, 128, N, 2, R, dtype, row, offsets, d["X"], 128, d["A"], d["B"], None, d["scale"], memory, y_dtype, N + pad)
        ref.check(view, want, allow)
        between = torch.ones(memory.numel(), dtype=torch.bool, device=memory.device)
        torch.as_strided(between, (M, N), (N + pad, 1)).fill_(False)
        assert torch.equal(memory[between], before[between])


@pytest.mark.parametrize("M,R", [(40, 16), (2400, 16), (1400, 64), (800, 128)])
@pytest.mark.parametrize("y_dtype", [qg.BF16, qg.F32])
def test_the_same_bits_wherever_the_rows_start(M, R, y_dtype):
    c = make(M, 512, 264, 3, R, qg.BF16, y_dtype, mixed(M, 3))
    outs = []
    for pad in (0, 1, 2, 3, 8):
        d = dict(c, Y=torch.zeros(M, 264 + pad, dtype=c["Y"].dtype, device=c["Y"].device))
        d["Y"][:, :264] = c["Y"]
        run(d)
        outs.append(d["Y"][:, :264].clone())
        assert not bool(d["Y"][:, 264:].any())
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
