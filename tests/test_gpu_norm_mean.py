"""LAYER norms of rows whose mean is large beside their spread, at widths that are no power of two (1 / K is rounded there)."""
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests import _serve_ref as ref
from tests._util import ensure_built
from tests.test_gpu_norm import DEV, check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("post", [0, 1])
@pytest.mark.parametrize("M,K", [(5, 64), (5, 192), (5, 448), (400, 1344), (4, 3584), (700, 3584), (3, 7168), (320, 7168), (305, 9728), (2, 20032)])
@pytest.mark.parametrize("x_dtype,value", [(qg.BF16, 100.0), (qg.BF16, -0.10009765625), (qg.F16, 1000.0), (qg.F16, 0.0999755859375), (qg.F32, 1543.0)])
def test_rows_of_one_value_are_zero(M, K, x_dtype, value, post):
    """K times the value and every sum on the way are exact: the values have 8, 11 or 12 bits (1543), and a sum is a value times a
    number of pieces of 8, of 12 bits at most. So the mean is the value, and the centred values are 0."""
    c = make(M, K, qg.NORM_LAYER, x_dtype, qg.F32, qg.F32, post=post, gate="none", residual=False, affine="both")
    c["X"].fill_(value)
    S, Y = run(c)
    assert torch.equal(Y, c["bias"].expand(M, K))
    if post:
        assert not bool(S.any())


@pytest.mark.parametrize("mean", [100.0, 1000.0])
@pytest.mark.parametrize("M,K", [(4, 3584), (500, 3584), (2, 7168), (305, 9728), (2, 20032)])
def test_a_large_mean(M, K, mean):
    check(make(M, K, qg.NORM_LAYER, qg.F32, qg.F32, qg.F32, post=0, gate="none", residual=False, mean=mean))


@pytest.mark.parametrize("K", [448, 3584, 7168, 20032])
def test_nan_and_infinity_stay_in_their_rows(K):
    c = make(6, K, qg.NORM_LAYER, qg.BF16, qg.F32, qg.F32)
    c["X"][1, 3], c["X"][4, K - 1] = float("nan"), float("inf")
    good = torch.tensor([0, 2, 3, 5], device=DEV)
    S, Y = run(c)
    assert bool(torch.isnan(Y[1]).all()) and bool(torch.isnan(Y[4]).all())
    for n in ("X", "residual"):
        c[n] = c[n][good].contiguous()
    c["M"] = 4
    S2, Y2 = run(c)
    assert torch.equal(S[good], S2) and torch.equal(Y[good], Y2)
    check(c)
