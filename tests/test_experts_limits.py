"""Sizes past what the 4-bit and mixture-of-experts calls can count are refused, not wrapped around (no GPU:
every call here fails its checks before a launch)."""
import pytest

from tests._util import ensure_built
from tests.test_experts_abi import GROUPED, RUN, UNSUP, call


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("K", [1 << 30, (1 << 30) + 64, (1 << 31) - 64])
@pytest.mark.parametrize("fmt", [1, 2, 3, 4])
def test_products_refuse_long_rows(K, fmt):
    """A 16-bit row of 2^30 values has more bytes than an int counts: no product would be issued."""
    assert call("qgemm_grouped_run", GROUPED, dict(T=1, E=1, N=1, K=K, fmt=fmt)) == UNSUP
    if fmt >= 3:
        assert call("qgemm_fp4_run", RUN, dict(M=1, N=1, K=K, fmt=fmt)) == UNSUP
