"""Sizes past what the 4-bit and mixture-of-experts calls can count are refused, not wrapped around (no GPU:
every call here fails its checks before a launch)."""
import pytest

import weight_quantized_gemm_gb300 as qg
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


@pytest.mark.parametrize("rows", [(1 << 30) + 1, (1 << 31) - 127, (1 << 31) - 1])
def test_sizes_of_too_many_rows_are_zero(rows):
    """More rows than a call takes; near 2^31 rounding them up to a tile wrapped around."""
    assert qg.qgemm_fp4_codes_bytes(rows, 64) == 0
    for fmt in (3, 4):
        for layout in (0, 1):
            assert qg.qgemm_fp4_scales_bytes(rows, 64, fmt, layout) == 0


def test_sizes_of_the_most_rows():
    rows, K = 1 << 30, 128
    assert qg.qgemm_fp4_codes_bytes(rows, K) == rows * 64
    assert qg.qgemm_fp4_scales_bytes(rows, K, 3, 0) == rows * 16
    assert qg.qgemm_fp4_scales_bytes(rows, K, 4, 1) == rows // 128 * 2 * 512


@pytest.mark.parametrize("K", [(1 << 31) - 64, (1 << 30) + 64])
def test_sizes_of_the_longest_rows(K):
    assert qg.qgemm_fp4_codes_bytes(3, K) == 3 * (K // 2)
    for fmt, block in ((3, 32), (4, 16)):
        n = K // block
        assert qg.qgemm_fp4_scales_bytes(3, K, fmt, 0) == 3 * (-(-n // 16) * 16)
        assert qg.qgemm_fp4_scales_bytes(3, K, fmt, 1) == -(-n // 4) * 512


@pytest.mark.parametrize("args", [dict(M=1 << 30, N=1 << 30), dict(M=1 << 30, N=1 << 24, act=0), dict(M=1, N=1 << 30, K=1 << 20)])
def test_dense_refuses_tiles_past_counting(args):
    assert call("qgemm_fp4_run", RUN, args) == UNSUP
    assert "tiles" in qg.qgemm_last_error()


@pytest.mark.parametrize("args", [dict(T=1 << 30, N=1 << 30, fmt=2), dict(T=4, E=1024, N=1 << 30, fmt=4), dict(T=1 << 30, E=1024, N=1 << 24),
                                  dict(T=1, E=1024, N=1 << 20, K=1 << 14)])
def test_grouped_refuses_tiles_past_counting(args):
    assert call("qgemm_grouped_run", GROUPED, args) == UNSUP
    assert "tiles" in qg.qgemm_last_error()
