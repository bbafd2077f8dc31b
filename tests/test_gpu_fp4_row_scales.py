"""qgemm_fp4_dequant with row scales of any size (GPU): code * block scale * row scale in float32, rounded
to the output type. The product of the three is exact in float64; it must not be lost where code * block
scale alone passes float32's range and the row scale brings it back, nor where it is subnormal."""
import numpy as np
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests import _experts_ref as ref
from tests._util import ensure_built, torch_dtype

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("fmt", [3, 4])
def test_row_scales(fmt, dt, layout):
    B = ref.BLOCK[fmt]
    K = 256 * B
    g = np.random.default_rng(3).random(12).astype(np.float32) + np.float32(0.5)
    g = np.concatenate([g * np.float32(2.0 ** e) for e in (0, -20, 30, -126, 100)]
                       + [np.array([1.0, 0.0, -0.0, 1e-40, 3e38, 2.0 ** -120, 0.99999994, 0.25, np.inf, np.nan], np.float32), -g[:3]])
    M = len(g)
    codes = np.tile(np.arange(K) % 16, (M, 1)).astype(np.uint8)
    byte = np.tile(np.arange(256) % 128 if fmt == 4 else np.arange(256), (M, 1)).astype(np.uint8)     # every scale, NaN too
    y = torch.full((M, K), 7.0, dtype=torch_dtype(dt), device=DEV)
    sb = torch.from_numpy((ref.rows_layout if layout == 0 else ref.tiled_layout)(byte, K, fmt)).to(DEV)
    qg.qgemm_fp4_dequant(M, K, fmt, layout, torch.from_numpy(ref.pack(codes)).to(DEV), sb, torch.from_numpy(g).to(DEV), y, dt)
    with np.errstate(over="ignore", invalid="ignore"):
        want = torch.from_numpy(ref.values(codes, byte, g, fmt).astype(np.float32)).to(torch_dtype(dt)).double().numpy()
    got = y.double().cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True), f"{(got != want).sum() - np.isnan(want).sum()} of {got.size} differ"
    number = ~np.isnan(want)
    assert np.array_equal(np.signbit(got[number]), np.signbit(want[number]))
