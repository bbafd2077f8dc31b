"""Adapters on values at the edges: infinities, the ranges of the middle values H = A x, and how many of their bits count. Each
case runs on the kernel for few rows and on the one for many."""
import math

import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests._util import ensure_built
from tests.test_gpu_lora import DEV, make, run

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


ROWS = [24, 2400]           # few rows, many rows (300 and more where the rank is above 128)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("dtype,y_dtype", [(qg.F16, qg.F32), (qg.BF16, qg.F32), (qg.F16, qg.F16), (qg.BF16, qg.BF16)])
@pytest.mark.parametrize("R,ranks", [(8, [1, 8]), (24, [3, 17]), (40, [9, 33]), (72, [16, 65]), (136, [7, 129])])
def test_an_infinite_input_gives_infinity_at_every_rank(R, ranks, dtype, y_dtype, M):
    """All values of A and B above 0: with an infinite x every H, and so every y, is that infinity. What pads a rank must not
    make it a NaN (0 * inf)."""
    c = make(M, 128, 70, 2, R, dtype, y_dtype, [i % 2 for i in range(M)])
    c["rank"] = ranks
    c["A"], c["B"] = c["A"].abs() + 0.125, c["B"].abs() + 0.125
    before = c["Y"].clone()
    c["X"][2, 5], c["X"][3, 5], c["X"][M - 1, 100] = INF, -INF, INF
    run(c)
    assert bool((c["Y"][2] == INF).all()) and bool((c["Y"][3] == -INF).all()) and bool((c["Y"][M - 1] == INF).all())
    others = torch.tensor([m for m in range(M) if m not in (2, 3, M - 1)], device=DEV)
    assert bool(torch.isfinite(c["Y"][others]).all()) and bool((c["Y"][others] != before[others]).any())


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("dtype", [qg.F16, qg.BF16])
def test_an_infinite_middle_value_beside_a_large_one(M, dtype):
    """H = (inf, 2^18), B = (1, -1): the sum is inf, though 2^18 is beyond f16."""
    c = make(M, 128, 40, 1, 16, dtype, qg.F32, [0] * M, scaled=False)
    c["X"].fill_(1.0)
    c["A"].zero_()
    c["A"][0, 0, 3] = INF
    c["A"][0, 1].fill_(2048.0)
    c["B"].zero_()
    c["B"][0, :, 0], c["B"][0, :, 1] = 1.0, -1.0
    c["rank"] = [2]
    run(c)
    assert bool((c["Y"] == INF).all())


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("down", [4, 14, 20, 26, 30])
@pytest.mark.parametrize("large", [2.0 ** -14, 1.0, 32768.0])
def test_a_small_middle_value_beside_a_large_one(M, down, large):
    """f16, H = (h, h 2^-down (1 + ...)) and B = (0, 1): y is the small one. It is off by 2^-23 of itself or 2^-39 of the large one at most
    (half a step of the smallest f16, where the largest value is scaled to 2^14 at least), and by float32's two roundings."""
    c = make(M, 128, 40, 1, 16, qg.F16, qg.F32, [0] * M, scaled=False)
    c["Y"].zero_(), c["X"].zero_(), c["A"].zero_(), c["B"].zero_()
    c["X"][:, 0], c["X"][:, 1] = large, 2.0 ** (-down // 2)
    c["X"][:, 1] *= large
    small = torch.linspace(1.0, 1.999, M, device=DEV).half()                        # 11 bits, times 11 bits: H has 22
    c["X"][:, 1] *= small
    c["A"][0, 0, 0], c["A"][0, 1, 1] = 1.0, 1.4990234375 * 2.0 ** (-down - (-down // 2))
    c["B"][0, :, 1] = 1.0
    c["rank"] = [2]
    want = c["X"][:, 1].double() * float(c["A"][0, 1, 1])
    run(c)
    off = (c["Y"].double() - want[:, None]).abs()
    allow = want * (2.0 ** -23 + 2.0 ** -23) + 2.0 ** -39 * large
    assert bool((off <= allow[:, None]).all()), float((off / allow[:, None]).max())


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("dtype", [qg.F16, qg.BF16])
def test_a_float32_result_has_float32_bits_of_the_middle_values(M, dtype):
    """H = 1 + 2^-6 + 2^-12 + 2^-18 + 2^-21 exactly and B = 1: a float32 y has all of it but the last rounding (f16: within 2^-23 of
    H), which two terms of bf16 miss by 2^-21."""
    c = make(M, 128, 40, 1, 16, dtype, qg.F32, [0] * M, scaled=False)
    c["Y"].zero_(), c["X"].zero_(), c["A"].zero_(), c["B"].zero_()
    bits = [0, -6, -12, -18, -21]
    for i, e in enumerate(bits):
        c["X"][:, 16 * i] = 2.0 ** (e // 2)
        c["A"][0, 0, 16 * i] = 2.0 ** (e - e // 2)
    c["B"][0, :, 0] = 1.0
    c["rank"] = [1]
    want = sum(2.0 ** e for e in bits)
    run(c)
    assert float((c["Y"].double() - want).abs().max()) <= want * 2.0 ** -23


@pytest.mark.parametrize("dtype", [qg.F16, qg.BF16])
@pytest.mark.parametrize("M,K,R", [(19600, 16384, 64), (9800, 16384, 128), (9800, 8192, 256), (1000, 65536, 128), (2400, 131072, 16)])
def test_long_sums_are_float32_sums(M, K, R, dtype):
    """Values above 0, so that nothing cancels and every cut-off adds up. The tensor cores cut a running sum off by 2 u of it at most; the
    first product's chains are 16 steps long (32 u of the whole), added up in float32 (a rounding for each chain of an
    accumulator, each accumulator, and each of 8 blocks), the second one's have a step for 16 ranks; the terms of H
    hold 2^-23 = 2 u of it, the smaller ones' products are 2^-8 of the whole or less and add 1 u, and the last sum rounds once."""
    if dtype == qg.BF16 and R > 128:
        pytest.skip("takes the kernel for few rows")
    N = 40
    g = torch.Generator(device=DEV).manual_seed(M + R)
    dt = torch.float16 if dtype == qg.F16 else torch.bfloat16
    X = torch.rand(M, K, generator=g, device=DEV, dtype=torch.float32).to(dt)
    A = (torch.rand(1, R, K, generator=g, device=DEV) * 0.01).to(dt)
    B = torch.rand(1, N, R, generator=g, device=DEV).to(dt)
    Y = torch.zeros(M, N, device=DEV)
    row = torch.arange(M, dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    qg.qgemm_lora_run(M, K, N, 1, R, dtype, row, offsets, X, K, A, B, None, None, Y, qg.F32, N)
    u = 2.0 ** -24
    rp = max(16, 1 << (R - 1).bit_length())
    sums = (256 if rp <= 64 else 512) // rp
    bound = u * (32 + -(-K // 64 // (4 * sums)) + sums + 8 + 2 * R / 16 + 2 + 1 + 2)
    for rows in torch.arange(M, device=DEV).split(1024):
        want = (X[rows].double() @ A[0].double().T) @ B[0].double().T
        off = float(((Y[rows].double() - want).abs() / want).max())
        assert off <= bound, (off / u, bound / u)


@pytest.mark.parametrize("dtype", [qg.F16, qg.BF16])
@pytest.mark.parametrize("M,K,R,L", [(2000, 65536, 16, 1), (2000, 32768, 32, 100), (1200, 65536, 64, 1), (700, 65536, 128, 40), (240, 65536, 256, 40), (9, 131072, 16, 1)])
def test_long_sums_of_few_rows_are_float32_sums(M, K, R, L, dtype):
    """The same for the kernel for few rows: chains of 16 or 32 steps in the first product, a rounding for each of them and each of 8
    warps and 8 blocks; 3 steps for 16 ranks in the second, 128 ranks at a time."""
    N = 40
    g = torch.Generator(device=DEV).manual_seed(M + R)
    dt = torch.float16 if dtype == qg.F16 else torch.bfloat16
    X = torch.rand(M, K, generator=g, device=DEV).to(dt)
    A = (torch.rand(L, R, K, generator=g, device=DEV) * 0.01).to(dt)
    B = torch.rand(L, N, R, generator=g, device=DEV).to(dt)
    Y = torch.zeros(M, N, device=DEV)
    row = torch.arange(M, dtype=torch.int32, device=DEV)
    at = [M * l // L for l in range(L + 1)]
    qg.qgemm_lora_run(M, K, N, L, R, dtype, row, torch.tensor(at, dtype=torch.int32, device=DEV), X, K, A, B, None, None, Y, qg.F32, N)
    u, chain = 2.0 ** -24, 16 if R <= 32 else 32
    bound = u * (2 * chain + -(-K // 8 // 16 // chain) + 16 + 2 * 3 * min(R / 16, 8) + 2 + 2 + 1)
    for l in range(L):
        x = X[at[l]: at[l + 1]].double()
        want = (x @ A[l].double().T) @ B[l].double().T
        off = float(((Y[at[l]: at[l + 1]].double() - want).abs() / want).max())
        assert off <= bound, (off / u, bound / u)
