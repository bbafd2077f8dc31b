"""Every form of the product kernel against the float64 definition (GPU): tiles of 32 and 128 rows by one
block, K shared by a cluster of 2, 4 and 8 blocks, and pairs of blocks on tiles of 256 rows x 256
channels, in all four operand formats, dense and over ragged groups. Each test asserts the form that its
shape takes, so that a change of the rule cannot move it elsewhere unseen."""
import ctypes

import numpy as np
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests import _experts_ref as ref
from tests._util import ensure_built, torch_dtype
from tests.test_gpu_fp4 import check_out, gpu_quant, host, operands

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def plan(M, E, grouped, K, N, fmt):
    """Rows of a tile and blocks that share its K."""
    rows, split = ctypes.c_int(), ctypes.c_int()
    qg.load().qg_group_plan(M, E, int(grouped), K, N, fmt, ctypes.byref(rows), ctypes.byref(split))
    return rows.value, split.value


def group_operands(sizes, N, K, fmt, first, seed):
    """Operands of ragged groups that start at row `first`: (A, B, offsets, float64 A, B per expert, their scales)."""
    E, T = len(sizes), first + sum(sizes) + 2
    g = torch.Generator(device=DEV).manual_seed(seed)
    a, b = torch.randn(T, K, generator=g, device=DEV), torch.randn(E, N, K, generator=g, device=DEV) * 0.05
    offsets = torch.tensor(np.concatenate(([0], np.cumsum(sizes))) + first, dtype=torch.int32, device=DEV)
    if fmt < 3:
        a, b = a.to(torch_dtype(fmt)), b.to(torch_dtype(fmt))
        return (a, None, None), (b, None, None), offsets, host(a), host(b), None, [None] * E
    A, Q = gpu_quant(a, T, K, fmt), [gpu_quant(b[e], N, K, fmt, 1) for e in range(E)]
    B = [torch.cat([q[i] for q in Q]) if Q[0][i] is not None else None for i in range(3)]
    b64 = [ref.values(*ref.quantize(host(b[e]), fmt)[:2], None, fmt) for e in range(E)]
    return (A, B, offsets, ref.values(*ref.quantize(host(a), fmt)[:2], None, fmt), b64, None if A[2] is None else host(A[2]),
            [None if q[2] is None else host(q[2]) for q in Q])


def run_groups(sizes, N, K, fmt, dt, act, bias, form, first=3):
    E, T = len(sizes), first + sum(sizes) + 2
    assert plan(T, E, True, K, N, fmt) == form
    A, B, offsets, a64, b64, sa, sb = group_operands(sizes, N, K, fmt, first, N + K)
    bias_t = torch.randn(E, N, device=DEV) if bias else None
    C = torch.full((T, N // 2 if act == 4 else N), 5.0, dtype=torch_dtype(dt), device=DEV)
    call = lambda out: qg.qgemm_grouped_run(T, E, K, N, fmt, offsets, A[0], A[1], A[2], B[0], B[1], B[2], bias_t, act, out, dt)
    call(C)
    assert qg.qgemm_status() == 0
    assert torch.all(C[:first] == 5) and torch.all(C[T - 2 :] == 5)          # rows of no group
    at = first
    for e, n in enumerate(sizes):
        if n:
            check_out(C[at : at + n], *ref.product(a64[at : at + n], b64[e], None if sa is None else sa[at : at + n], sb[e],
                                                   None if bias_t is None else host(bias_t[e]), act, None), dt)
        at += n
    again = torch.full_like(C, 5.0)
    call(again)
    assert torch.equal(C, again)


# Several tiles a pair (the accumulators in turn), ragged last rows and channels, a last stage of one
# MMA, one row in the last tile, every epilogue.
@pytest.mark.parametrize("M,K,N,dt,act,bias,residual", [
    (513, 4096, 4000, 2, 0, True, True), (2048, 1024, 14336, 2, 2, True, False), (1100, 2112, 9001, 0, 0, True, False),
    (3000, 1216, 6002, 2, 4, True, True), (257, 4160, 8000, 1, 3, False, True), (2048, 1984, 5000, 0, 4, False, False),
    (530, 4096, 4002, 1, 1, True, False)])
@pytest.mark.parametrize("fmt", [3, 4])
def test_pairs(M, K, N, dt, act, bias, residual, fmt):
    dense(M, K, N, dt, act, bias, residual, fmt, (256, 1))


@pytest.mark.parametrize("M,K,N,dt,act,bias,residual,form", [
    (128, 9728, 2500, 2, 0, True, True, (128, 4)), (120, 9728, 1200, 0, 2, True, False, (128, 8)), (256, 9728, 601, 1, 0, False, True, (128, 8)),
    (256, 9728, 600, 2, 4, True, False, (128, 8)),
    (300, 4096, 4096, 2, 3, True, True, (128, 1)), (1100, 832, 5000, 1, 4, True, False, (128, 1)), (2047, 2560, 3002, 0, 0, True, True, (128, 1)),
    (5, 4096, 500, 2, 4, True, True, (32, 8)), (40, 8192, 300, 0, 1, True, False, (32, 8)), (100, 4096, 1001, 2, 0, False, True, (32, 4)),
    (129, 9728, 1250, 1, 2, True, False, (32, 2)), (1, 256, 24001, 2, 0, True, True, (32, 1))])
@pytest.mark.parametrize("fmt", [3, 4])
def test_single_blocks_and_clusters(M, K, N, dt, act, bias, residual, form, fmt):
    dense(M, K, N, dt, act, bias, residual, fmt, form)


def dense(M, K, N, dt, act, bias, residual, fmt, form):
    assert plan(M, 1, False, K, N, fmt) == form
    A, B, a64, b64 = operands(M, N, K, fmt, M + N + K)
    cols = N // 2 if act == 4 else N
    bias_t = torch.randn(N, device=DEV) if bias else None
    res = torch.randn(M, cols, device=DEV).to(torch_dtype(dt)) if residual else None
    # (the buffer has a row more than C, which must stay as it is)
    whole = torch.full((M + 1, cols), 5.0, dtype=torch_dtype(dt), device=DEV)
    C = whole[:M]
    call = lambda out: qg.qgemm_fp4_run(M, K, N, fmt, A[0], A[1], A[2], B[0], B[1], B[2], bias_t, act, res, out, dt)
    call(C)
    assert qg.qgemm_status() == 0
    check_out(C, *ref.product(a64, b64, None if A[2] is None else host(A[2]), None if B[2] is None else host(B[2]),
                              None if bias_t is None else host(bias_t), act, None if res is None else host(res)), dt)
    assert torch.all(whole[M] == 5)
    again = torch.empty_like(C)
    call(again)
    assert torch.equal(C, again)
    if residual:
        call(res)
        assert torch.equal(C, res)          # in place


UNEVEN = [0, 700, 1, 257, 33, 511]
MORE = [900, 0, 300, 1, 2000, 256, 17]


@pytest.mark.parametrize("sizes,K,N,dt,act,bias", [
    (UNEVEN, 4096, 1300, 2, 0, True), (UNEVEN, 1600, 7000, 0, 4, False), (MORE, 2048, 2570, 2, 4, True), (MORE, 4160, 4001, 1, 2, True),
    ([300, 0, 0, 212], 4160, 4000, 2, 1, False)])
@pytest.mark.parametrize("fmt", [1, 2, 3, 4])
def test_grouped_pairs(sizes, K, N, dt, act, bias, fmt):
    run_groups(sizes, N, K, fmt, dt, act, bias, (256, 1))


@pytest.mark.parametrize("sizes,K,N,dt,act,bias,form", [
    (UNEVEN, 832, 2570, 2, 4, True, (128, 1)), (MORE, 8192, 381, 0, 0, True, (128, 1)), ([128, 0, 120], 2560, 5120, 2, 2, False, (128, 1)),
    (UNEVEN, 9728, 250, 2, 4, True, (128, 4)), (MORE, 9728, 249, 0, 0, True, (128, 2)), ([256], 9728, 600, 1, 3, True, (128, 8)),
    ([300, 0, 0, 212], 9728, 250, 2, 0, False, (128, 8)),
    ([128, 0, 120], 9728, 250, 2, 4, True, (32, 4)), ([256], 9728, 250, 0, 1, False, (32, 8)), ([128, 0, 120], 1600, 7000, 2, 0, True, (32, 1))])
@pytest.mark.parametrize("fmt", [1, 2, 3, 4])
def test_grouped_single_blocks_and_clusters(sizes, K, N, dt, act, bias, form, fmt):
    run_groups(sizes, N, K, fmt, dt, act, bias, form)
