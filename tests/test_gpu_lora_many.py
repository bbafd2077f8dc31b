"""Adapters over many rows (the tensor cores' asynchronous path): tiles that end anywhere, cut K and N, waits that run out."""
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests import _serve_ref as ref
from tests._util import ensure_built
from tests.test_gpu_lora import DEV, check, grouped, make, mixed, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("dtype,y_dtype", [(qg.F16, qg.F32), (qg.BF16, qg.BF16), (qg.BF16, qg.F32), (qg.F16, qg.BF16)])
@pytest.mark.parametrize("M,K,N,L,R", [
    (2304, 64, 1, 1, 8), (2500, 192, 129, 3, 16), (2305, 4096, 328, 2, 16), (1600, 448, 250, 40, 24), (1537, 1088, 64, 2, 32), (1300, 704, 191, 5, 40),
    (2400, 320, 520, 700, 64), (800, 960, 96, 3, 72), (4300, 128, 40, 64, 16), (2800, 192, 72, 40, 96),
    (20000, 64, 24, 300, 8), (1025, 2560, 264, 1, 128), (9000, 128, 72, 9, 128)])
def test_many_rows(M, K, N, L, R, dtype, y_dtype):
    check(make(M, K, N, L, R, dtype, y_dtype, mixed(M, L, M), seed=M + R, ragged=M % 100 == 0))


@pytest.mark.parametrize("dtype", [qg.F16, qg.BF16])
@pytest.mark.parametrize("y_dtype", [qg.F32, qg.BF16])
@pytest.mark.parametrize("M,K,N,L,R", [(1000, 320, 136, 3, 136), (900, 1024, 72, 2, 200), (1500, 512, 200, 4, 256), (256, 64, 33, 1, 256),
                                       (257, 2560, 264, 70, 144)])
def test_ranks_above_128(M, K, N, L, R, dtype, y_dtype):
    check(make(M, K, N, L, R, dtype, y_dtype, mixed(M, L, M), seed=M + R, ragged=True))
    check(make(M, K, N, L, R, dtype, y_dtype, mixed(M, L, M), seed=M + R + 1))


@pytest.mark.parametrize("pad_x,pad_y", [(0, 1), (8, 3), (64, 8), (0, 4)])
@pytest.mark.parametrize("y_dtype", [qg.F32, qg.BF16])
def test_strides(pad_x, pad_y, y_dtype):
    check(make(2310, 128, 201, 3, 16, qg.BF16, y_dtype, mixed(2310, 3), pad_x=pad_x, pad_y=pad_y, scaled=False))


@pytest.mark.parametrize("count", [1, 15, 127, 128, 129, 2303, 2304])
def test_tiles_that_end_anywhere(count):
    check(make(2304, 128, 72, 4, 16, qg.BF16, qg.BF16, [2] * count + [-1] * (2304 - count)))


def test_runs_and_scattered_rows_give_the_same():
    """A row's result depends on the row and its adapter, not on its neighbours in the tile."""
    M, L = 2560, 4
    c = make(M, 512, 136, L, 16, qg.BF16, qg.F32, [m // 640 for m in range(M)])
    before = c["Y"].clone()
    run(c)
    first = c["Y"].clone()
    order = torch.randperm(M, device=DEV)
    d = dict(c, adapter=[c["adapter"][i] for i in order.tolist()], X=c["X"][order].contiguous(), Y=before[order].contiguous())
    run(d)
    assert torch.equal(d["Y"], first[order])


def test_past_the_rank_nothing_is_used():
    c = make(1600, 192, 70, 6, 40, qg.BF16, qg.F32, [i % 6 for i in range(1600)])
    c["rank"] = [0, 1, 7, 18, 40, 99]
    for l, r in enumerate(c["rank"]):
        c["A"][l, r:] = float("nan")
        c["B"][l, :, r:] = float("nan")
    check(c)


def test_nan_stays_in_its_row_and_rows_outside_are_skipped():
    M, K, N = 2400, 128, 64
    c = make(M, K, N, 2, 16, qg.F16, qg.F32, [i % 2 for i in range(M)])
    c["X"][3, 5] = float("nan")
    before = c["Y"].clone()
    row, offsets = grouped(c["adapter"], 2)
    row[10], row[1300] = M + 5, -7           # skipped: rows 20 and (1300 - 1200) * 2 + 1 of the batch
    skipped = [20, 201]
    owner = [-1 if m in skipped else a for m, a in enumerate(c["adapter"])]
    qg.qgemm_lora_run(M, K, N, 2, 16, c["dtype"], row, offsets, c["X"], K, c["A"], c["B"], None, c["scale"], c["Y"], qg.F32, N)
    assert bool(torch.isnan(c["Y"][3]).all())
    c["X"][3] = 0
    want, allow = ref.lora(before, c["X"], c["A"], c["B"], owner, None, c["scale"])
    good = torch.tensor([m for m in range(M) if m != 3], device=DEV)
    ref.check(c["Y"][good], want[good], allow[good])


@pytest.mark.parametrize("factor", [2.0 ** 14, 2.0 ** -13])
def test_f16_middle_values_beyond_f16(factor):
    c = make(2400, 256, 64, 2, 16, qg.F16, qg.F32, [i % 2 for i in range(2400)])
    c["X"] = (c["X"].float().clamp(-2, 2) * factor).half()
    if factor > 1:
        c["A"] = (c["A"].float() * 64).half()
    else:
        c["Y"].zero_()
    check(c)


def test_two_at_once_and_in_a_graph():
    """Two batches on two streams at the same time, then both captured: the bits of one after the other."""
    cs = [make(2600, 1024, 520, 5, r, qg.BF16, qg.BF16, mixed(2600, 5, r), seed=r) for r in (16, 64)]
    before = [c["Y"].clone() for c in cs]
    plans = [run(c) for c in cs]
    want = [c["Y"].clone() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]

    def again(c, plan, stream):
        qg.qgemm_lora_run(c["M"], c["K"], c["N"], c["L"], c["R"], c["dtype"], *plan, c["X"], c["K"], c["A"], c["B"], None, c["scale"], c["Y"],
                          c["y_dtype"], c["N"], stream)

    for _ in range(3):
        for c, b in zip(cs, before):
            c["Y"].copy_(b)
        torch.cuda.synchronize()
        for c, p, s in zip(cs, plans, streams):
            again(c, p, s)
        torch.cuda.synchronize()
        for c, w in zip(cs, want):
            assert torch.equal(c["Y"], w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, p in zip(cs, plans):
            again(c, p, None)
    for c, b in zip(cs, before):
        c["Y"].copy_(b)
    graph.replay()
    for c, w in zip(cs, want):
        assert torch.equal(c["Y"], w)


@pytest.mark.parametrize("M,R", [(2304, 16), (1300, 64), (900, 128), (300, 256)])
def test_waits_that_run_out(M, R):
    """One wait runs out on purpose: the call returns, the status says so, and the next calls give their bits."""
    c = make(M, 512, 200, 3, R, qg.BF16, qg.BF16, mixed(M, 3))
    before = c["Y"].clone()
    plan = run(c)
    torch.cuda.synchronize()
    want = c["Y"].clone()
    limit, stall = qg.qgemm_set_option(qg.OPT_WAIT_LIMIT_US, 2000), qg.qgemm_set_option(qg.OPT_DEBUG_STALL, 1)
    try:
        c["Y"].copy_(before)
        qg.qgemm_lora_run(M, 512, 200, 3, R, qg.BF16, *plan, c["X"], 512, c["A"], c["B"], None, c["scale"], c["Y"], qg.BF16, 200)
        assert qg.qgemm_status() == -6
    finally:
        qg.qgemm_set_option(qg.OPT_WAIT_LIMIT_US, limit)
        qg.qgemm_set_option(qg.OPT_DEBUG_STALL, stall)
    assert qg.qgemm_status() == 0
    for _ in range(2):
        c["Y"].copy_(before)
        qg.qgemm_lora_run(M, 512, 200, 3, R, qg.BF16, *plan, c["X"], 512, c["A"], c["B"], None, c["scale"], c["Y"], qg.BF16, 200)
        assert qg.qgemm_status() == 0 and torch.equal(c["Y"], want)


@pytest.mark.parametrize("y_dtype", [qg.F32, qg.BF16])
@pytest.mark.parametrize("M,R", [(2560, 16), (1300, 64), (900, 128), (300, 256)])
@pytest.mark.parametrize("limit_us,stall", [(1, 0), (1, 1), (2000, 1)])
def test_waits_that_run_out_with_products_in_flight(M, R, y_dtype, limit_us, stall):
    """A bound so short that the waits run out while products are in flight, wherever that is; and the diagnostic wait behind
    the first products. The block's own shared and tensor memory is all that those touch, and the next calls give their
    bits."""
    c = make(M, 1024, 520, 3, R, qg.F16, y_dtype, mixed(M, 3))
    before = c["Y"].clone()
    plan = run(c)
    torch.cuda.synchronize()
    want = c["Y"].clone()

    def call():
        c["Y"].copy_(before)
        qg.qgemm_lora_run(M, 1024, 520, 3, R, qg.F16, *plan, c["X"], 1024, c["A"], c["B"], None, c["scale"], c["Y"], y_dtype, 520)

    prev = qg.qgemm_set_option(qg.OPT_WAIT_LIMIT_US, limit_us), qg.qgemm_set_option(qg.OPT_DEBUG_STALL, stall)
    try:
        for _ in range(3):
            call()
        status = qg.qgemm_status()
    finally:
        qg.qgemm_set_option(qg.OPT_WAIT_LIMIT_US, prev[0])
        qg.qgemm_set_option(qg.OPT_DEBUG_STALL, prev[1])
    assert status == -6 or (stall == 0 and status == 0)
    assert qg.qgemm_status() == 0
    for _ in range(2):
        call()
        assert qg.qgemm_status() == 0 and torch.equal(c["Y"], want)


# stages of 64 of K in each of 8 blocks: as many as the accumulators take without being emptied, one and some more, and several rounds
@pytest.mark.parametrize("M,R,stages", [(300, 256, (8, 9, 10, 16, 17, 25)), (900, 128, (16, 17, 20, 33)), (1300, 64, (16, 17, 33)), (1600, 32, (32, 33, 66)),
                                        (2304, 16, (64, 65, 130))])
@pytest.mark.parametrize("dtype,y_dtype", [(qg.F16, qg.F32), (qg.BF16, qg.BF16), (qg.BF16, qg.F32)])
def test_accumulators_that_are_emptied(M, R, stages, dtype, y_dtype):
    for n in stages:
        check(make(M, 64 * 8 * n, 40, 1, R, dtype, y_dtype, mixed(M, 1, n, none=0.02), seed=n, ragged=False))
