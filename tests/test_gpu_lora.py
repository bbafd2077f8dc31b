"""Adapters: the order of rows by adapter against its definition, the products against float64."""
import random

import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests import _serve_ref as ref
from tests._util import ensure_built, torch_dtype

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def grouped(adapter, L):
    ids = torch.tensor(adapter, dtype=torch.int32, device=DEV)
    row, offsets = torch.full((max(len(adapter), 1),), 77, dtype=torch.int32, device=DEV), torch.full((L + 1,), 77, dtype=torch.int32, device=DEV)
    qg.qgemm_lora_group(len(adapter), L, ids, row, offsets)
    return row[: len(adapter)], offsets


@pytest.mark.parametrize("M,L,kind", [
    (0, 1, "any"), (1, 1, "any"), (1, 1024, "any"), (3, 2, "none"), (64, 32, "any"), (127, 7, "outside"), (128, 1, "one"), (129, 5, "last"),
    (1000, 1000, "any"), (4095, 3, "any"), (4097, 3, "outside"), (5000, 1024, "any"), (9001, 40, "runs")])
def test_group(M, L, kind):
    r = random.Random(M + L)
    adapter = {"any": lambda: [r.randrange(L) for _ in range(M)], "none": lambda: [-1] * M, "one": lambda: [0] * M, "last": lambda: [L - 1] * M,
               "outside": lambda: [r.choice((-5, -1, L, (1 << 31) - 1, -(1 << 31), r.randrange(L))) for _ in range(M)],
               "runs": lambda: [(i // 300) % L for i in range(M)]}[kind]()
    row, offsets = grouped(adapter, L)
    want_row, want_offsets = ref.group(adapter, L)
    assert row.tolist() == want_row and offsets.tolist() == want_offsets


def make(M, K, N, L, R, dtype, y_dtype, adapter, seed=0, ragged=False, pad_x=0, pad_y=0, scaled=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = torch_dtype(dtype)
    X = torch.randn(M, K + pad_x, generator=g, device=DEV).to(dt)
    A = (torch.randn(L, R, K, generator=g, device=DEV) * K ** -0.5).to(dt)
    B = (torch.randn(L, N, R, generator=g, device=DEV) * 0.2).to(dt)
    Y = torch.randn(M, N + pad_y, generator=g, device=DEV).to(torch_dtype(y_dtype))
    rank = [int(v) for v in torch.randint(0, R + 1, (L,), generator=torch.Generator().manual_seed(seed))] if ragged else None
    scale = (0.5 + torch.rand(L, generator=g, device=DEV)) if scaled else None
    return dict(M=M, K=K, N=N, L=L, R=R, dtype=dtype, y_dtype=y_dtype, adapter=adapter, X=X, A=A, B=B, Y=Y, rank=rank, scale=scale)


def run(c, stream=None):
    row, offsets = grouped(c["adapter"], c["L"])
    rank = torch.tensor(c["rank"], dtype=torch.int32, device=DEV) if c["rank"] is not None else None
    qg.qgemm_lora_run(c["M"], c["K"], c["N"], c["L"], c["R"], c["dtype"], row, offsets, c["X"], c["X"].shape[1], c["A"], c["B"], rank, c["scale"],
                      c["Y"], c["y_dtype"], c["Y"].shape[1], stream)
    return row, offsets


def check(c):
    before = c["Y"].clone()
    want, allow = ref.lora(before[:, : c["N"]], c["X"][:, : c["K"]], c["A"], c["B"], c["adapter"], c["rank"], c["scale"])
    run(c)
    torch.cuda.synchronize()
    ref.check(c["Y"][:, : c["N"]], want, allow)
    assert torch.equal(c["Y"][:, c["N"]:], before[:, c["N"]:])                # the rest of a joined projection
    free = torch.tensor([not 0 <= i < c["L"] for i in c["adapter"]], device=DEV)
    assert torch.equal(c["Y"][free], before[free])                            # rows without an adapter


def mixed(M, L, seed=0, none=0.1):
    r = random.Random(seed)
    return [-1 if r.random() < none else r.randrange(L) for _ in range(M)]


@pytest.mark.parametrize("dtype", [qg.F16, qg.BF16])
@pytest.mark.parametrize("y_dtype", [qg.F32, qg.F16, qg.BF16])
@pytest.mark.parametrize("M,K,N,L,R", [(1, 64, 1, 1, 8), (1, 4096, 4096, 3, 16), (5, 128, 33, 2, 24), (17, 320, 100, 1, 32), (40, 576, 520, 7, 64),
                                       (33, 1024, 264, 2, 72), (20, 256, 96, 3, 128), (18, 192, 40, 2, 256)])
def test_few_rows(M, K, N, L, R, dtype, y_dtype):
    check(make(M, K, N, L, R, dtype, y_dtype, mixed(M, L, M), seed=M + R, ragged=R in (24, 72, 256)))


@pytest.mark.parametrize("dtype,y_dtype", [(qg.F16, qg.F32), (qg.BF16, qg.BF16), (qg.BF16, qg.F32), (qg.F16, qg.F16)])
@pytest.mark.parametrize("M,K,N,L,R", [(1024, 128, 96, 3, 16), (1100, 256, 250, 40, 32), (1500, 192, 128, 5, 64), (1030, 128, 72, 2, 128),
                                       (1025, 64, 64, 1000, 8), (1040, 128, 40, 3, 256)])
def test_many_rows(M, K, N, L, R, dtype, y_dtype):
    check(make(M, K, N, L, R, dtype, y_dtype, mixed(M, L, M), seed=M + R, ragged=M % 4 == 0))


@pytest.mark.parametrize("pad_x,pad_y", [(0, 1), (8, 3), (64, 8), (0, 4)])
@pytest.mark.parametrize("M,y_dtype", [(19, qg.BF16), (19, qg.F32), (1030, qg.F16)])
def test_strides(M, y_dtype, pad_x, pad_y):
    check(make(M, 128, 71, 3, 16, qg.BF16 if y_dtype != qg.F16 else qg.F16, y_dtype, mixed(M, 3), pad_x=pad_x, pad_y=pad_y, scaled=False))


@pytest.mark.parametrize("M", [16, 17, 64, 65, 1087, 1088, 1089])
def test_one_adapter_has_all_rows(M):
    check(make(M, 128, 64, 5, 16, qg.BF16, qg.BF16, [3] * M))


def test_no_row_has_an_adapter():
    check(make(30, 128, 64, 5, 16, qg.BF16, qg.BF16, [-1, 5] * 15))


def test_past_the_rank_nothing_is_used():
    """NaN in the unused rows of A and columns of B, ranks that are no multiple of anything, and ranks out of range."""
    c = make(24, 192, 70, 6, 40, qg.BF16, qg.F32, [i % 6 for i in range(24)])
    c["rank"] = [0, 1, 7, 18, 40, 99]
    for l, r in enumerate(c["rank"]):
        c["A"][l, r:] = float("nan")
        c["B"][l, :, r:] = float("nan")
    check(c)
    c["rank"][0] = -3
    check(c)


def test_nan_and_infinity_stay_in_their_rows():
    c = make(12, 128, 64, 2, 16, qg.F16, qg.F32, [i % 2 for i in range(12)])
    c["X"][3, 5], c["X"][8, 100] = float("nan"), float("inf")
    before = c["Y"].clone()
    run(c)
    bad = torch.tensor([3, 8], device=DEV)
    assert bool(torch.isnan(c["Y"][3]).all()) and not bool(torch.isfinite(c["Y"][8]).any())
    good = torch.tensor([m for m in range(12) if m not in (3, 8)], device=DEV)
    c["X"][bad] = 0
    want, allow = ref.lora(before, c["X"], c["A"], c["B"], c["adapter"], None, c["scale"])
    ref.check(c["Y"][good], want[good], allow[good])


@pytest.mark.parametrize("factor", [2.0 ** 14, 2.0 ** -13])
def test_f16_middle_values_beyond_f16(factor):
    """H = A x of 2^17 and more, and of 2^-26 and less: the result stays a float32 sum."""
    c = make(20, 256, 64, 2, 16, qg.F16, qg.F32, [i % 2 for i in range(20)])
    c["X"] = (c["X"].float().clamp(-2, 2) * factor).half()
    if factor > 1:
        c["A"] = (c["A"].float() * 64).half()
    else:
        c["Y"].zero_()
    check(c)


def test_offsets_that_are_not_in_order():
    """Offsets are held to [0, M] and to the largest before them; entries of row outside the batch are skipped."""
    M, K, N, L, R = 20, 128, 64, 5, 16
    c = make(M, K, N, L, R, qg.BF16, qg.F32, [0] * M)
    row = torch.tensor([3, -1, 5, 99, 7, 0, 1, 2, 4, 6] + [8] * 10, dtype=torch.int32, device=DEV)
    offsets = torch.tensor([-4, 3, 1, 5, 5, 9], dtype=torch.int32, device=DEV)     # adapters 0: 0-2, 2: 3-4, 4: 5-8
    owner = [-1] * M
    for i, m in enumerate(row.tolist()[:9]):
        if 0 <= m < M:
            owner[m] = 0 if i < 3 else (2 if i < 5 else 4)
    want, allow = ref.lora(c["Y"], c["X"], c["A"], c["B"], owner, None, c["scale"])
    qg.qgemm_lora_run(M, K, N, L, R, c["dtype"], row, offsets, c["X"], K, c["A"], c["B"], None, c["scale"], c["Y"], qg.F32, N)
    ref.check(c["Y"], want, allow)


@pytest.mark.parametrize("M,L,none", [(1, 1024, 0.0), (40, 33, 0.2), (200, 255, 0.0), (300, 256, 0.5), (333, 257, 0.1), (700, 513, 0.0), (500, 1000, 0.3),
                                      (1100, 1024, 0.0), (2400, 1000, 0.1)])
def test_many_adapters(M, L, none):
    check(make(M, 128, 40, L, 16, qg.BF16, qg.F32, mixed(M, L, M, none=none), seed=L))


@pytest.mark.parametrize("L", [31, 90, 256, 600, 1024])
@pytest.mark.parametrize("M", [57, 2500])
def test_many_offsets_that_are_not_in_order(M, L):
    r = random.Random(L + M)
    c = make(M, 64, 24, L, 16, qg.BF16, qg.F32, [0] * M)
    given = sorted(r.randrange(M + 1) for _ in range(L + 1))
    for _ in range(L // 3):
        given[r.randrange(L + 1)] = r.choice((-9, -(1 << 31), 0, r.randrange(M + 1)))
    owner, row = [-1] * M, list(range(M))
    r.shuffle(row)
    held = min(max(given[0], 0), M)
    for l in range(L):
        end = max(min(max(given[l + 1], 0), M), held)
        for i in range(held, end):
            owner[row[i]] = l
        held = end
    want, allow = ref.lora(c["Y"], c["X"], c["A"], c["B"], owner, None, c["scale"])
    to = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    qg.qgemm_lora_run(M, 64, 24, L, 16, c["dtype"], to(row), to(given), c["X"], 64, c["A"], c["B"], None, c["scale"], c["Y"], qg.F32, 24)
    ref.check(c["Y"], want, allow)


def test_same_bits_every_time_and_on_another_stream():
    c = make(77, 1024, 333, 6, 64, qg.BF16, qg.F32, mixed(77, 6))
    before = c["Y"].clone()
    run(c)
    first = c["Y"].clone()
    side = torch.cuda.Stream()
    for _ in range(3):
        c["Y"].copy_(before)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(c)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(c["Y"], first)


def test_captured_with_its_order():
    """The order and the products in one graph, replayed with other adapters."""
    M, L = 50, 9
    c = make(M, 256, 128, L, 16, qg.BF16, qg.BF16, mixed(M, L))
    ids = torch.tensor(c["adapter"], dtype=torch.int32, device=DEV)
    row, offsets = torch.empty(M, dtype=torch.int32, device=DEV), torch.empty(L + 1, dtype=torch.int32, device=DEV)

    def step():
        qg.qgemm_lora_group(M, L, ids, row, offsets)
        qg.qgemm_lora_run(M, 256, 128, L, 16, qg.BF16, row, offsets, c["X"], 256, c["A"], c["B"], None, c["scale"], c["Y"], qg.BF16, 128)

    before = c["Y"].clone()
    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        adapter = mixed(M, L, seed, none=0.4)
        ids.copy_(torch.tensor(adapter, dtype=torch.int32))
        c["Y"].copy_(before)
        graph.replay()
        want, allow = ref.lora(before, c["X"], c["A"], c["B"], adapter, None, c["scale"])
        ref.check(c["Y"], want, allow)


def test_offsets_past_32_bits():
    """X and Y whose last rows start beyond 2^32 bytes."""
    M, K, N, ld = 33, 128, 64, 1 << 26
    X = torch.empty(M * ld, dtype=torch.bfloat16, device=DEV).view(M, ld)
    Y = torch.empty(M * ld, dtype=torch.bfloat16, device=DEV).view(M, ld)
    c = make(M, K, N, 2, 16, qg.BF16, qg.BF16, mixed(M, 2))
    X[:, :K], Y[:, :N] = c["X"], c["Y"]
    c["X"], small = X, c["Y"]
    row, offsets = grouped(c["adapter"], 2)
    want, allow = ref.lora(small, X[:, :K], c["A"], c["B"], c["adapter"], None, c["scale"])
    qg.qgemm_lora_run(M, K, N, 2, 16, qg.BF16, row, offsets, X, ld, c["A"], c["B"], None, c["scale"], Y, qg.BF16, ld)
    ref.check(Y[:, :N], want, allow)
