"""Mixture-of-experts operators on the GPU: routing (bit for bit in its whole numbers), the grouped
product over ragged groups and the weighted combination, against _experts_ref.py in float64."""
import numpy as np
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests import _experts_ref as ref
from tests._util import ensure_built, half_ulp, torch_dtype
from tests.test_gpu_fp4 import check_out, gpu_quant, host

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


# ---------------------------------------------------------------- routing
def gpu_route(x, k, renorm):
    T, E = x.shape
    dt = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[x.dtype]
    out = [torch.full((T, k), -9, dtype=torch.int32, device=DEV), torch.full((T, k), -9.0, device=DEV),
           torch.full((T, k), -9, dtype=torch.int32, device=DEV), torch.full((T * k,), -9, dtype=torch.int32, device=DEV),
           torch.full((E + 1,), -9, dtype=torch.int32, device=DEV)]
    wsb = qg.qgemm_moe_route_workspace_bytes(T, E, k)
    ws = torch.full((max(wsb, 16),), 0xEE, dtype=torch.uint8, device=DEV)
    qg.qgemm_moe_route(T, E, k, x, dt, x.stride(0), renorm, *out, ws, wsb)
    return out


def check_route(x, k, renorm):
    got = gpu_route(x, k, renorm)
    want = ref.route(host(x), k, renorm)
    for n, g, w in zip(("expert", "weight", "slot", "row", "offsets"), got, want):
        if n == "weight":
            # float32 exp, a sum of at most E terms and a quotient: E + 8 roundings of 2^-23 at the most
            assert np.all(np.abs(host(g) - w) <= (x.shape[1] + 8) * 2.0 ** -23 * w + 1e-38), n
        else:
            assert np.array_equal(g.cpu().numpy(), w), n


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("T,E,k,dt", [(1, 8, 2, 2), (1, 1, 1, 0), (8, 64, 8, 2), (33, 60, 4, 1), (128, 128, 8, 0), (129, 16, 1, 2),
                                      (700, 256, 8, 0), (2500, 33, 6, 2), (5, 1024, 32, 0), (32, 1023, 32, 2), (20000, 64, 30, 2), (300, 1024, 32, 0), (5000, 8, 8, 1), (64, 1000, 32, 2)])
def test_route(T, E, k, dt, renorm):
    g = torch.Generator(device=DEV).manual_seed(T + E + k)
    x = torch.randn(T, E, generator=g, device=DEV).to(torch_dtype(dt))
    check_route(x, k, renorm)


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("T", [20, 500])
def test_route_ties_masks_and_strides(T, renorm):
    """Equal logits (also -0 and 0), experts masked for all, rows with fewer than k experts left or
    none, NaN, the lowest finite value, infinities; rows further apart than E."""
    E, k = 40, 6
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randint(-2, 3, (T, E + 9), generator=g, device=DEV).float()
    x[::2] *= -0.0
    x[:, 3] = x[:, 17] = float("-inf")
    x[1] = float("-inf")
    x[2, 4:] = float("-inf")
    x[4, 5] = float("nan")
    x[5] = float("nan")
    x[6, :20] = float("-inf")
    x[7] = torch.finfo(torch.float32).min
    x[8, 11] = x[8, 30] = float("inf")
    x[9] = float("inf")
    x[10, 2:] = torch.finfo(torch.float32).min
    check_route(x[:, :E], k, renorm)


def test_route_all_to_one_and_none():
    x = torch.full((400, 12), -5.0, device=DEV)
    x[:, 7] = 1.0
    check_route(x, 1, 1)
    check_route(torch.full((400, 12), float("-inf"), device=DEV), 3, 0)
    check_route(torch.full((3, 12), float("nan"), device=DEV), 3, 1)


def test_route_no_tokens():
    off = torch.full((9,), -9, dtype=torch.int32, device=DEV)
    qg.qgemm_moe_route(0, 8, 2, None, 0, 8, 0, None, None, None, None, off)
    assert torch.all(off == 0)


# ---------------------------------------------------------------- grouped product
GROUPS = {
    "one row": [1],
    "one each": [1] * 20,
    "ragged": [0, 5, 0, 0, 130, 1, 300, 0],
    "decode": [2, 0, 1, 3, 17, 0, 16, 1, 0, 33],
    "all empty": [0] * 6,
    "last only": [0, 0, 0, 257],
    "many experts": [(i * 7) % 5 for i in range(200)],
    "tile edges": [128, 64, 256, 32, 127, 129, 255, 31],
}


@pytest.mark.parametrize("fmt", [1, 2, 3, 4])
@pytest.mark.parametrize("name,N,K,dt,act,bias", [
    ("one row", 128, 64, 0, 0, False), ("one row", 2560, 1024, 2, 4, True), ("one each", 136, 320, 2, 0, True),
    ("ragged", 200, 192, 0, 2, True), ("ragged", 512, 1024, 2, 4, False), ("decode", 330, 448, 1, 4, True),
    ("decode", 513, 2560, 0, 0, True), ("all empty", 128, 128, 2, 0, False), ("last only", 130, 576, 1, 3, True),
    ("many experts", 96, 256, 2, 1, True), ("tile edges", 384, 512, 0, 0, False), ("tile edges", 254, 768, 2, 4, True)])
def test_grouped(name, N, K, dt, act, bias, fmt):
    sizes = GROUPS[name]
    E, used = len(sizes), sum(sizes)
    first, T = 3, 3 + used + 2                          # rows before and after the groups
    offsets = torch.tensor(np.concatenate(([0], np.cumsum(sizes))) + first, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(N + K + E)
    a = torch.randn(T, K, generator=g, device=DEV)
    b = torch.randn(E, N, K, generator=g, device=DEV) * 0.05
    if fmt >= 3:
        A = gpu_quant(a, T, K, fmt)
        Bs = [gpu_quant(b[e], N, K, fmt, 1) for e in range(E)]
        B = [torch.cat([t[i] for t in Bs]) if Bs[0][i] is not None else None for i in range(3)]
        a64 = ref.values(*ref.quantize(host(a), fmt)[:2], None, fmt)
        b64 = [ref.values(*ref.quantize(host(b[e]), fmt)[:2], None, fmt) for e in range(E)]
        sa = None if A[2] is None else host(A[2])
        sb = None if B[2] is None else host(B[2]).reshape(E, N)
    else:
        A, B = [a.to(torch_dtype(fmt)), None, None], [b.to(torch_dtype(fmt)), None, None]
        a64, b64, sa, sb = host(A[0]), host(B[0]), None, None
    bias_t = torch.randn(E, N, generator=g, device=DEV) if bias else None
    cols = N // 2 if act == 4 else N
    C = torch.full((T, cols), 5.0, dtype=torch_dtype(dt), device=DEV)
    qg.qgemm_grouped_run(T, E, K, N, fmt, offsets, A[0], A[1], A[2], B[0], B[1], B[2], bias_t, act, C, dt)
    assert qg.qgemm_status() == 0
    assert torch.all(C[:first] == 5) and torch.all(C[first + used:] == 5)      # rows of no group
    at = first
    for e, n in enumerate(sizes):
        if n:
            R, err = ref.product(a64[at : at + n], b64[e], None if sa is None else sa[at : at + n], None if sb is None else sb[e],
                                 None if bias_t is None else host(bias_t[e]), act, None)
            check_out(C[at : at + n], R, err, dt)
        at += n
    again = torch.full_like(C, 5.0)
    qg.qgemm_grouped_run(T, E, K, N, fmt, offsets, A[0], A[1], A[2], B[0], B[1], B[2], bias_t, act, again, dt)
    assert torch.equal(C, again)


def test_grouped_offsets_out_of_range():
    """Offsets past the rows, negative or decreasing never reach outside A and C."""
    T, E, K, N = 70, 5, 128, 130
    a = torch.randn(T, K, device=DEV).bfloat16()
    b = torch.randn(E, N, K, device=DEV).bfloat16()
    guard = torch.full((T + 4, N), 5.0, device=DEV)
    for off in ([0, 30, 200, 1 << 30, 1 << 30, 1 << 30], [-50, -3, 10, 10, 40, 70], [70, 20, 5, 5, 5, 0]):
        C = guard[2:-2]
        C.fill_(5.0)
        qg.qgemm_grouped_run(T, E, K, N, 2, torch.tensor(off, dtype=torch.int32, device=DEV), a, None, None, b, None, None,
                             None, 0, C, 0)
        assert qg.qgemm_status() == 0
        assert torch.all(guard[:2] == 5) and torch.all(guard[-2:] == 5)
        want = torch.full((T, N), 5.0)
        for e in range(E):
            lo = min(max(off[e], 0), T)
            hi = min(max(off[e + 1], lo), T)
            want[lo:hi] = (a[lo:hi].float() @ b[e].float().T).cpu()
        assert torch.allclose(C.cpu(), want, rtol=1e-3, atol=1e-3)


@pytest.mark.parametrize("fmt", [2, 3])
def test_grouped_weights_past_32_bits(fmt):
    """Experts whose weights lie more than 2^32 bytes (and 2^31 values) into the array."""
    E, N, K = (300, 2048, 4096) if fmt == 2 else (300, 4096, 8192)
    T, per = 6, 2
    last = [0, 254, 299]
    b = torch.randint(0, 256, (E, N, K // 2 if fmt == 3 else 2 * K), dtype=torch.uint8, device=DEV)
    sizes = torch.zeros(E, dtype=torch.int64)
    sizes[last] = per
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64), sizes.cumsum(0))).to(torch.int32).to(DEV)
    if fmt == 3:
        a, a_s, _ = gpu_quant(torch.randn(T, K, device=DEV), T, K, 3)
        one = qg.qgemm_fp4_scales_bytes(N, K, 3, 1)
        b_s = torch.randint(118, 122, (E * one,), dtype=torch.uint8, device=DEV)
    else:
        b = b.view(torch.int16).bitwise_and_(0x3FFF).view(torch.bfloat16)      # finite, below 2
        a, a_s, b_s = torch.randn(T, K, device=DEV).bfloat16(), None, None
    C = torch.zeros(T, N, device=DEV)
    qg.qgemm_grouped_run(T, E, K, N, fmt, offsets, a, a_s, None, b, b_s, None, None, 0, C, 0)
    assert qg.qgemm_status() == 0
    for i, e in enumerate(last):
        rows = slice(per * i, per * (i + 1))
        if fmt == 3:
            a64 = ref.values(ref.unpack(a[rows].cpu().numpy()), a_s.cpu().numpy().reshape(T, -1)[rows, : K // 32], None, 3)
            tiles = b_s[e * one : (e + 1) * one].cpu().numpy().reshape(N // 128, K // 128, 32, 4, 4)
            sc = tiles.transpose(0, 3, 2, 1, 4).reshape(N, K // 32)
            b64 = ref.values(ref.unpack(b[e].cpu().numpy()), sc, None, 3)
        else:
            a64, b64 = host(a[rows]), host(b[e])
        check_out(C[rows], *ref.product(a64, b64, None, None, None, 0, None), 0)


@pytest.mark.parametrize("T,N,K", [(70, 130, 1024), (20, 256, 4096), (300, 200, 512)])
def test_grouped_offsets_that_go_back(T, N, K):
    """Entries below an earlier one count as it: groups never overlap, also where blocks share tiles."""
    off = [0, T // 2, 0, T, 3, T, 0, T - 1, T, -5, T + 9]
    E = len(off) - 1
    a, b = torch.randn(T, K, device=DEV).bfloat16(), torch.randn(E, N, K, device=DEV).bfloat16()
    C = torch.full((T, N), 5.0, device=DEV)
    qg.qgemm_grouped_run(T, E, K, N, 2, torch.tensor(off, dtype=torch.int32, device=DEV), a, None, None, b, None, None, None, 0, C, 0)
    assert qg.qgemm_status() == 0
    for rows, e in ((slice(0, T // 2), 0), (slice(T // 2, T), 2)):
        check_out(C[rows], *ref.product(host(a[rows]), host(b[e]), None, None, None, 0, None), 0)


@pytest.mark.parametrize("fmt", [2, 3, 4])
def test_layer_inputs_of_the_call_before(fmt):
    """Kernels come up behind the one before them: every call reads what that one wrote, on buffers
    that change from call to call without a wait in between."""
    T, K, N, E = 96, 1024, 512, 4
    off = torch.tensor([0, 24, 48, 72, 96], dtype=torch.int32, device=DEV)
    b = torch.randn(E, N, K, device=DEV) * 0.05
    if fmt == 2:
        Bt = [b.bfloat16(), None, None]
    else:
        Q = [gpu_quant(b[e], N, K, fmt, 1) for e in range(E)]
        Bt = [torch.cat([q[i] for q in Q]) if Q[0][i] is not None else None for i in range(3)]
    xs = [torch.randn(T, K, device=DEV).bfloat16() for _ in range(6)]
    slot, one = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1), torch.ones(T, 1, device=DEV)

    def step(x, a, C, out):
        if fmt == 2:
            qg.qgemm_moe_combine(T, 1, K, T, x, 2, slot, one, None, a[0], 2)
        else:
            qg.qgemm_fp4_quant(T, K, x, 2, K, T, None, fmt, 0, *a)
        qg.qgemm_grouped_run(T, E, K, N, fmt, off, a[0], *(a[1:] if fmt != 2 else (None, None)), *Bt, None, 0, C, 2)
        qg.qgemm_moe_combine(T, 1, N, T, C, 2, slot, one, None, out, 2)

    def buffers():
        a = [torch.empty(T, K, dtype=torch.bfloat16, device=DEV)] if fmt == 2 else list(gpu_quant(xs[0], T, K, fmt))
        return a, torch.empty(T, N, dtype=torch.bfloat16, device=DEV)

    want = []
    for x in xs:
        a, C = buffers()
        out = torch.empty_like(C)
        step(x, a, C, out)
        torch.cuda.synchronize()
        want.append(out)
    a, C = buffers()
    outs = [torch.empty_like(C) for _ in range(60)]
    for i, out in enumerate(outs):                      # one set of buffers for all
        step(xs[i % 6], a, C, out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 6]), i


# ---------------------------------------------------------------- combination
@pytest.mark.parametrize("T,k,N,ydt,odt,residual", [(1, 1, 1, 0, 0, False), (8, 4, 2560, 2, 2, True), (5, 3, 77, 1, 0, True),
                                                    (130, 8, 1024, 2, 1, False), (33, 6, 520, 0, 2, True), (9, 32, 130, 1, 1, False),
                                                    (4, 0, 64, 2, 2, True), (1000, 2, 264, 0, 0, False)])
def test_combine(T, k, N, ydt, odt, residual):
    g = torch.Generator(device=DEV).manual_seed(T * N)
    R = T * k
    y = torch.randn(max(R, 1), N, generator=g, device=DEV).to(torch_dtype(ydt))
    slot = torch.randperm(max(R, 1), generator=g, device=DEV)[:R].to(torch.int32).view(T, k)
    if T > 4 and k > 1:
        slot[1, 0] = -1
        slot[2] = -1
        slot[3, 1] = R                                  # outside Y
    w = torch.rand(T, k, generator=g, device=DEV)
    res = torch.randn(T, N, generator=g, device=DEV).to(torch_dtype(odt)) if residual else None
    out = torch.full((T, N), 9.0, dtype=torch_dtype(odt), device=DEV)
    qg.qgemm_moe_combine(T, k, N, R, y, ydt, slot, w, res, out, odt)
    y64, s, w64 = host(y), slot.cpu().numpy(), host(w)
    want, size = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j in range(k):
            if 0 <= s[t, j] < R:
                want[t] += w64[t, j] * y64[s[t, j]]
                size[t] += np.abs(w64[t, j] * y64[s[t, j]])
    if residual:
        want += host(res)
        size += np.abs(host(res))
    # k fused multiply-adds and the residual, each rounded at 2^-24 of at most the terms' sum
    check_out(out, want, (k + 1) * 2.0 ** -24 * size, odt)
    if residual:
        qg.qgemm_moe_combine(T, k, N, R, y, ydt, slot, w, res, res, odt)
        assert torch.equal(res, out)


# ---------------------------------------------------------------- the layer
@pytest.mark.parametrize("fmt", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 12, 300])
def test_layer_of_experts(T, fmt):
    """Route, quantize and gather, gate / up with SwiGLU, quantize, down, combine: every step's output
    is the definition's of the inputs that the step was given."""
    E, k, H, F = 10, 3, 256, 192
    x = torch.randn(T, H, device=DEV).bfloat16()
    expert, weight, slot, row, offsets = gpu_route(torch.randn(T, E, device=DEV), k, 1)
    R = T * k
    w1, w2 = torch.randn(E, 2 * F, H, device=DEV) * 0.06, torch.randn(E, H, F, device=DEV) * 0.07

    def layer(a, rows, w, act):
        """One grouped product of a's rows, and its float64 definition."""
        N, K = w.shape[1:]
        off, cols = offsets.cpu().numpy(), N // 2 if act == 4 else N
        C = torch.zeros(R, cols, dtype=torch.bfloat16, device=DEV)
        if fmt == 2:
            A, Bt = [a[rows.long()] if rows is not None else a, None, None], [w.bfloat16(), None, None]
            a64, b64, sa, sb = host(A[0]), host(Bt[0]), None, [None] * E
        else:
            A = gpu_quant(a, R, K, fmt, 0, rows)
            Q = [gpu_quant(w[e].contiguous(), N, K, fmt, 1) for e in range(E)]
            Bt = [torch.cat([q[i] for q in Q]) if Q[0][i] is not None else None for i in range(3)]
            src = host(a)[rows.cpu().numpy()] if rows is not None else host(a)
            a64 = ref.values(*ref.quantize(src, fmt)[:2], None, fmt)
            b64 = [ref.values(*ref.quantize(host(w[e]), fmt)[:2], None, fmt) for e in range(E)]
            sa = None if A[2] is None else host(A[2])
            sb = [None if q[2] is None else host(q[2]) for q in Q]
        qg.qgemm_grouped_run(R, E, K, N, fmt, offsets, A[0], A[1], A[2], Bt[0], Bt[1], Bt[2], None, act, C, 2)
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                check_out(C[lo:hi], *ref.product(a64[lo:hi], b64[e], None if sa is None else sa[lo:hi], sb[e], None, act, None), 2)
        return C

    h = layer(x, row, w1, 4)
    y = layer(h, None, w2, 0)
    out = torch.empty_like(x)
    qg.qgemm_moe_combine(T, k, H, R, y, 2, slot, weight, x, out, 2)
    want = (host(y)[slot.cpu().numpy()] * host(weight)[..., None]).sum(1) + host(x)
    size = (np.abs(host(y))[slot.cpu().numpy()] * host(weight)[..., None]).sum(1) + np.abs(host(x))
    check_out(out, want, (k + 1) * 2.0 ** -24 * size, 2)
