"""4-bit floating point on the GPU: quantization (bit for bit), its inverse, weight packing and the
product of two 4-bit operands, against the float64 definitions of _experts_ref.py."""
import numpy as np
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests import _experts_ref as ref
from tests._util import ensure_built, half_ulp, torch_dtype

pytestmark = pytest.mark.gpu
DEV = "cuda"
MX, NV = qg.FMT_MXFP4, qg.FMT_NVFP4


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def host(t):
    return t.double().cpu().numpy()


def gpu_quant(x, M, K, fmt, layout=0, rows=None, stream=None):
    """Codes [M][K], raw scale bytes and row scales of the library's quantization of x (a 2-D tensor,
    possibly with padded rows)."""
    codes = torch.full((M, K // 2), 0xEE, dtype=torch.uint8, device=DEV)
    sb = torch.full((qg.qgemm_fp4_scales_bytes(M, K, fmt, layout),), 0xEE, dtype=torch.uint8, device=DEV)
    rs = torch.full((M,), -5.0, device=DEV) if fmt == NV else None
    dt = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[x.dtype]
    qg.qgemm_fp4_quant(M, K, x, dt, x.stride(0), x.shape[0], rows, fmt, layout, codes, sb, rs, stream)
    return codes, sb, rs


def check_quant(x64, codes, sb, rs, fmt, layout, K):
    c, byte, row = ref.quantize(x64, fmt)
    good = np.repeat(byte != 255, 32, 1) if fmt == MX else np.isfinite(row)[:, None] & np.ones((1, K), bool)
    assert np.array_equal(ref.unpack(codes.cpu().numpy())[good], c[good])
    lay = (ref.rows_layout if layout == 0 else ref.tiled_layout)(byte, K, fmt)
    assert np.array_equal(sb.cpu().numpy().reshape(lay.shape), lay)
    if fmt == NV:
        assert np.array_equal(host(rs), row, equal_nan=True)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("M,K", [(1, 64), (3, 192), (130, 1024), (7, 4160), (2, 20480)])
def test_quant_bits(M, K, dt, fmt):
    g = torch.Generator(device=DEV).manual_seed(M * K + dt)
    x = torch.randn(M, K, generator=g, device=DEV) * torch.exp2(torch.randint(-6, 7, (M, K // 16), generator=g, device=DEV).float()).repeat_interleave(16, 1)
    x = x.to(torch_dtype(dt))
    for layout in (0, 1):
        check_quant(host(x), *gpu_quant(x, M, K, fmt, layout), fmt, layout, K)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [0, 1, 2])
def test_quant_ties_and_edges(fmt, dt):
    """Every tie of the code grid at several block scales, values one step off the ties, zeros of
    both signs, blocks of zeros, subnormals, the largest values."""
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 3.0, 4.0, 0.0, -0.0, 7.0, 0.1])
    rows = []
    for s in (1.0, 0.875, 1.125, 13.0, 240.0, 2.0 ** -8):
        b = ties * s
        rows.append(np.concatenate([b, -b, np.zeros(16), b * 1.0078125, b * 0.9921875, [6 * s] + [0] * 15, b / 16, -b]))
    x = torch.tensor(np.stack(rows), dtype=torch.float32).to(torch_dtype(dt))
    fi = torch.finfo(torch_dtype(dt))
    x = torch.cat([x, x * 2.0 ** -12, torch.zeros_like(x[:1]), torch.full_like(x[:1], -0.0), torch.full_like(x[:1], fi.max),
                   torch.full_like(x[:1], fi.smallest_normal), x[:1] * (fi.max / 2048), x[:1] * (fi.tiny * 4)]).to(DEV)
    tiny = torch.zeros_like(x[:1])
    tiny[0, ::5] = fi.tiny / 4                          # subnormal in f16 and bf16, and in f32
    x = torch.cat([x, tiny])
    M, K = x.shape
    check_quant(host(x), *gpu_quant(x, M, K, fmt), fmt, 0, K)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_quant_infinities_and_nan(fmt):
    x = torch.randn(4, 256, device=DEV, dtype=torch.bfloat16)
    x[1, 70] = float("nan")
    x[2, 255] = float("-inf")
    codes, sb, rs = gpu_quant(x, 4, 256, fmt)
    check_quant(host(x), codes, sb, rs, fmt, 0, 256)
    y = torch.empty_like(x)
    qg.qgemm_fp4_dequant(4, 256, fmt, 0, codes, sb, rs, y, 2)
    bad = torch.isnan(y).cpu().numpy()
    want = np.zeros((4, 256), bool)
    if fmt == MX:
        want[1, 64:96] = want[2, 224:] = True
    else:
        want[1] = want[2] = True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_quant_gather_and_strides(fmt):
    K = 320
    full = torch.randn(50, K + 24, device=DEV, dtype=torch.float16)
    x = full[:, :K]                                     # rows of K values, K + 24 apart
    rows = torch.tensor([49, 0, 0, -1, 7, 50, 1 << 30, 12, -(1 << 31), 3], dtype=torch.int32, device=DEV)
    got = gpu_quant(x, 10, K, fmt, 0, rows)
    src = np.zeros((10, K))
    for i, r in enumerate(rows.tolist()):
        if 0 <= r < 50:
            src[i] = host(x)[r]
    check_quant(src, *got, fmt, 0, K)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_quant_and_dequant_past_32_bits(fmt):
    """Rows more than 2^32 bytes and 2^31 values into X, Y and past 2^30 into the codes."""
    M, K = 530000, 4160
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV).normal_()
    codes, sb, rs = gpu_quant(x, M, K, fmt)
    y = torch.empty_like(x)
    qg.qgemm_fp4_dequant(M, K, fmt, 0, codes, sb, rs, y, 2)
    for m in (0, 258111, 516223, M - 1):                # around 2^30 and 2^31 values, and the last
        c, byte, row = ref.quantize(host(x[m : m + 1]), fmt)
        assert np.array_equal(ref.unpack(codes[m : m + 1].cpu().numpy()), c)
        want = ref.values(c, byte, row, fmt)
        assert np.array_equal(host(y[m : m + 1]), want)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [0, 1, 2])
def test_dequant(fmt, dt):
    """Every code under every scale byte; one rounding to the output type."""
    K = 4096 if fmt == NV else 8192
    M = 5
    codes = torch.arange(K, dtype=torch.int32).remainder(16).to(torch.uint8).repeat(M, 1)
    byte = torch.arange(K // ref.BLOCK[fmt], dtype=torch.int32).remainder(127 if fmt == NV else 256).to(torch.uint8).repeat(M, 1)
    row = torch.tensor([1.0, 2.0 ** -30, 3.7, 2.0 ** 20, 1e-3]) if fmt == NV else None
    packed = torch.from_numpy(ref.pack(codes.numpy())).to(DEV)
    R = ref.values(codes.numpy(), byte.numpy(), None if row is None else row.double().numpy(), fmt)
    for layout in (0, 1):
        sb = torch.from_numpy((ref.rows_layout if layout == 0 else ref.tiled_layout)(byte.numpy(), K, fmt)).to(DEV)
        y = torch.full((M, K), 7.0, dtype=torch_dtype(dt), device=DEV)
        qg.qgemm_fp4_dequant(M, K, fmt, layout, packed, sb, None if row is None else row.to(DEV), y, dt)
        with np.errstate(over="ignore"):
            want = torch.from_numpy(R.astype(np.float32)).to(torch_dtype(dt))
        assert torch.equal(torch.nan_to_num(y.cpu(), nan=123.0), torch.nan_to_num(want, nan=123.0))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("K,N", [(64, 1), (192, 40), (1024, 130), (448, 256)])
def test_pack(K, N, fmt):
    W = torch.randn(K, N, device=DEV) * 0.02
    Bp = torch.full((qg.qgemm_fp4_codes_bytes(N, K),), 0xEE, dtype=torch.uint8, device=DEV)
    Bs = torch.full((qg.qgemm_fp4_scales_bytes(N, K, fmt, 1),), 0xEE, dtype=torch.uint8, device=DEV)
    bs = torch.full((N,), -1.0, device=DEV) if fmt == NV else None
    qg.qgemm_fp4_pack(W, K, N, fmt, Bp, Bs, bs)
    check_quant(host(W.T), Bp.view(N, K // 2), Bs, bs, fmt, 1, K)


def operands(M, N, K, fmt, seed):
    """Quantized random operands: (A tensors, B tensors, float64 A without row scales, same of B)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    a = torch.randn(M, K, generator=g, device=DEV)
    a[:, :: max(K // 7, 1)] *= 30
    b = torch.randn(N, K, generator=g, device=DEV) * 0.05
    A, B = gpu_quant(a, M, K, fmt, 0), gpu_quant(b, N, K, fmt, 1)
    full = []
    for x in (a, b):
        c, byte, _ = ref.quantize(host(x), fmt)
        full.append(ref.values(c, byte, None, fmt))
    return A, B, full[0], full[1]


def check_out(C, R, err, dt):
    got = host(C)
    assert got.shape == R.shape
    off = np.abs(got - R) - err - half_ulp(R, dt)
    assert np.all(off <= 0), f"worst {off.max():.3e} past the bound at {np.unravel_index(off.argmax(), off.shape)}"


RUNS = [
    # M, N, K, c_dtype, act, bias, residual
    (1, 128, 64, 0, 0, False, False),
    (1, 1, 64, 0, 0, False, False),
    (1, 2560, 4096, 2, 0, True, False),
    (2, 136, 128, 1, 1, True, True),
    (5, 200, 192, 0, 2, True, True),
    (16, 513, 320, 0, 3, False, True),
    (17, 96, 1024, 2, 2, True, False),
    (31, 1000, 2560, 2, 0, False, True),
    (33, 128, 256, 0, 4, True, False),
    (64, 330, 576, 1, 4, True, True),
    (77, 129, 4160, 2, 0, True, True),
    (100, 384, 512, 0, 0, False, False),
    (128, 256, 1024, 2, 3, True, False),
    (129, 127, 448, 0, 0, True, False),
    (192, 500, 768, 1, 2, False, False),
    (256, 1024, 2560, 2, 0, True, True),
    (300, 258, 832, 0, 4, False, False),
    (511, 640, 1984, 2, 1, True, False),
    (1025, 2000, 704, 1, 0, False, True),
    (2048, 2560, 1024, 2, 4, True, False),
]


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("M,N,K,dt,act,bias,residual", RUNS)
def test_run(M, N, K, dt, act, bias, residual, fmt):
    A, B, a64, b64 = operands(M, N, K, fmt, M + N + K)
    cols = N // 2 if act == 4 else N
    bias_t = torch.randn(N, device=DEV) if bias else None
    res = torch.randn(M, cols, device=DEV).to(torch_dtype(dt)) if residual else None
    R, err = ref.product(a64, b64, A[2] if A[2] is None else host(A[2]), B[2] if B[2] is None else host(B[2]),
                         None if bias_t is None else host(bias_t), act, None if res is None else host(res))
    # rows of C around the output stay as they are
    guard = torch.full((M + 2, cols), 5.0, dtype=torch_dtype(dt), device=DEV)
    off = cols * guard.element_size()
    C = guard[1 : M + 1] if off % 16 == 0 else torch.full((M, cols), 5.0, dtype=torch_dtype(dt), device=DEV)
    qg.qgemm_fp4_run(M, K, N, fmt, A[0], A[1], A[2], B[0], B[1], B[2], bias_t, act, res, C, dt)
    assert qg.qgemm_status() == 0
    check_out(C, R, err, dt)
    assert torch.all(guard[0] == 5) and torch.all(guard[-1] == 5)
    again = torch.empty_like(C, memory_format=torch.contiguous_format)
    qg.qgemm_fp4_run(M, K, N, fmt, A[0], A[1], A[2], B[0], B[1], B[2], bias_t, act, res, again, dt)
    assert torch.equal(C, again)                        # the same bits every time
    if residual:
        qg.qgemm_fp4_run(M, K, N, fmt, A[0], A[1], A[2], B[0], B[1], B[2], bias_t, act, res, res, dt)
        assert torch.equal(C, res)                      # in place


@pytest.mark.parametrize("fmt", [MX, NV])
def test_run_nan_stays_in_its_row(fmt):
    """A NaN or infinity in one activation row, and in one weight channel, reaches that row and that
    column of C and nothing else."""
    M, N, K = 40, 300, 512
    a, w = torch.randn(M, K, device=DEV), torch.randn(K, N, device=DEV)
    a[7, 100], w[3, 211] = float("nan"), float("inf")
    A = gpu_quant(a, M, K, fmt)
    Bp = torch.empty(qg.qgemm_fp4_codes_bytes(N, K), dtype=torch.uint8, device=DEV)
    Bs = torch.empty(qg.qgemm_fp4_scales_bytes(N, K, fmt, 1), dtype=torch.uint8, device=DEV)
    bs = torch.empty(N, device=DEV) if fmt == NV else None
    qg.qgemm_fp4_pack(w, K, N, fmt, Bp, Bs, bs)
    C = torch.zeros(M, N, device=DEV)
    qg.qgemm_fp4_run(M, K, N, fmt, A[0], A[1], A[2], Bp, Bs, bs, None, 0, None, C, 0)
    want = torch.zeros(M, N, dtype=torch.bool)
    want[7], want[:, 211] = True, True
    assert torch.equal(torch.isnan(C).cpu(), want)


def test_other_stream_and_graph():
    """On another stream, and captured into a graph and replayed on changed inputs."""
    M, N, K = 24, 512, 1024
    A, B, _, _ = operands(M, N, K, MX, 1)
    C0, C1 = torch.zeros(M, N, device=DEV), torch.zeros(M, N, device=DEV)
    qg.qgemm_fp4_run(M, K, N, MX, A[0], A[1], None, B[0], B[1], None, None, 0, None, C0, 0)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        qg.qgemm_fp4_run(M, K, N, MX, A[0], A[1], None, B[0], B[1], None, None, 0, None, C1, 0)
    st.synchronize()
    assert torch.equal(C0, C1)
    x = torch.randn(M, K, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.qgemm_fp4_quant(M, K, x, 0, K, M, None, MX, 0, A[0], A[1])
        qg.qgemm_fp4_run(M, K, N, MX, A[0], A[1], None, B[0], B[1], None, None, 0, None, C1, 0)
    x.copy_(torch.randn(M, K, device=DEV))
    g.replay()
    A2 = gpu_quant(x, M, K, MX)
    qg.qgemm_fp4_run(M, K, N, MX, A2[0], A2[1], None, B[0], B[1], None, None, 0, None, C0, 0)
    torch.cuda.synchronize()
    assert torch.equal(C0, C1)
