"""The 4-bit floating-point and mixture-of-experts calls without a GPU: sizes and refusals."""
import pytest

import weight_quantized_gemm_gb300 as qg
from tests._util import ensure_built

FAKE = 1 << 40          # an aligned address that is never dereferenced (calls fail first)
ARG, UNSUP, ALIGN, WS, CUDA = -1, -2, -3, -4, -5


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def test_sizes():
    assert qg.qgemm_fp4_codes_bytes(3, 128) == 192
    assert qg.qgemm_fp4_codes_bytes(3, 100) == 0
    assert qg.qgemm_fp4_scales_bytes(3, 4096, 3, 0) == 3 * 128
    assert qg.qgemm_fp4_scales_bytes(3, 4096, 4, 0) == 3 * 256
    assert qg.qgemm_fp4_scales_bytes(3, 64, 3, 0) == 3 * 16                  # pitch of 16
    assert qg.qgemm_fp4_scales_bytes(129, 4096, 3, 1) == 2 * 32 * 512
    assert qg.qgemm_fp4_scales_bytes(128, 192, 4, 1) == 3 * 512
    assert qg.qgemm_fp4_scales_bytes(128, 192, 3, 1) == 2 * 512              # 6 scales: two tiles of 4
    assert qg.qgemm_fp4_scales_bytes(128, 192, 2, 1) == 0 and qg.qgemm_fp4_scales_bytes(128, 192, 3, 2) == 0
    assert qg.qgemm_fp4_scales_bytes(1 << 22, 1 << 14, 4, 0) == 1 << 32      # past 32 bits
    assert qg.qgemm_moe_route_workspace_bytes(1, 64, 8) == 0
    assert qg.qgemm_moe_route_workspace_bytes(4096, 64, 8) > 0
    assert qg.qgemm_moe_route_workspace_bytes(4096, 64, 65) == 0


def call(fn, defaults, args):
    a = dict(defaults)
    unknown = set(args) - set(a)
    assert not unknown
    a.update(args)
    return getattr(qg.load(), fn)(*a.values())


QUANT = dict(M=4, K=128, X=FAKE, x_dtype=2, ldx=128, x_rows=4, rows=None, fmt=4, layout=0, codes=FAKE, scales=FAKE, row_scale=FAKE,
             stream=None)


@pytest.mark.parametrize("args,code", [
    (dict(M=-1), ARG), (dict(K=0), ARG), (dict(K=96), UNSUP), (dict(fmt=2), ARG), (dict(x_dtype=3), ARG), (dict(layout=2), ARG),
    (dict(ldx=127), ARG), (dict(x_rows=3), ARG), (dict(x_rows=-1), ARG), (dict(X=None), ARG), (dict(codes=None), ARG),
    (dict(scales=None), ARG), (dict(row_scale=None), ARG), (dict(X=FAKE + 2), ALIGN), (dict(codes=FAKE + 8), ALIGN),
    (dict(rows=FAKE + 4), ALIGN), (dict(ldx=130), ALIGN), (dict(M=(1 << 30) + 1, x_rows=(1 << 31) - 1), UNSUP), (dict(K=1 << 26, ldx=1 << 26), UNSUP), (dict(M=0, X=None), 0)])
def test_quant_refuses(args, code):
    assert call("qgemm_fp4_quant", QUANT, args) == code


DEQUANT = dict(M=4, K=128, fmt=3, layout=0, codes=FAKE, scales=FAKE, row_scale=None, Y=FAKE, y_dtype=2, stream=None)


@pytest.mark.parametrize("args,code", [
    (dict(M=-1), ARG), (dict(K=32), UNSUP), (dict(fmt=1), ARG), (dict(layout=-1), ARG), (dict(y_dtype=9), ARG), (dict(codes=None), ARG),
    (dict(Y=None), ARG), (dict(Y=FAKE + 4), ALIGN), (dict(row_scale=FAKE + 4), ALIGN), (dict(M=0), 0)])
def test_dequant_refuses(args, code):
    assert call("qgemm_fp4_dequant", DEQUANT, args) == code


PACK = dict(W=FAKE, K=128, N=4, fmt=4, Bp=FAKE, Bs=FAKE, b_scale=FAKE, stream=None)


@pytest.mark.parametrize("args,code", [
    (dict(K=100), UNSUP), (dict(N=-1), ARG), (dict(fmt=0), ARG), (dict(W=None), ARG), (dict(Bs=None), ARG), (dict(b_scale=None), ARG),
    (dict(Bp=FAKE + 1), ALIGN), (dict(N=0, W=None), 0)])
def test_pack_refuses(args, code):
    assert call("qgemm_fp4_pack", PACK, args) == code


RUN = dict(M=4, K=128, N=64, fmt=3, A=FAKE, As=FAKE, a_scale=None, Bp=FAKE, Bs=FAKE, b_scale=None, bias=None, act=0, residual=None,
           C=FAKE, c_dtype=2, stream=None)


@pytest.mark.parametrize("args,code", [
    (dict(fmt=2), ARG), (dict(fmt=5), ARG), (dict(M=-1), ARG), (dict(N=-1), ARG), (dict(K=0), ARG), (dict(K=96), UNSUP),
    (dict(act=5), ARG), (dict(act=-1), ARG), (dict(act=4, N=63), UNSUP), (dict(c_dtype=3), ARG), (dict(A=None), ARG), (dict(As=None), ARG),
    (dict(Bs=None), ARG), (dict(C=None), ARG), (dict(C=FAKE + 2), ALIGN), (dict(a_scale=FAKE + 4), ALIGN), (dict(bias=FAKE + 8), ALIGN),
    (dict(residual=FAKE + 2), ALIGN), (dict(M=(1 << 31) - 1), UNSUP), (dict(N=(1 << 30) + 2), UNSUP), (dict(M=0, A=None), 0), (dict(N=0), 0)])
def test_run_refuses(args, code):
    assert call("qgemm_fp4_run", RUN, args) == code


GROUPED = dict(T=4, E=2, K=128, N=64, fmt=3, offsets=FAKE, A=FAKE, As=FAKE, a_scale=None, Bp=FAKE, Bs=FAKE, b_scale=None, bias=None,
               act=0, C=FAKE, c_dtype=2, stream=None)


@pytest.mark.parametrize("args,code", [
    (dict(fmt=0), ARG), (dict(T=-1), ARG), (dict(E=-1), ARG), (dict(E=1025), UNSUP), (dict(K=65), UNSUP), (dict(offsets=None), ARG),
    (dict(offsets=FAKE + 4), ALIGN), (dict(act=4, N=3), UNSUP), (dict(As=None), ARG), (dict(fmt=2, As=None, Bs=None, Bp=FAKE + 2), ALIGN),
    (dict(T=0, offsets=None), 0), (dict(E=0), 0), (dict(N=0), 0)])
def test_grouped_refuses(args, code):
    assert call("qgemm_grouped_run", GROUPED, args) == code


ROUTE = dict(T=200, E=8, k=2, logits=FAKE, dtype=0, ld=8, renorm=1, expert=FAKE, weight=FAKE, slot=FAKE, row=FAKE, offsets=FAKE, ws=FAKE,
             ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("args,code", [
    (dict(T=-1), ARG), (dict(E=0), ARG), (dict(k=0), ARG), (dict(k=9), ARG), (dict(dtype=4), ARG), (dict(renorm=2), ARG), (dict(ld=7), ARG),
    (dict(E=2000, ld=2000), UNSUP), (dict(E=64, ld=64, k=33), UNSUP), (dict(T=1 << 30), UNSUP), (dict(offsets=None), ARG),
    (dict(expert=None), ARG), (dict(row=FAKE + 4), ALIGN), (dict(ws=None), WS), (dict(ws_bytes=16), WS)])
def test_route_refuses(args, code):
    if "T" in args and args["T"] == 1 << 30:
        args = dict(args, k=4)
    assert call("qgemm_moe_route", ROUTE, args) == code


COMBINE = dict(T=4, k=2, N=64, R=8, Y=FAKE, y_dtype=2, slot=FAKE, weight=FAKE, residual=None, out=FAKE, out_dtype=2, stream=None)


@pytest.mark.parametrize("args,code", [
    (dict(T=-1), ARG), (dict(k=-1), ARG), (dict(R=-1), ARG), (dict(y_dtype=7), ARG), (dict(out_dtype=-1), ARG), (dict(Y=None), ARG),
    (dict(slot=None), ARG), (dict(out=None), ARG), (dict(out=FAKE + 2), ALIGN), (dict(N=1 << 23), UNSUP), (dict(T=0, out=None), 0),
    (dict(N=0), 0)])
def test_combine_refuses(args, code):
    assert call("qgemm_moe_combine", COMBINE, args) == code


@pytest.mark.parametrize("args", [dict(T=(1 << 30) + 1, k=1), dict(T=(1 << 31) - 1, k=0), dict(T=1, k=(1 << 31) - 1), dict(T=1 << 27, k=9)])
def test_combine_refuses_too_many_pairs(args):
    assert call("qgemm_moe_combine", COMBINE, args) == UNSUP


def test_swiglu_stays_with_the_new_products():
    assert qg.load().qgemm_run_fused(1, 128, 64, 1, 64, FAKE, 2, FAKE, FAKE, None, 4, None, FAKE, 2, FAKE, 1 << 20, None) == ARG


def test_injected_failures():
    calls = [("qgemm_fp4_quant", QUANT), ("qgemm_fp4_dequant", DEQUANT), ("qgemm_fp4_pack", PACK), ("qgemm_fp4_run", RUN),
             ("qgemm_grouped_run", GROUPED), ("qgemm_moe_route", ROUTE), ("qgemm_moe_combine", COMBINE)]
    for fn, defaults in calls:
        qg.qgemm_set_option(qg.OPT_FAULT_INJECT, 1)
        assert call(fn, defaults, {}) == CUDA
        assert "simulated" in qg.qgemm_last_error()
        assert qg.qgemm_get_option(qg.OPT_FAULT_INJECT) == 0
