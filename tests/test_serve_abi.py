"""The calls around the layers (adapters, norms, log probabilities) without a GPU: refusals."""
import pytest

import weight_quantized_gemm_gb300 as qg
from tests._util import ensure_built
from tests.test_experts_abi import ALIGN, ARG, CUDA, FAKE, UNSUP, call


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


GROUP = dict(M=4, L=8, adapter=FAKE, row=FAKE, offsets=FAKE, stream=None)


@pytest.mark.parametrize("args,code", [
    (dict(M=-1), ARG), (dict(L=0), ARG), (dict(L=1025), UNSUP), (dict(M=(1 << 30) + 1), UNSUP), (dict(adapter=None), ARG), (dict(row=None), ARG),
    (dict(offsets=None), ARG), (dict(M=0, offsets=None), ARG), (dict(adapter=FAKE + 4), ALIGN), (dict(row=FAKE + 8), ALIGN), (dict(offsets=FAKE + 4), ALIGN)])
def test_group_refuses(args, code):
    assert call("qgemm_lora_group", GROUP, args) == code


LORA = dict(M=4, K=128, N=100, L=8, R=16, dtype=2, row=FAKE, offsets=FAKE, X=FAKE, ldx=128, A=FAKE, B=FAKE, rank=None, scale=None, Y=FAKE,
            y_dtype=2, ldy=100, stream=None)


@pytest.mark.parametrize("args,code", [
    (dict(M=-1), ARG), (dict(K=0), ARG), (dict(N=-1), ARG), (dict(L=0), ARG), (dict(R=0), ARG), (dict(dtype=0), ARG), (dict(dtype=3), ARG),
    (dict(y_dtype=3), ARG), (dict(ldx=127), ARG), (dict(ldy=99), ARG), (dict(K=96, ldx=96), UNSUP), (dict(R=12), UNSUP), (dict(R=264), UNSUP),
    (dict(L=1025), UNSUP), (dict(M=(1 << 30) + 1), UNSUP), (dict(N=(1 << 30) + 1, ldy=1 << 31), UNSUP), (dict(ldy=1 << 60), UNSUP),
    (dict(row=None), ARG), (dict(offsets=None), ARG), (dict(X=None), ARG), (dict(A=None), ARG), (dict(B=None), ARG), (dict(Y=None), ARG),
    (dict(X=FAKE + 8), ALIGN), (dict(Y=FAKE + 2), ALIGN), (dict(rank=FAKE + 4), ALIGN), (dict(scale=FAKE + 4), ALIGN), (dict(ldx=132), ALIGN),
    (dict(M=0, X=None), 0), (dict(N=0, ldy=0, Y=None), 0)])
def test_lora_refuses(args, code):
    assert call("qgemm_lora_run", LORA, args) == code


NORM = dict(M=4, K=128, kind=1, eps=1e-5, X=FAKE, x_dtype=2, ldx=128, x_scale=1.0, post=1, post_weight=FAKE, gate=FAKE, ldg=0, residual=FAKE,
            r_scale=1.0, S=FAKE, s_dtype=0, weight=FAKE, bias=None, Y=FAKE, y_dtype=2, stream=None)
NORM["Y"] = FAKE + 4096


@pytest.mark.parametrize("args,code", [
    (dict(M=-1), ARG), (dict(K=0), ARG), (dict(K=96, ldx=96), UNSUP), (dict(K=32832, ldx=32832), UNSUP), (dict(M=(1 << 30) + 1), UNSUP),
    (dict(kind=0), ARG), (dict(kind=3), ARG), (dict(eps=-1e-5), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(x_dtype=3), ARG), (dict(s_dtype=-1), ARG), (dict(y_dtype=4), ARG), (dict(post=2), ARG), (dict(post=0), ARG), (dict(ldx=120), ARG),
    (dict(ldg=64), ARG), (dict(ldg=-8), ARG), (dict(ldx=1 << 60), UNSUP), (dict(X=None), ARG), (dict(S=None, Y=None), ARG), (dict(X=FAKE + 2), ALIGN),
    (dict(weight=FAKE + 4), ALIGN), (dict(gate=FAKE + 8), ALIGN), (dict(ldx=132), ALIGN), (dict(ldg=132), ALIGN), (dict(Y=FAKE, y_dtype=0), ARG),
    (dict(Y=FAKE, ldx=136), ARG), (dict(M=0, X=None), 0)])
def test_norm_refuses(args, code):
    assert call("qgemm_norm_run", NORM, args) == code


LOGP = dict(T=4, V=1001, logits=FAKE, dtype=2, ld=1001, scale=1.0, token=FAKE, logprob=FAKE, entropy=FAKE, k=5, top=FAKE, top_logprob=FAKE,
            stream=None)


@pytest.mark.parametrize("args,code", [
    (dict(T=-1), ARG), (dict(V=0), ARG), (dict(k=-1), ARG), (dict(k=33), UNSUP), (dict(dtype=3), ARG), (dict(ld=1000), ARG), (dict(scale=0.0), ARG),
    (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(T=(1 << 30) + 1), UNSUP),
    (dict(V=(1 << 30) + 1, ld=1 << 31), UNSUP), (dict(ld=1 << 60), UNSUP), (dict(logits=None), ARG), (dict(token=None), ARG), (dict(logprob=None), ARG),
    (dict(top=None), ARG), (dict(top_logprob=None), ARG), (dict(logits=FAKE + 2), ALIGN), (dict(token=FAKE + 4), ALIGN), (dict(top=FAKE + 4), ALIGN),
    (dict(T=0, logits=None), 0), (dict(token=None, logprob=None, entropy=None, k=0), 0)])
def test_logprobs_refuses(args, code):
    assert call("qgemm_logprobs", LOGP, args) == code


def test_injected_failures():
    for fn, defaults in (("qgemm_lora_group", GROUP), ("qgemm_lora_run", LORA), ("qgemm_norm_run", NORM), ("qgemm_logprobs", LOGP)):
        qg.qgemm_set_option(qg.OPT_FAULT_INJECT, 1)
        assert call(fn, defaults, {}) == CUDA
        assert "simulated" in qg.qgemm_last_error()
        assert qg.qgemm_get_option(qg.OPT_FAULT_INJECT) == 0
