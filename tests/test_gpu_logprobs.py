"""Log probabilities, entropy and the likeliest tokens against their definitions in float64."""
import math

import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests import _serve_ref as ref
from tests._util import ensure_built, torch_dtype

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def run(x, dtype, V, k, scale=1.0, token=None, entropy=True, stream=None):
    T, ld = x.shape
    lp = torch.full((T,), 7.0, device=DEV) if token is not None else None
    h = torch.full((T,), 7.0, device=DEV) if entropy else None
    top = torch.full((T, k), 77, dtype=torch.int32, device=DEV) if k else None
    tlp = torch.full((T, k), 7.0, device=DEV) if k else None
    qg.qgemm_logprobs(T, V, x, dtype, ld, scale, token, lp, h, k, top, tlp, stream)
    return dict(logprob=lp, entropy=h, top=top, top_logprob=tlp)


def check(x, dtype, V, k, scale=1.0, token=None):
    got = run(x, dtype, V, k, scale, token)
    want = ref.logprobs(x[:, :V], scale, token, k)
    close(got, want, k, token)


def close(got, want, k, token):
    allow = want["allow"]
    u = 4 * ref.U                       # (z - M) scale and the two differences: half a step each
    if token is not None:
        ref.check(got["logprob"], want["logprob"], allow + u * want["logprob"].abs().nan_to_num(posinf=0))
    # ln S as above, and a sum of terms each as exact as its weight, over S
    h = want["entropy"]
    ref.check(got["entropy"], h, allow * 2 * (1 + h))
    if k:
        assert torch.equal(got["top"], want["top"])
        ref.check(got["top_logprob"], want["top_logprob"], allow[:, None] + u * want["top_logprob"].abs().nan_to_num(posinf=0))


def logits(T, ld, dtype, seed=0, std=2.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + T + ld)
    return (torch.randn(T, ld, generator=g, device=DEV) * std).to(torch_dtype(dtype)), torch.randint(ld, (T,), generator=g, device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("dtype", [qg.F32, qg.F16, qg.BF16])
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (2, 2, 5), (3, 7, 32), (4, 33, 0), (5, 255, 1), (2, 1000, 20), (9, 4097, 32), (1, 8192, 8), (1, 16385, 32),
                                   (2, 32769, 5), (1, 131072, 32), (3, 50001, 20), (160, 5003, 8), (330, 2048, 5), (40, 20000, 17)])
def test_sizes(T, V, k, dtype):
    x, token = logits(T, V, dtype)
    check(x, dtype, V, k, token=token.clamp(max=V - 1))


@pytest.mark.parametrize("dtype", [qg.F32, qg.F16, qg.BF16])
@pytest.mark.parametrize("V,ld", [(1000, 1001), (1001, 1008), (999, 1003), (4096, 4099)])
def test_rows_that_start_anywhere(V, ld, dtype):
    x, token = logits(9, ld, dtype)
    x[:, V:] = INF                     # behind the row: not part of it
    check(x, dtype, V, 9, 0.7, token.clamp(max=V - 1))


@pytest.mark.parametrize("dtype", [qg.F32, qg.F16, qg.BF16])
@pytest.mark.parametrize("T", [1, 3, 400])
def test_ties_go_to_the_lowest_token(T, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    V = 9000
    x = torch.randint(-2, 3, (T, V), generator=g, device=DEV).float()
    x[0] = 1.0                                            # one value everywhere
    x[T // 2, ::3] = -0.0
    x = x.to(torch_dtype(dtype))
    check(x, dtype, V, 32, token=torch.full((T,), 5, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("order", ["falling", "rising", "one thread"])
def test_best_values_in_unlucky_places(order):
    """All the best values with one thread (pieces 512 apart), and rows in order."""
    V, dtype = 40000, qg.F32
    x = torch.arange(V, dtype=torch.float32, device=DEV).flip(0) if order == "falling" else torch.arange(V, dtype=torch.float32, device=DEV)
    if order == "one thread":
        x = torch.randn(V, device=DEV)
        x[4 * 7:: 4 * 512] = 50 + torch.arange(len(x[4 * 7:: 4 * 512]), device=DEV).float()
    x = x[None].repeat(2, 1) * 0.01
    check(x, dtype, V, 32, token=torch.tensor([3, V - 1], dtype=torch.int32, device=DEV))
    check(x.repeat(300, 1), dtype, V, 32, token=torch.full((600,), 11, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("dtype", [qg.F32, qg.F16, qg.BF16])
@pytest.mark.parametrize("T,V", [(6, 3000), (6, 60000), (400, 700)])
def test_masks_infinities_and_nan(T, V, dtype):
    x, token = logits(T, V, dtype)
    x[0] = -INF                                           # nothing is left
    x[1] = NAN
    x[2, : V - 1] = -INF                                  # one token is left
    x[3, ::2], x[3, 1] = NAN, -INF
    x[4, 5], x[4, V - 1] = INF, INF                       # two share it
    x[5, 3:] = torch.finfo(torch_dtype(dtype)).min        # masked with the lowest finite value
    token[:6] = torch.tensor([0, 3, V - 1, 7, 5, 2], dtype=torch.int32)
    check(x, dtype, V, 10, 1.0, token)
    token[:6] = torch.tensor([V - 1, 2, 0, 0, 6, 9], dtype=torch.int32)
    check(x, dtype, V, 10, 1.0, token)


def test_tokens_outside_are_zero():
    x, _ = logits(4, 500, qg.BF16)
    check(x, qg.BF16, 500, 3, token=torch.tensor([-1, 500, 1 << 30, 499], dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("scale", [1e-30, 0.01, 3.0, 50.0, 1e30])
def test_scales(scale):
    x, token = logits(5, 3001, qg.F32)
    check(x, qg.F32, 3001, 5, scale, token)


@pytest.mark.parametrize("T,V,ld,place,above", [(1, 5000, 5000, 17, 14.0), (3, 131072, 131072, 99999, 20.0), (300, 9001, 9003, 0, 16.0), (5, 40000, 40001, 39999, 25.0),
                                                (2, 600, 601, 300, 9.0)])
@pytest.mark.parametrize("dtype", [qg.F32, qg.BF16])
def test_rows_that_one_logit_dominates(T, V, ld, place, above, dtype):
    """-ln p of a token that is nearly certain: small, and good to a few units of its own size. Terms of t below 60 doublings: t is off by
    3 u t, the powers and rescaled sums by 2^-22 each (4 of them), and n additions a thread and block."""
    x, token = logits(T, ld, dtype, std=1.0)
    x[:, place] = above
    token[:] = place
    got = run(x, dtype, V, 3, 1.25, token)
    z = x[:, :V].double() * 1.25
    rest = torch.exp(z - z[:, place:place + 1])
    rest[:, place] = 0
    want = torch.log1p(rest.sum(-1))
    bound = 4 * 2.0 ** -22 + 3 * 60 * math.log(2) * ref.U + (V / 256 + 64) * ref.U
    assert bool((want < 0.4).all())
    assert bool(((got["logprob"].double() + want).abs() <= want * bound).all())
    assert bool(((got["top_logprob"][:, 0].double() + want).abs() <= want * bound).all())
    h = want - (torch.where(rest > 0, z - z[:, place:place + 1], 0) * rest).sum(-1) / (1 + rest.sum(-1))
    assert bool(((got["entropy"].double() - h).abs() <= h * 2 * bound).all())


def test_rising_logits_far_apart():
    """Each value far above the ones before: the sums' reference moves at every step."""
    x = (torch.arange(6000, device=DEV).float() * 8)[None].repeat(3, 1)
    check(x, qg.F32, 6000, 4, token=torch.tensor([5999, 5998, 0], dtype=torch.int32, device=DEV))
    check(x.flip(1).contiguous(), qg.F32, 6000, 4, token=torch.tensor([5999, 1, 0], dtype=torch.int32, device=DEV))


def test_outputs_alone():
    x, token = logits(7, 3000, qg.F16)
    want = ref.logprobs(x, 1.0, token, 6)
    both = run(x, qg.F16, 3000, 6, token=token)
    close(both, want, 6, token)
    assert torch.equal(run(x, qg.F16, 3000, 0, token=token, entropy=False)["logprob"], both["logprob"])
    assert torch.equal(run(x, qg.F16, 3000, 0)["entropy"], both["entropy"])
    alone = run(x, qg.F16, 3000, 6, entropy=False)
    assert torch.equal(alone["top"], both["top"]) and torch.equal(alone["top_logprob"], both["top_logprob"])


def test_rows_past_32_bits():
    ld = 1 << 28
    x = torch.empty(17 * ld, dtype=torch.bfloat16, device=DEV).view(17, ld)
    small, token = logits(17, 4000, qg.BF16)
    x[:, :4000] = small
    got = run(x, qg.BF16, 4000, 5, token=token)
    close(got, ref.logprobs(small, 1.0, token, 5), 5, token)


def test_a_long_row():
    """2^25 logits: sums of many terms, and more than 32 pieces a thread."""
    V = 1 << 25
    x, token = logits(1, V, qg.BF16)
    check(x, qg.BF16, V, 32, token=token)


def test_another_stream_and_a_graph():
    x, token = logits(5, 30000, qg.BF16)
    first = run(x, qg.BF16, 30000, 8, token=token)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run(x, qg.BF16, 30000, 8, token=token)
    torch.cuda.current_stream().wait_stream(side)
    for n in first:
        assert torch.equal(first[n], again[n])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(x, qg.BF16, 30000, 8, token=token)
    x.copy_(x.flip(1))
    graph.replay()
    close(out, ref.logprobs(x, 1.0, token, 8), 8, token)
