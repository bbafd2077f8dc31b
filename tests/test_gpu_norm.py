"""The step between two blocks (norm, gate, residual sum, norm) against its definition in float64."""
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests import _serve_ref as ref
from tests._util import ensure_built, torch_dtype

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = 96


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def make(M, K, kind, x_dtype, s_dtype, y_dtype, post=1, gate="channel", residual=True, affine="both", pad=0, seed=0, mean=0.3):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + M + K)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    xt, st = torch_dtype(x_dtype), torch_dtype(s_dtype)
    c = dict(M=M, K=K, kind=kind, x_dtype=x_dtype, s_dtype=s_dtype, y_dtype=y_dtype, post=post)
    c["X"] = (randn(M, K + pad) + mean).to(xt)
    c["post_weight"] = 1 + 0.2 * randn(K) if post else None
    c["gate"] = {"none": None, "channel": randn(K).to(xt), "row": randn(M, K + pad).to(xt)}[gate]
    c["ldg"] = K + pad if gate == "row" else 0
    c["residual"] = (3 * randn(M, K)).to(st) if residual else None
    c["weight"] = 1 + 0.2 * randn(K) if affine != "none" else None
    c["bias"] = randn(K) if affine == "both" else None
    return c


def run(c, S="new", Y="new", eps=1e-5, x_scale=1.5, r_scale=0.75):
    M, K = c["M"], c["K"]
    # values behind the last row stay as they were
    new = lambda dt: torch.full((M * K + GUARD,), 7.0, dtype=torch_dtype(dt), device=DEV)  # noqa: E731
    S_ = new(c["s_dtype"]) if S == "new" else S
    Y_ = new(c["y_dtype"]) if Y == "new" else Y
    qg.qgemm_norm_run(M, K, c["kind"], eps, c["X"], c["x_dtype"], c["X"].shape[1], x_scale, c["post"], c["post_weight"], c["gate"], c["ldg"],
                      c["residual"], r_scale, S_, c["s_dtype"], c["weight"], c["bias"], Y_, c["y_dtype"])
    out = []
    for b, kind in ((S_, S), (Y_, Y)):
        if kind == "new":
            assert bool((b[M * K:] == 7).all())
            b = b[: M * K].view(M, K)
        out.append(b)
    return out


def want(c, eps=1e-5, x_scale=1.5, r_scale=0.75):
    K = c["K"]
    gate = c["gate"][..., :K] if c["gate"] is not None else None
    return ref.norm(c["X"][:, :K], c["kind"], eps, x_scale, c["post"], c["post_weight"], gate, c["residual"], r_scale, c["weight"], c["bias"])


def check(c, **kw):
    s, es, y, ey = want(c, **kw)
    S, Y = run(c, **kw)
    ref.check(S, s, es, "S")
    ref.check(Y, y, ey, "Y")


@pytest.mark.parametrize("kind", [qg.NORM_RMS, qg.NORM_LAYER])
@pytest.mark.parametrize("x_dtype", [qg.F32, qg.F16, qg.BF16])
@pytest.mark.parametrize("s_dtype", [qg.F32, qg.F16, qg.BF16])
@pytest.mark.parametrize("y_dtype", [qg.F32, qg.F16, qg.BF16])
@pytest.mark.parametrize("M,K", [(3, 128), (5, 4160), (2, 9728)])
def test_types(M, K, x_dtype, s_dtype, y_dtype, kind):
    check(make(M, K, kind, x_dtype, s_dtype, y_dtype))


@pytest.mark.parametrize("kind", [qg.NORM_RMS, qg.NORM_LAYER])
@pytest.mark.parametrize("M,K", [(1, 64), (9, 64), (1001, 192), (7, 256), (6, 320), (5, 2048), (3, 4096), (300, 4096), (305, 4096), (310, 320), (306, 1088), (306, 2240), (305, 9728), (305, 10304), (305, 64), (2, 8192), (3, 8256), (2, 16384), (1, 16448), (2, 32768)])
def test_sizes(M, K, kind):
    check(make(M, K, kind, qg.BF16, qg.F32, qg.BF16, gate="row"))


@pytest.mark.parametrize("post", [0, 1])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("affine", ["none", "weight", "both"])
def test_parts(post, gate, residual, affine):
    check(make(6, 1024, qg.NORM_RMS, qg.BF16, qg.BF16, qg.BF16, post, gate, residual, affine, pad=64))


def test_post_without_weight_and_single_outputs():
    c = make(6, 1024, qg.NORM_LAYER, qg.F16, qg.F32, qg.F16)
    c["post_weight"] = None
    s, es, y, ey = want(c)
    S, none = run(c, Y=None)
    ref.check(S, s, es)
    none, Y = run(c, S=None)
    ref.check(Y, y, ey)


@pytest.mark.parametrize("K", [512, 4096, 9728])
def test_in_place(K):
    """S over the residual, Y over X."""
    c = make(40, K, qg.NORM_RMS, qg.BF16, qg.F32, qg.BF16)
    s, es, y, ey = want(c)
    run(c, S=c["residual"], Y=c["X"])
    ref.check(c["residual"], s, es)
    ref.check(c["X"], y, ey)


@pytest.mark.parametrize("kind", [qg.NORM_RMS, qg.NORM_LAYER])
@pytest.mark.parametrize("x_dtype,s_dtype", [(qg.BF16, qg.F32), (qg.F16, qg.F16), (qg.F32, qg.BF16)])
@pytest.mark.parametrize("M,K", [(4000, 256), (4000, 320), (1500, 1088), (1000, 2240), (500, 4096), (460, 4160), (310, 5120), (310, 5184), (310, 6144), (310, 6208),
                                 (310, 8192)])
def test_more_rows_than_the_gpu_takes_at_once(M, K, x_dtype, s_dtype, kind):
    """Several pieces of a row to a thread; S over the residual."""
    c = make(M, K, kind, x_dtype, s_dtype, x_dtype, gate="row")
    s, es, y, ey = want(c)
    S, Y = run(c, S=c["residual"])
    ref.check(S, s, es)
    ref.check(Y, y, ey)


@pytest.mark.parametrize("kind", [qg.NORM_RMS, qg.NORM_LAYER])
def test_a_large_mean(kind):
    """Values 1000 +- 1: the variance is not the difference of two sums."""
    check(make(4, 4096, kind, qg.F32, qg.F32, qg.F32, post=0, gate="none", residual=False, mean=1000.0))


def test_rows_of_zeros_and_constants():
    c = make(3, 512, qg.NORM_LAYER, qg.BF16, qg.F32, qg.F32, post=0, gate="none", residual=False, affine="none")
    c["X"][0], c["X"][1] = 0, 5
    S, Y = run(c)
    assert not bool(S[0].any()) and not bool(Y[:2].any())      # the mean of equal values is exact: 5 * 512 / 512
    c["kind"] = qg.NORM_RMS
    check(c)


def test_nan_and_infinity_stay_in_their_rows():
    c = make(5, 512, qg.NORM_RMS, qg.BF16, qg.F32, qg.F32)
    c["X"][1, 3], c["X"][3, 500] = float("nan"), float("inf")
    s, es, y, ey = want(c)
    S, Y = run(c)
    good = torch.tensor([0, 2, 4], device=DEV)
    ref.check(S[good], s[good], es[good])
    ref.check(Y[good], y[good], ey[good])
    assert bool(torch.isnan(Y[1]).all()) and bool(torch.isnan(Y[3, 500]))


def test_rows_past_32_bits():
    M, K, ld = 17, 128, 1 << 28
    X = torch.empty(M * ld, dtype=torch.float16, device=DEV).view(M, ld)
    c = make(M, K, qg.NORM_RMS, qg.F16, qg.F16, qg.F16)
    X[:, :K] = c["X"]
    c["X"] = X
    check(c)


def test_another_stream_and_a_graph():
    c = make(33, 4096, qg.NORM_RMS, qg.BF16, qg.BF16, qg.BF16)
    S, Y = run(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        S2, Y2 = run(c)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(S, S2) and torch.equal(Y, Y2)
    S3, Y3 = torch.zeros_like(S), torch.zeros_like(Y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, S=S3, Y=Y3)
    for scale in (1.0, 2.0):
        c["X"].copy_((c["X"].float() * scale).bfloat16())
        graph.replay()
        s, es, y, ey = want(c)
        ref.check(S3, s, es)
        ref.check(Y3, y, ey)
