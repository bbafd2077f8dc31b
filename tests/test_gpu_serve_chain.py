"""A served step around a layer, as the calls are used together: the rows' order by adapter, norm, the 4-bit layer, its
adapters, norm behind and in front, an Int4 layer, the last projection, log probabilities. Each step is held to its
definition in float64 on its inputs as stored; then the whole step is captured and replayed with other inputs."""
import pytest
import torch

import weight_quantized_gemm_gb300 as qg
from tests import _serve_ref as ref
from tests._util import ensure_built

pytestmark = pytest.mark.gpu
DEV = "cuda"
K, V, L, R = 512, 3001, 6, 16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


class Step:
    def __init__(self, M, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.M = M
        self.x, self.stream = randn(M, K).bfloat16(), 2 * randn(M, K)
        self.ids = torch.randint(-1, L, (M,), generator=g, device=DEV, dtype=torch.int32)
        self.token = torch.randint(V, (M,), generator=g, device=DEV, dtype=torch.int32)
        self.norms = [1 + 0.1 * randn(K) for _ in range(3)]
        # an MXFP4 layer, its adapters, an Int4 layer and a 16-bit projection to the vocabulary
        w = randn(K, K) * K ** -0.5
        self.w4, self.w4s = torch.empty(qg.qgemm_fp4_codes_bytes(K, K), dtype=torch.uint8, device=DEV), torch.empty(
            qg.qgemm_fp4_scales_bytes(K, K, qg.FMT_MXFP4, qg.SCALES_TILED), dtype=torch.uint8, device=DEV)
        qg.qgemm_fp4_pack(w, K, K, qg.FMT_MXFP4, self.w4, self.w4s)
        self.a, self.b = (randn(L, R, K) * K ** -0.5).bfloat16(), (0.2 * randn(L, K, R)).bfloat16()
        self.scale = 0.5 + torch.rand(L, generator=g, device=DEV)
        self.i4 = torch.empty(qg.qgemm_packed_bytes(K, K, qg.MODE_INT4), dtype=torch.uint8, device=DEV)
        self.i4t = torch.empty(qg.qgemm_table_bytes(K, K, qg.MODE_INT4, 64) // 4, device=DEV)
        qg.qgemm_pack(randn(K, K) * K ** -0.5, K, K, qg.MODE_INT4, 64, 0, self.i4, self.i4t)
        self.head = torch.empty(qg.qgemm_packed_bytes(K, V, qg.MODE_FLOAT, qg.BF16), dtype=torch.uint8, device=DEV)
        qg.qgemm_pack(randn(K, V) * 0.2, K, V, qg.MODE_FLOAT, 0, qg.BF16, self.head, None)
        empty = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
        self.row, self.offsets = empty(M, dt=torch.int32), empty(L + 1, dt=torch.int32)
        self.s1, self.y1, self.s2, self.y2, self.h, self.shared, self.i = empty(M, K, dt=torch.float32), empty(M, K), empty(M, K, dt=torch.float32), \
            empty(M, K), empty(M, K), empty(M, K), empty(M, K)
        self.codes, self.scales = empty(qg.qgemm_fp4_codes_bytes(M, K), dt=torch.uint8), empty(
            qg.qgemm_fp4_scales_bytes(M, K, qg.FMT_MXFP4, qg.SCALES_ROWS), dt=torch.uint8)
        self.logits = empty(M, V)
        self.logprob, self.entropy, self.top, self.top_logprob = empty(M, dt=torch.float32), empty(M, dt=torch.float32), empty(M, 4, dt=torch.int32), empty(
            M, 4, dt=torch.float32)
        wsb = max(qg.qgemm_workspace_bytes(M, K, n, m, b, qg.BF16, qg.BF16) for n, m, b in ((K, qg.MODE_INT4, 64), (V, qg.MODE_FLOAT, 0)))
        self.ws = empty(max(wsb, 16), dt=torch.uint8)

    def run(self):
        M = self.M
        qg.qgemm_lora_group(M, L, self.ids, self.row, self.offsets)
        qg.qgemm_norm_run(M, K, qg.NORM_RMS, 1e-6, self.x, qg.BF16, K, 1.0, 0, None, None, 0, self.stream, 1.0, self.s1, qg.F32, self.norms[0], None,
                          self.y1, qg.BF16)
        qg.qgemm_fp4_quant(M, K, self.y1, qg.BF16, K, M, None, qg.FMT_MXFP4, qg.SCALES_ROWS, self.codes, self.scales)
        qg.qgemm_fp4_run(M, K, K, qg.FMT_MXFP4, self.codes, self.scales, None, self.w4, self.w4s, None, None, qg.ACT_NONE, None, self.h, qg.BF16)
        self.shared.copy_(self.h)
        qg.qgemm_lora_run(M, K, K, L, R, qg.BF16, self.row, self.offsets, self.y1, K, self.a, self.b, None, self.scale, self.h, qg.BF16, K)
        qg.qgemm_norm_run(M, K, qg.NORM_RMS, 1e-6, self.h, qg.BF16, K, 0.5, 1, self.norms[1], None, 0, self.s1, 1.0, self.s2, qg.F32, self.norms[2],
                          None, self.y2, qg.BF16)
        qg.qgemm_run(M, K, K, qg.MODE_INT4, 64, self.y2, qg.BF16, self.i4, self.i4t, self.i, qg.BF16, self.ws)
        qg.qgemm_run(M, K, V, qg.MODE_FLOAT, 0, self.i, qg.BF16, self.head, None, self.logits, qg.BF16, self.ws)
        qg.qgemm_logprobs(M, V, self.logits, qg.BF16, V, 1.0, self.token, self.logprob, self.entropy, 4, self.top, self.top_logprob)

    def check(self):
        row, offsets = ref.group(self.ids.tolist(), L)
        assert self.row.tolist() == row and self.offsets.tolist() == offsets
        s, es, y, ey = ref.norm(self.x, 1, 1e-6, 1.0, 0, None, None, self.stream, 1.0, self.norms[0], None)
        ref.check(self.s1, s, es, "stream")
        ref.check(self.y1, y, ey, "norm")
        want, allow = ref.lora(self.shared, self.y1, self.a, self.b, self.ids.tolist(), None, self.scale)
        ref.check(self.h, want, allow, "adapters")
        s, es, y, ey = ref.norm(self.h, 1, 1e-6, 0.5, 1, self.norms[1], None, self.s1, 1.0, self.norms[2], None)
        ref.check(self.s2, s, es, "second stream")
        ref.check(self.y2, y, ey, "second norm")
        want = ref.logprobs(self.logits, 1.0, self.token, 4)
        assert torch.equal(self.top, want["top"])
        for n in ("logprob", "entropy", "top_logprob"):
            w = want[n]
            a = want["allow"] if w.dim() == 1 else want["allow"][:, None]
            ref.check(getattr(self, n), w, 2 * a * (1 + w.abs()), n)
        # the layers between are checked by tests of their own: here, that they are fed and not empty
        assert bool((self.shared != 0).any()) and bool((self.i != 0).any()) and bool(torch.isfinite(self.logits).all())


@pytest.mark.parametrize("M", [1, 9, 77, 2400])
def test_step(M):
    s = Step(M)
    s.run()
    torch.cuda.synchronize()
    assert qg.qgemm_status() == 0
    s.check()


@pytest.mark.parametrize("M", [3, 40])
def test_step_in_a_graph_with_other_inputs(M):
    s = Step(M)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (1, 2):
        t = Step(M, seed)
        for n in ("x", "stream", "ids", "token"):
            getattr(s, n).copy_(getattr(t, n))
        graph.replay()
        torch.cuda.synchronize()
        s.check()
    assert qg.qgemm_status() == 0
