"""A mixture-of-experts feed-forward layer with 4-bit weights and activations, as a server runs it.

    python examples/moe_layer.py [--tokens 256] [--experts 32] [--topk 4] [--hidden 2560] [--inner 2560] [--format mxfp4]

Per call, for hidden states x [tokens][hidden] and router logits [tokens][experts]:

    route      each token's top-k experts and weights, and the expert-sorted order of the pairs
    quantize   each pair's hidden state, gathered into that order, to 4 bits
    gate / up  the experts' first projections with SwiGLU, [pairs][inner]
    quantize   the inner activations to 4 bits
    down       the experts' second projections, [pairs][hidden]
    combine    each token's weighted sum of its experts' rows, added to x

The group sizes never leave the GPU, so a step can be captured into a CUDA graph. With
``--format bf16`` the same layer runs on 16-bit weights, without the quantization steps.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_quantized_gemm_gb300 as qg  # noqa: E402

FORMATS = {"mxfp4": qg.FMT_MXFP4, "nvfp4": qg.FMT_NVFP4, "bf16": qg.FMT_BF16}


def pack_experts(w, fmt):
    """Expert weights w [E][N][K] (float32 or bf16) as (codes, tiled block scales, channel scales)."""
    E, N, K = w.shape
    if fmt == qg.FMT_BF16:
        return w.to(torch.bfloat16).contiguous(), None, None
    one = qg.qgemm_fp4_scales_bytes(N, K, fmt, qg.SCALES_TILED)
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(E, one, dtype=torch.uint8, device=w.device)
    row = torch.empty(E, (N + 3) // 4 * 4, dtype=torch.float32, device=w.device)      # (rows 16-byte aligned)
    for e in range(E):
        qg.qgemm_fp4_quant(N, K, w[e].to(torch.float32).contiguous(), qg.F32, K, N, None, fmt, qg.SCALES_TILED, codes[e], scales[e], row[e])
    return codes, scales, row[:, :N].contiguous() if fmt == qg.FMT_NVFP4 else None


class MoeLayer:
    """Weights, and the buffers of one step for up to `tokens` tokens."""

    def __init__(self, w1, w2, topk, tokens, fmt=qg.FMT_MXFP4):
        # w1 [E][2 inner][hidden], gate and up channels alternating; w2 [E][hidden][inner]
        self.E, two, self.hidden = w1.shape
        self.inner, self.k, self.fmt, self.tokens = two // 2, topk, fmt, tokens
        self.w1, self.w2 = pack_experts(w1, fmt), pack_experts(w2, fmt)
        dev, pairs = w1.device, tokens * topk
        empty = lambda *s, dtype: torch.empty(*s, dtype=dtype, device=dev)
        self.expert, self.slot = empty(tokens, topk, dtype=torch.int32), empty(tokens, topk, dtype=torch.int32)
        self.weight, self.row = empty(tokens, topk, dtype=torch.float32), empty(pairs, dtype=torch.int32)
        self.offsets = empty(self.E + 1, dtype=torch.int32)
        self.scratch = empty(max(qg.qgemm_moe_route_workspace_bytes(tokens, self.E, topk), 16), dtype=torch.uint8)
        self.h, self.y = empty(pairs, self.inner, dtype=torch.bfloat16), empty(pairs, self.hidden, dtype=torch.bfloat16)
        if fmt != qg.FMT_BF16:
            self.a = [self._activation(pairs, K, dev) for K in (self.hidden, self.inner)]

    def _activation(self, rows, K, dev):
        scales = torch.empty(qg.qgemm_fp4_scales_bytes(rows, K, self.fmt, qg.SCALES_ROWS), dtype=torch.uint8, device=dev)
        return (torch.empty(rows, K // 2, dtype=torch.uint8, device=dev), scales,
                torch.empty(rows, device=dev) if self.fmt == qg.FMT_NVFP4 else None)

    def _project(self, pairs, x, rows, step, w, act, out):
        """One projection of every pair: x's rows (gathered by `rows` if given) through the experts."""
        N, K = w[0].shape[1], x.shape[1]
        if self.fmt == qg.FMT_BF16:
            a, a_s, a_row = (x if rows is None else x.index_select(0, rows.clamp(min=0))), None, None
        else:
            a, a_s, a_row = self.a[step]
            qg.qgemm_fp4_quant(pairs, K, x, qg.BF16, K, x.shape[0], rows, self.fmt, qg.SCALES_ROWS, a, a_s, a_row)
        qg.qgemm_grouped_run(pairs, self.E, K, N, self.fmt, self.offsets, a, a_s, a_row, *w, None, act, out, qg.BF16)

    def __call__(self, x, logits, out):
        """out = x + the experts' weighted sum, for bf16 x [T][hidden] and float32 logits [T][E], T <= tokens."""
        T = x.shape[0]
        pairs = T * self.k
        row, h, y = self.row[:pairs], self.h[:pairs], self.y[:pairs]
        qg.qgemm_moe_route(T, self.E, self.k, logits, qg.F32, logits.stride(0), 1, self.expert, self.weight, self.slot, row,
                           self.offsets, self.scratch)
        self._project(pairs, x, row, 0, self.w1, qg.ACT_SWIGLU, h)
        self._project(pairs, h, None, 1, self.w2, qg.ACT_NONE, y)
        qg.qgemm_moe_combine(T, self.k, self.hidden, pairs, y, qg.BF16, self.slot, self.weight, x, out, qg.BF16)
        return out


def plain_layer(x, logits, w1, w2, topk):
    """The layer in float32, unquantized."""
    p, expert = torch.sort(torch.softmax(logits, -1), dim=-1, descending=True, stable=True)
    p, expert = p[:, :topk], expert[:, :topk]
    p = p / p.sum(-1, keepdim=True)
    out = x.float().clone()
    for e in range(w1.shape[0]):
        t, j = torch.where(expert == e)
        v = x[t].float() @ w1[e].float().T
        h = torch.nn.functional.silu(v[:, 0::2]) * v[:, 1::2]
        out.index_add_(0, t, p[t, j, None] * (h @ w2[e].float().T))
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--topk", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=2560)
    ap.add_argument("--inner", type=int, default=2560)
    ap.add_argument("--format", choices=sorted(FORMATS), default="mxfp4")
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    dev = "cuda"
    w1 = (torch.randn(a.experts, 2 * a.inner, a.hidden, device=dev) * a.hidden ** -0.5).bfloat16()
    w2 = (torch.randn(a.experts, a.hidden, a.inner, device=dev) * a.inner ** -0.5).bfloat16()
    layer = MoeLayer(w1, w2, a.topk, a.tokens, FORMATS[a.format])
    x = torch.randn(a.tokens, a.hidden, device=dev).bfloat16()
    logits = torch.randn(a.tokens, a.experts, device=dev)
    out = torch.empty_like(x)
    layer(x, logits, out)
    assert qg.qgemm_status() == 0
    want = plain_layer(x, logits, w1, w2, a.topk)
    delta = want - x.float()
    err = float((out.float() - want).norm() / delta.norm())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, logits, out)
    for _ in range(3):
        graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) * 1e3 / 20
    print(f"{a.format}: {a.tokens} tokens, {a.experts} experts, top {a.topk}, {a.hidden} -> {a.inner}: {us:.1f} us a step, "
          f"distance to the unquantized layer {err:.3f} of its contribution")
    return err


if __name__ == "__main__":
    main()
