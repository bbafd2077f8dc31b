"""The operators of a mixture-of-experts layer in 4-bit floating point, as measured cases.

Five operators that such a layer is made of, each with its plain form (elementary torch operations
in float32) and the library's call:

  quant    microscaled 4-bit quantization of activation rows, and back to the values it stands for
  linear   product of two 4-bit operands, with bias, activation and residual
  route    top-k expert choice of each token, with the expert-sorted order of the chosen pairs
  grouped  the experts' products over ragged groups of rows, in 4-bit or 16-bit operands
  combine  each token's weighted sum of its experts' output rows

Formats. A 4-bit value is e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte with
the even index in the low half. "mx": one e8m0 scale (a power of two) for each 32 values of a row.
"nv": one e4m3 scale for each 16 values, and one float32 scale for each row.
"""
import math

import numpy as np
import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"f32": 0, "f16": 1, "bf16": 2, "mx": 3, "nv": 4}     # the library's numbers of types and formats
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}
BLOCK = {"mx": 32, "nv": 16}
ROWS, TILED = 0, 1                                          # layouts of the block scales
E2M1 = torch.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0), device=DEV)
SIX = torch.full((), 6.0, device=DEV)      # a tensor, so that dividing by it is a division


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the activation rows of a few decoded tokens: the call's latency
        dict(name="quant_decode", op="quant", m=4, k=4096, fmt="mx", dtype="bf16"),
        # a long prompt's activations in front of the widest layer's output projection: bandwidth
        dict(name="quant_prefill", op="quant", m=16384, k=14336, fmt="nv", dtype="bf16"),
        # one token through a feed-forward projection: the weights' bytes
        dict(name="linear_decode", op="linear", m=1, k=4096, n=11008, fmt="mx", out="bf16", act="none", bias=False, residual=False),
        # an odd batch of decoded tokens through a down projection, added to the residual stream
        dict(name="linear_batch", op="linear", m=77, k=9728, n=2560, fmt="nv", out="bf16", act="none", bias=True, residual=True),
        # a prompt through the widest projection: the tensor cores
        dict(name="linear_prefill", op="linear", m=2048, k=4096, n=14336, fmt="mx", out="bf16", act="silu", bias=True, residual=False),
        # routing of a few decoded tokens: the call's latency
        dict(name="route_decode", op="route", t=8, e=64, k=8, dtype="bf16", renorm=True),
        # routing of a batch of long prompts
        dict(name="route_prefill", op="route", t=16384, e=128, k=8, dtype="f32", renorm=False),
        # sixteen decoded tokens at four experts each: most experts hold two rows, some none
        dict(name="grouped_decode", op="grouped", t=64, e=32, k=2560, n=9728, fmt="mx", out="bf16", act="none", bias=True, skew=0.5),
        # long prompts through the experts' gate and up projections, with SwiGLU
        dict(name="grouped_prefill", op="grouped", t=32768, e=32, k=2560, n=5120, fmt="mx", out="bf16", act="swiglu", bias=False, skew=0.5),
        # the same step in 16-bit weights with few experts, strongly uneven
        dict(name="grouped_bf16", op="grouped", t=4099, e=8, k=4096, n=2560, fmt="bf16", out="bf16", act="none", bias=False, skew=1.0),
        # a few decoded tokens' expert outputs, summed
        dict(name="combine_decode", op="combine", t=8, k=4, n=4096, dtype="bf16", residual=True),
        # long prompts' expert outputs, summed
        dict(name="combine_prefill", op="combine", t=16384, k=8, n=2560, dtype="bf16", residual=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _draw(rng)
    while 3072 in case.values():     # no configuration of the library has this size
        case = _draw(rng)
    return case


def _draw(rng):
    op = rng.choice(("quant", "linear", "route", "grouped", "combine"))
    if op == "quant":
        return dict(op=op, m=_log(rng, 1, 16384), k=64 * _log(rng, 4, 224), fmt=rng.choice(("mx", "nv")), dtype=rng.choice(("f32", "f16", "bf16")))
    if op == "linear":
        return dict(op=op, m=_log(rng, 1, 2048), k=64 * _log(rng, 8, 152), n=_log(rng, 500, 6000), fmt=rng.choice(("mx", "nv")),
                    out=rng.choice(("f32", "f16", "bf16")), act=rng.choice(("none", "relu", "silu", "gelu")), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    if op == "route":
        e = rng.choice((8, 16, 60, 64, 128, 256))
        return dict(op=op, t=_log(rng, 1, 16384), e=e, k=rng.randint(1, min(e, 8)), dtype=rng.choice(("f32", "f16", "bf16")), renorm=rng.random() < 0.5)
    if op == "grouped":
        act = rng.choice(("none", "silu", "swiglu"))
        return dict(op=op, t=_log(rng, 1, 16384), e=_log(rng, 4, 64), k=64 * _log(rng, 8, 64), n=2 * _log(rng, 256, 1280),
                    fmt=rng.choice(("mx", "nv", "bf16", "f16")), out=rng.choice(("f16", "bf16")), act=act, bias=rng.random() < 0.5,
                    skew=rng.choice((0.0, 0.5, 1.0)))
    return dict(op=op, t=_log(rng, 1, 16384), k=rng.randint(1, 8), n=8 * _log(rng, 64, 512), dtype=rng.choice(("f16", "bf16", "f32")), residual=rng.random() < 0.5)


def sizes(case):
    """The rows of each expert of a grouped case: a multinomial with log-normal expert weights."""
    g = np.random.default_rng([case["t"], case["e"], case["n"], case["k"]])
    w = np.exp(case["skew"] * g.standard_normal(case["e"]))
    return g.multinomial(case["t"], w / w.sum())


def _width(fmt):
    """Bytes of one value of an operand in this format, with its share of the block scales."""
    return {"mx": 0.5 + 1 / 32, "nv": 0.5 + 1 / 16, "bf16": 2, "f16": 2}[fmt]


def work(case):
    op, size = case["op"], {"f32": 4, "f16": 2, "bf16": 2}
    if op == "quant":      # the rows in, codes and scales out; codes and scales in, the values out
        n = case["m"] * case["k"]
        return {"bytes": int(2 * n * (size[case["dtype"]] + _width(case["fmt"]))), "flops": 4 * n}
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        out = size[case["out"]] * m * n
        return {"bytes": int(_width(case["fmt"]) * k * (m + n)) + out * (2 if case["residual"] else 1) + (4 * n if case["bias"] else 0),
                "flops": 2 * m * k * n}
    if op == "route":
        t, e, k = case["t"], case["e"], case["k"]
        return {"bytes": t * e * size[case["dtype"]] + 16 * t * k + 4 * (e + 1), "flops": 4 * t * e}
    if op == "grouped":
        t, k, n = case["t"], case["k"], case["n"]
        used = int((sizes(case) > 0).sum())
        cols = n // 2 if case["act"] == "swiglu" else n
        return {"bytes": int(_width(case["fmt"]) * k * (t + used * n)) + size[case["out"]] * t * cols + 4 * (case["e"] + 1)
                + (4 * used * n if case["bias"] else 0), "flops": 2 * t * k * n}
    t, k, n = case["t"], case["k"], case["n"]
    return {"bytes": size[case["dtype"]] * t * n * (k + 1 + (1 if case["residual"] else 0)) + 8 * t * k, "flops": 2 * t * k * n}


# ---------------------------------------------------------------- the formats, in float32
def pow2(e):
    """2**e for whole e from -126 to 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def quantize(x, fmt):
    """Rows of float32 as (codes [.., K/2], block scales [.., K/block], row scales [..] or None).

    mx: scale 2**(floor(log2(max)) - 2), the power of two that brings the block's largest value to
    [4, 8); nv: row scale 2**(floor(log2(row max)) - 10), block scale the e4m3 value nearest to the
    block's max / 6. The code is the nearest e2m1 value, ties to the even code, at most 6."""
    b = BLOCK[fmt]
    row = None
    if fmt == "nv":
        top = x.abs().amax(-1, keepdim=True)
        ge = (torch.frexp(top)[1] - 11).clamp(-116, 117)
        row = torch.where(top > 0, pow2(ge), torch.ones_like(top))
        x = x * torch.where(top > 0, pow2(-ge), torch.ones_like(top))
        row = row.squeeze(-1)
    x = x.unflatten(-1, (-1, b))
    top = x.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        se = torch.where(top > 0, (torch.frexp(top)[1] - 3).clamp(-127, 125), -127)
        scales = (se + 127).to(torch.uint8)
        a, step = (x * pow2(-se)).abs(), torch.ones_like(top)
    else:
        step = (top / SIX).clamp(max=448).to(torch.float8_e4m3fn)
        scales = step.view(torch.uint8)
        step = step.to(torch.float32)
        a = torch.where(step > 0, x.abs(), torch.zeros_like(x))
    mag = ((a > 0.25 * step).to(torch.uint8) + (a >= 0.75 * step) + (a > 1.25 * step) + (a >= 1.75 * step)
           + (a > 2.5 * step) + (a >= 3.5 * step) + (a > 5 * step))
    code = (mag + 8 * ((x < 0) | ((x == 0) & torch.signbit(x))).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], scales.squeeze(-1), row


def values(codes, scales, row, fmt):
    """The float32 values that codes, block scales and row scales stand for."""
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = E2M1.index_select(0, both.flatten().to(torch.int32)).view(both.shape).unflatten(-1, (-1, BLOCK[fmt]))
    if fmt == "mx":
        s = torch.where(scales == 0, 2.0 ** -127, (scales.to(torch.int32) << 23).view(torch.float32))
    else:
        s = scales.view(torch.float8_e4m3fn).to(torch.float32)
    v = (v * s.unsqueeze(-1)).flatten(-2)
    return v if row is None else v * row.unsqueeze(-1)


def pitch(k, fmt):
    """Bytes between two rows of block scales: a multiple of 16."""
    return -(-(k // BLOCK[fmt]) // 16) * 16


def by_rows(scales, k, fmt):
    """Block scales [rows, K/block] as the library reads an activation's: rows of pitch() bytes."""
    out = torch.zeros(scales.shape[0], pitch(k, fmt), dtype=torch.uint8, device=scales.device)
    out[:, : scales.shape[1]] = scales
    return out


def by_tiles(scales):
    """Block scales [.., N, K/block] as the library reads a weight's: tiles of 128 rows x 4 scales,
    512 bytes each, where row r's four lie at 16 (r % 32) + 4 (r / 32); zeros past the ends."""
    *lead, n, kb = scales.shape
    nt, kt = -(-n // 128), -(-kb // 4)
    full = torch.zeros(*lead, nt * 128, kt * 4, dtype=torch.uint8, device=scales.device)
    full[..., :n, :kb] = scales
    t = full.view(*lead, nt, 4, 32, kt, 4)
    d = len(lead)
    return t.permute(*range(d), d, d + 3, d + 2, d + 1, d + 4).contiguous()


# ---------------------------------------------------------------- inputs
def activations(g, rows, k):
    """Normal values in which a few channels run some twenty times larger."""
    x = torch.randn(rows, k, generator=g, device=DEV)
    c = torch.rand(k, generator=g, device=DEV)
    return x * torch.where(c < 0.01, 20.0, 1.0)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case, op=op)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std

    def empty(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    if op == "quant":
        m, k, fmt, dt = case["m"], case["k"], case["fmt"], DTYPES[case["dtype"]]
        s["x"] = activations(g, m, k).to(dt)
        s["codes"], s["scales"] = empty(m, k // 2, dtype=torch.uint8), empty(m, pitch(k, fmt), dtype=torch.uint8)
        s["row"] = empty(m, dtype=torch.float32) if fmt == "nv" else None
        s["y"] = empty(m, k, dtype=dt)
    elif op == "linear":
        m, k, n, fmt = case["m"], case["k"], case["n"], case["fmt"]
        s["a"], s["as"], s["ar"] = quantize(activations(g, m, k), fmt)
        s["w"], s["ws"], s["wr"] = quantize(randn(n, k, std=0.02), fmt)
        s["as_rows"], s["ws_tiles"] = by_rows(s["as"], k, fmt), by_tiles(s["ws"])
        s["bias"] = randn(n, std=0.5) if case["bias"] else None
        s["residual"] = randn(m, n).to(DTYPES[case["out"]]) if case["residual"] else None
        s["c"] = empty(m, n, dtype=DTYPES[case["out"]])
    elif op == "route":
        t, e, k = case["t"], case["e"], case["k"]
        s["logits"] = (randn(t, e) + randn(1, e)).to(DTYPES[case["dtype"]])     # some experts are liked better
        s["expert"], s["slot"] = empty(t, k, dtype=torch.int32), empty(t, k, dtype=torch.int32)
        s["weight"] = empty(t, k, dtype=torch.float32)
        s["row"], s["offsets"] = empty(t * k, dtype=torch.int32), empty(e + 1, dtype=torch.int32)
        # block histograms of the pairs: at most one block of pairs to each of 160 thread blocks
        s["scratch"] = empty(4 * 160 * e + 256, dtype=torch.uint8)
    elif op == "grouped":
        t, e, k, n, fmt = case["t"], case["e"], case["k"], case["n"], case["fmt"]
        rows = sizes(case)
        s["most"] = int(rows.max())
        s["offsets"] = torch.tensor(np.concatenate(([0], np.cumsum(rows))), dtype=torch.int32, device=DEV)
        if fmt in BLOCK:
            s["a"], s["as"], s["ar"] = quantize(activations(g, t, k), fmt)
            s["w"], s["ws"], s["wr"] = quantize(randn(e, n, k, std=0.02), fmt)
            s["as_rows"], s["ws_tiles"] = by_rows(s["as"], k, fmt), by_tiles(s["ws"])
        else:
            s["a"], s["w"] = activations(g, t, k).to(DTYPES[fmt]), randn(e, n, k, std=0.02).to(DTYPES[fmt])
            s["as_rows"] = s["ar"] = s["ws_tiles"] = s["wr"] = None
        s["bias"] = randn(e, n, std=0.5) if case["bias"] else None
        s["c"] = empty(t, n // 2 if case["act"] == "swiglu" else n, dtype=DTYPES[case["out"]])
    else:
        t, k, n, dt = case["t"], case["k"], case["n"], DTYPES[case["dtype"]]
        s["y"] = randn(t * k, n).to(dt)
        s["slot"] = torch.randperm(t * k, generator=g, device=DEV).view(t, k).to(torch.int32)
        s["weight"] = torch.softmax(randn(t, k), -1)
        s["residual"] = randn(t, n).to(dt) if case["residual"] else None
        s["out"] = empty(t, n, dtype=dt)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return run_own(s) if own else PLAIN[s["op"]](s)


def run_own(s):
    import weight_quantized_gemm_gb300 as qg

    c, op = s["case"], s["op"]
    if op == "quant":
        m, k, fmt, dt = c["m"], c["k"], CODES[c["fmt"]], CODES[c["dtype"]]
        qg.qgemm_fp4_quant(m, k, s["x"], dt, k, m, None, fmt, ROWS, s["codes"], s["scales"], s["row"])
        qg.qgemm_fp4_dequant(m, k, fmt, ROWS, s["codes"], s["scales"], s["row"], s["y"], dt)
        return s["y"]
    if op == "linear":
        qg.qgemm_fp4_run(c["m"], c["k"], c["n"], CODES[c["fmt"]], s["a"], s["as_rows"], s["ar"], s["w"], s["ws_tiles"], s["wr"], s["bias"],
                         ACTS[c["act"]], s["residual"], s["c"], CODES[c["out"]])
        return s["c"]
    if op == "route":
        qg.qgemm_moe_route(c["t"], c["e"], c["k"], s["logits"], CODES[c["dtype"]], c["e"], int(c["renorm"]), s["expert"], s["weight"],
                           s["slot"], s["row"], s["offsets"], s["scratch"])
        return {n: s[n] for n in ("expert", "weight", "slot", "row", "offsets")}
    if op == "grouped":
        qg.qgemm_grouped_run(c["t"], c["e"], c["k"], c["n"], CODES[c["fmt"]], s["offsets"], s["a"], s["as_rows"], s["ar"], s["w"],
                             s["ws_tiles"], s["wr"], s["bias"], ACTS[c["act"]], s["c"], CODES[c["out"]])
        return s["c"]
    qg.qgemm_moe_combine(c["t"], c["k"], c["n"], c["t"] * c["k"], s["y"], CODES[c["dtype"]], s["slot"], s["weight"], s["residual"], s["out"],
                         CODES[c["dtype"]])
    return s["out"]


def activate(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "swiglu":       # columns 2j and 2j + 1 are the gate and the up projection of output j
        gate, up = v[..., 0::2], v[..., 1::2]
        return gate / (1 + torch.exp(-gate)) * up
    return v


def plain_quant(s):
    fmt = s["case"]["fmt"]
    return values(*quantize(s["x"].to(torch.float32), fmt), fmt).to(s["x"].dtype)


def plain_linear(s):
    c = s["case"]
    v = values(s["a"], s["as"], s["ar"], c["fmt"]) @ values(s["w"], s["ws"], s["wr"], c["fmt"]).T
    if s["bias"] is not None:
        v = v + s["bias"]
    v = activate(v, c["act"])
    if s["residual"] is not None:
        v = v + s["residual"].to(torch.float32)
    return v.to(s["c"].dtype)


def plain_route(s):
    c = s["case"]
    t, e, k = c["t"], c["e"], c["k"]
    x = s["logits"].to(torch.float32)
    order = torch.sort(x, dim=-1, descending=True, stable=True)      # ties: the lowest expert first
    top, expert = order.values[:, :k], order.indices[:, :k]
    over = torch.exp((top if c["renorm"] else x) - top[:, :1]).sum(-1, keepdim=True)
    weight = torch.exp(top - top[:, :1]) / over
    pairs = torch.sort(expert.reshape(-1), stable=True).indices      # by expert, then token
    slot = torch.empty(t * k, dtype=torch.int64, device=x.device)
    slot[pairs] = torch.arange(t * k, device=x.device)
    ends = torch.cumsum(torch.bincount(expert.reshape(-1), minlength=e), 0)
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device=x.device), ends))
    whole = dict(expert=expert, slot=slot.view(t, k), row=pairs // k, offsets=offsets)
    return dict({n: v.to(torch.int32) for n, v in whole.items()}, weight=weight)


def plain_grouped(s):
    c = s["case"]
    lo, hi = s["offsets"][:-1].long(), s["offsets"][1:].long()
    at = lo[:, None] + torch.arange(s["most"], device=lo.device)      # the rows of each expert, padded to the longest
    live = at < hi[:, None]
    if c["fmt"] in BLOCK:
        a, w = values(s["a"], s["as"], s["ar"], c["fmt"]), values(s["w"], s["ws"], s["wr"], c["fmt"])
    else:
        a, w = s["a"].to(torch.float32), s["w"].to(torch.float32)
    v = torch.bmm(a[at.clamp(max=c["t"] - 1)], w.transpose(1, 2))
    if s["bias"] is not None:
        v = v + s["bias"][:, None]
    return activate(v, c["act"])[live].to(s["c"].dtype)


def plain_combine(s):
    v = (s["y"][s["slot"].long()].to(torch.float32) * s["weight"][..., None]).sum(1)
    if s["residual"] is not None:
        v = v + s["residual"].to(torch.float32)
    return v.to(s["out"].dtype)


PLAIN = {"quant": plain_quant, "linear": plain_linear, "route": plain_route, "grouped": plain_grouped, "combine": plain_combine}


# ---------------------------------------------------------------- in 64 bits
def exact_values(codes, scales, row, fmt):
    """The values, by the fields of the formats."""
    both = torch.stack((codes % 16, codes // 16), -1).flatten(-2).to(torch.int16)
    sign, e, m = both // 8, (both // 2) % 4, (both % 2).double()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).clamp(min=0).double()))
    v = torch.where(sign == 1, -v, v)
    b = scales.to(torch.int16)
    if fmt == "mx":
        f = torch.exp2(b.double() - 127)
    else:
        f = torch.where(b < 8, b.double() / 512, (1 + (b % 8).double() / 8) * torch.exp2((b // 8).double() - 7))
    v = v * f.repeat_interleave(BLOCK[fmt], -1)
    return v if row is None else v * row.double()[..., None]


def exact_quant(x, fmt):
    """What quantizing the rows and reading them back gives, from the definition."""
    x = x.double()
    unit = torch.ones(x.shape[0], 1, 1, dtype=torch.float64, device=x.device)
    if fmt == "nv":
        top = x.abs().amax(-1)[:, None, None]
        unit = torch.where(top > 0, torch.exp2((torch.floor(torch.log2(top)) - 10).clamp(-116, 117)), unit)
    x = x.unflatten(-1, (-1, BLOCK[fmt])) / unit
    top = x.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        f = torch.where(top > 0, torch.exp2((torch.floor(torch.log2(top)) - 2).clamp(min=-127)), 0)
    else:
        r = (top / 6).float().double().clamp(max=448)
        q = torch.exp2(torch.floor(torch.log2(r)).clamp(min=-6) - 3)       # the distance of two e4m3 values there
        f = torch.where(r > 0, torch.round(r / q) * q, 0)
    a = torch.where(f > 0, x.abs() / f, 0)
    q = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.sign(x) * (torch.round(a / q) * q).clamp(max=6) * f * unit).flatten(-2)


def exact_activate(v, act):
    if act == "relu":
        return torch.where(v > 0, v, 0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "swiglu":
        v = v.unflatten(-1, (-1, 2))
        return v[..., 0] * torch.sigmoid(v[..., 0]) * v[..., 1]
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        return torch.cat([exact_quant(x, case["fmt"]) for x in s["x"].split(2048)])
    if op == "linear":
        a = exact_values(s["a"], s["as"], s["ar"], case["fmt"])
        v = a @ exact_values(s["w"], s["ws"], s["wr"], case["fmt"]).T
        v = exact_activate(v if s["bias"] is None else v + s["bias"].double(), case["act"])
        return v if s["residual"] is None else v + s["residual"].double()
    if op == "route":
        x = s["logits"].double()
        p = torch.softmax(x, -1)
        # larger first, and of equal ones the lower expert
        rank = (x[:, None, :] > x[:, :, None]).sum(-1) if case["t"] * case["e"] ** 2 < 1 << 30 else None
        if rank is None:
            rank = torch.cat([(y[:, None, :] > y[:, :, None]).sum(-1) for y in x.split(1024)])
        rank = rank * case["e"] + torch.arange(case["e"], device=x.device)
        expert = torch.argsort(rank, -1)[:, : case["k"]]
        w = torch.gather(p, 1, expert)
        return dict(expert=None, weight=w / w.sum(-1, keepdim=True) if case["renorm"] else w, slot=None, row=None, offsets=None)
    if op == "grouped":
        out = []
        for e, rows in enumerate(torch.arange(case["t"], device=DEV).split([int(n) for n in sizes(case)])):
            if case["fmt"] in BLOCK:
                pick = [None if v is None else v[rows] for v in (s["a"], s["as"], s["ar"])]
                a, w = exact_values(*pick, case["fmt"]), exact_values(s["w"][e], s["ws"][e], None if s["wr"] is None else s["wr"][e], case["fmt"])
            else:
                a, w = s["a"][rows].double(), s["w"][e].double()
            v = a @ w.T
            out.append(exact_activate(v if s["bias"] is None else v + s["bias"][e].double(), case["act"]))
        return torch.cat(out)
    v = torch.zeros(case["t"], case["n"], dtype=torch.float64, device=DEV)
    for j in range(case["k"]):
        v += s["weight"][:, j, None].double() * s["y"][s["slot"][:, j].long()].double()
    return v if s["residual"] is None else v + s["residual"].double()
