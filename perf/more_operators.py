"""The operators that stand around the linear layer in a served model, as measured cases.

Four operators, each with its plain form (elementary torch operations in float32) and the library's call:

  group     the rows of a batch in order of their request's low-rank adapter
  lora      the adapters' products, added to the shared projection's output
  norm      norm behind a block, gate, residual sum, and norm in front of the next block
  logprobs  log probabilities of given tokens, entropy, and the top alternatives
"""
import math

import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"f32": 0, "f16": 1, "bf16": 2}       # the library's numbers of types
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
KINDS = {"rms": 1, "layer": 2}
EPS = 1e-5


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the rows of a decoded batch, once a step: the call's latency
        dict(name="group_decode", op="group", m=64, l=32, none=0.1),
        # the tokens of a batch of long prompts
        dict(name="group_prefill", op="group", m=16384, l=200, none=0.1),
        # decoded tokens of sixteen requests at an attention projection: latency, and the adapters' bytes
        dict(name="lora_decode", op="lora", m=16, k=4096, n=4096, l=32, r=16, dtype="bf16", out="bf16", runs=1, none=0.0, ragged=False, pad=0),
        # an odd batch at a down projection, adapters of several ranks, float32 output
        dict(name="lora_batch", op="lora", m=77, k=9728, n=2560, l=24, r=64, dtype="f16", out="f32", runs=1, none=0.1, ragged=True, pad=0),
        # prompts of eight requests through the widest projection: the bytes of both sides
        dict(name="lora_prefill", op="lora", m=8192, k=4096, n=14336, l=8, r=16, dtype="bf16", out="bf16", runs=700, none=0.0, ragged=False, pad=0),
        # prompts of odd lengths at one part of a joined projection, wide adapters, some rows without one
        dict(name="lora_wide", op="lora", m=4099, k=2560, n=2560, l=5, r=128, dtype="bf16", out="bf16", runs=333, none=0.1, ragged=True, pad=2048),
        # a few decoded tokens in front of a projection: the call's latency
        dict(name="norm_decode", op="norm", m=4, k=4096, kind="rms", dtype="bf16", stream="bf16", out="bf16", post=False, gate="none", residual=True, affine="weight"),
        # long prompts: norm behind the block, gate of each channel, residual sum, norm in front of the next
        dict(name="norm_prefill", op="norm", m=16384, k=4096, kind="rms", dtype="bf16", stream="bf16", out="bf16", post=True, gate="channel", residual=True, affine="weight"),
        # an odd number of rows with a float32 residual stream and a gate of each value
        dict(name="norm_gated", op="norm", m=1023, k=9728, kind="layer", dtype="f16", stream="f32", out="f16", post=True, gate="row", residual=True, affine="both"),
        # one step of a few sequences over a large vocabulary: a row for many SMs
        dict(name="logprobs_decode", op="logprobs", t=4, v=128000, dtype="bf16", k=8, scale=1.25, masked=0.0),
        # an odd batch of float32 rows that start at odd places, a third of their logits masked
        dict(name="logprobs_batch", op="logprobs", t=77, v=50001, dtype="f32", k=20, scale=1.0, masked=0.3),
        # scoring whole prompts
        dict(name="logprobs_prefill", op="logprobs", t=4096, v=131072, dtype="bf16", k=5, scale=1.0, masked=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("group", "lora", "lora", "norm", "norm", "logprobs", "logprobs"))
    types = ("f32", "f16", "bf16")
    if op == "group":
        return dict(op=op, m=_log(rng, 1, 40000), l=_log(rng, 1, 1000), none=rng.choice((0.0, 0.1, 0.5)))
    if op == "lora":
        return dict(op=op, m=_log(rng, 1, 6000), k=64 * _log(rng, 8, 128), n=_log(rng, 500, 8192), l=_log(rng, 1, 64),
                    r=rng.choice((8, 16, 24, 32, 64, 96, 128, 256)), dtype=rng.choice(("f16", "bf16")), out=rng.choice(types),
                    runs=rng.choice((1, 50, 600)), none=rng.choice((0.0, 0.1, 0.5)), ragged=rng.random() < 0.5, pad=rng.choice((0, 0, 3, 512)))
    if op == "norm":
        k = 64 * _log(rng, 4, 224)
        return dict(op=op, m=min(_log(rng, 1, 16384), (1 << 25) // k), k=k, kind=rng.choice(("rms", "rms", "layer")), dtype=rng.choice(types),
                    stream=rng.choice(types), out=rng.choice(types), post=rng.random() < 0.5, gate=rng.choice(("none", "channel", "row")),
                    residual=rng.random() < 0.8, affine=rng.choice(("none", "weight", "both")))
    return dict(op=op, t=_log(rng, 1, 2000), v=_log(rng, 1000, 131072), dtype=rng.choice(types), k=rng.choice((0, 1, 5, 8, 20, 32)),
                scale=rng.choice((1.0, 1.25, 0.5)), masked=rng.choice((0.0, 0.0, 0.3, 0.999)))


def work(case):
    op = case["op"]
    if op == "group":
        return {"bytes": 8 * case["m"] + 4 * (case["l"] + 1), "flops": case["m"]}
    if op == "lora":
        m, k, n = case["m"], case["k"], case["n"]
        ids = adapters(case)
        used = sorted(set(i for i in ids if i >= 0))
        ranks = ranks_of(case)
        rows = sum(1 for i in ids if i >= 0)
        pairs = sum(ranks[i] for i in ids if i >= 0)
        return {"bytes": rows * (2 * k + 2 * SIZE[case["out"]] * n) + 2 * sum(ranks[i] for i in used) * (k + n) + 4 * (m + case["l"] + 1),
                "flops": 2 * pairs * (k + n)}
    if op == "norm":
        x, s, y = SIZE[case["dtype"]], SIZE[case["stream"]], SIZE[case["out"]]
        each = x + s + y + (s if case["residual"] else 0) + (x if case["gate"] == "row" else 0)
        once = (4 if case["post"] else 0) + {"none": 0, "weight": 4, "both": 8}[case["affine"]] + (x if case["gate"] == "channel" else 0)
        return {"bytes": case["m"] * case["k"] * each + case["k"] * once, "flops": 10 * case["m"] * case["k"]}
    return {"bytes": case["t"] * (case["v"] * SIZE[case["dtype"]] + 12 + 8 * case["k"]), "flops": 6 * case["t"] * case["v"]}


def adapters(case):
    """Each row's adapter (-1: none): runs of equal ids, as the tokens of one request are, of the mean length case["runs"]."""
    g = torch.Generator().manual_seed(case["m"] * 1000 + case["l"])
    m, runs = case["m"], case.get("runs", 1)
    count = m if runs == 1 else max(1, -(-m // runs))
    starts = torch.arange(m) if runs == 1 else torch.sort(torch.cat((torch.zeros(1, dtype=torch.int64), torch.randint(m, (count - 1,), generator=g)))).values
    ids = torch.randint(case["l"], (count,), generator=g)
    ids[torch.rand(count, generator=g) < case["none"]] = -1
    return ids[torch.searchsorted(starts, torch.arange(m), right=True) - 1].tolist()


def ranks_of(case):
    """Each adapter's rank: all of them R, or spread over 1 .. R."""
    if not case["ragged"]:
        return [case["r"]] * case["l"]
    g = torch.Generator().manual_seed(case["l"])
    return torch.randint(1, case["r"] + 1, (case["l"],), generator=g).tolist()


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case, op=op)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std

    def empty(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    if op == "group":
        m, l = case["m"], case["l"]
        ids = torch.randint(l, (m,), generator=g, device=DEV, dtype=torch.int32)
        s["adapter"] = torch.where(torch.rand(m, generator=g, device=DEV) < case["none"], -1, ids).to(torch.int32)
        s["row"], s["offsets"] = empty(m, dtype=torch.int32), empty(l + 1, dtype=torch.int32)
    elif op == "lora":
        m, k, n, l, r, dt = case["m"], case["k"], case["n"], case["l"], case["r"], DTYPES[case["dtype"]]
        # the same order as group's: it serves every projection of a step
        ids = torch.tensor(adapters(case), device=DEV)
        order = torch.sort(torch.where(ids < 0, l, ids), stable=True).indices
        counts = torch.bincount(ids[ids >= 0], minlength=l)
        s["offsets"] = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(counts, 0))).to(torch.int32)
        s["most"] = int(counts.max())
        s["row"] = torch.where(torch.arange(m, device=DEV) < counts.sum(), order, -1).to(torch.int32)
        s["x"] = (randn(m, k) * torch.where(torch.rand(k, generator=g, device=DEV) < 0.01, 10.0, 1.0)).to(dt)    # a few channels run larger
        s["a"] = randn(l, r, k, std=k ** -0.5).to(dt)
        s["b"] = randn(l, n, r, std=0.1).to(dt)
        s["rank"] = whole(ranks_of(case)) if case["ragged"] else None
        s["scale"] = 0.5 + torch.rand(l, generator=g, device=DEV)
        s["y"] = randn(m, n + case["pad"]).to(DTYPES[case["out"]])       # the shared projection's output
    elif op == "norm":
        m, k, dt = case["m"], case["k"], DTYPES[case["dtype"]]
        x = randn(m, k) * torch.where(torch.rand(k, generator=g, device=DEV) < 0.01, 20.0, 1.0)
        s["x"] = (x + 0.1).to(dt)
        s["post_weight"] = 1 + randn(k, std=0.1) if case["post"] else None
        s["gate"] = None if case["gate"] == "none" else torch.sigmoid(randn(k) if case["gate"] == "channel" else randn(m, k)).to(dt)
        s["residual"] = randn(m, k, std=4.0).to(DTYPES[case["stream"]]) if case["residual"] else None
        s["weight"] = None if case["affine"] == "none" else 1 + randn(k, std=0.1)
        s["bias"] = randn(k, std=0.1) if case["affine"] == "both" else None
        s["s"], s["y"] = empty(m, k, dtype=DTYPES[case["stream"]]), empty(m, k, dtype=DTYPES[case["out"]])
    else:
        t, v, k = case["t"], case["v"], case["k"]
        x = randn(t, v, std=2.0)
        if case["masked"]:
            x[torch.rand(t, v, generator=g, device=DEV) < case["masked"]] = -math.inf
        s["token"] = torch.randint(v, (t,), generator=g, device=DEV, dtype=torch.int32)
        x.scatter_(1, s["token"].long()[:, None], randn(t, 1, std=4.0) + 8)      # given tokens are likely ones
        s["logits"] = x.to(DTYPES[case["dtype"]])
        s["logprob"], s["entropy"] = empty(t, dtype=torch.float32), empty(t, dtype=torch.float32)
        s["top"], s["top_logprob"] = empty(t, k, dtype=torch.int32), empty(t, k, dtype=torch.float32)
    return s


R_SCALE, X_SCALE = 0.75, 1.5


# ---------------------------------------------------------------- one pass
def run(s):
    return run_own(s) if own else PLAIN[s["op"]](s)


def run_own(s):
    c, op = s["case"], s["op"]
    # the program that counted each adapter's rows has no call to make for a batch without any (neither has the plain form)
    if op == "lora" and not s["most"]:
        return s["y"]
    import weight_quantized_gemm_gb300 as qg

    if op == "group":
        qg.qgemm_lora_group(c["m"], c["l"], s["adapter"], s["row"], s["offsets"])
        return dict(row=s["row"], offsets=s["offsets"])
    if op == "lora":
        qg.qgemm_lora_run(c["m"], c["k"], c["n"], c["l"], c["r"], CODES[c["dtype"]], s["row"], s["offsets"], s["x"], c["k"], s["a"], s["b"],
                          s["rank"], s["scale"], s["y"], CODES[c["out"]], c["n"] + c["pad"])
        return s["y"]
    if op == "norm":
        k = c["k"]
        qg.qgemm_norm_run(c["m"], k, KINDS[c["kind"]], EPS, s["x"], CODES[c["dtype"]], k, X_SCALE, int(c["post"]), s["post_weight"], s["gate"],
                          k if c["gate"] == "row" else 0, s["residual"], R_SCALE, s["s"], CODES[c["stream"]], s["weight"], s["bias"], s["y"],
                          CODES[c["out"]])
        return dict(s=s["s"], y=s["y"])
    qg.qgemm_logprobs(c["t"], c["v"], s["logits"], CODES[c["dtype"]], c["v"], c["scale"], s["token"], s["logprob"], s["entropy"], c["k"],
                      s["top"], s["top_logprob"])
    return {n: s[n] for n in ("logprob", "entropy", "top", "top_logprob")}


def plain_group(s):
    c, ids = s["case"], s["adapter"]
    order = torch.sort(torch.where(ids < 0, c["l"], ids), stable=True).indices
    counts = torch.bincount(ids[ids >= 0], minlength=c["l"])
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device=ids.device), torch.cumsum(counts, 0)))
    row = torch.where(torch.arange(c["m"], device=ids.device) < counts.sum(), order, -1)
    return dict(row=row.to(torch.int32), offsets=offsets.to(torch.int32))


def plain_lora(s):
    c, y = s["case"], s["y"]
    if not s["most"]:
        return y
    lo, hi = s["offsets"][:-1].long(), s["offsets"][1:].long()
    at = lo[:, None] + torch.arange(s["most"], device=y.device)       # the rows of each adapter, padded to the most
    live = at < hi[:, None]
    rows = s["row"].long()[at.clamp(max=c["m"] - 1)].clamp(min=0)
    h = torch.bmm(s["x"][rows].to(torch.float32), s["a"].to(torch.float32).transpose(1, 2))
    if s["rank"] is not None:
        h = h * (torch.arange(c["r"], device=y.device) < s["rank"][:, None])[:, None, :]
    v = torch.bmm(h, s["b"].to(torch.float32).transpose(1, 2)) * s["scale"][:, None, None]
    rows = rows[live]
    part = y[:, : c["n"]]
    part[rows] = (part[rows].to(torch.float32) + v[live]).to(y.dtype)
    return y


def plain_normed(x, kind):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def plain_norm(s):
    c = s["case"]
    f = s["x"].to(torch.float32)
    if c["post"]:
        f = plain_normed(f, c["kind"]) * s["post_weight"]
    if s["gate"] is not None:
        f = f * s["gate"].to(torch.float32)
    f = f * X_SCALE
    if s["residual"] is not None:
        f = f + R_SCALE * s["residual"].to(torch.float32)
    y = plain_normed(f, c["kind"])
    if s["weight"] is not None:
        y = y * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return dict(s=f.to(s["s"].dtype), y=y.to(s["y"].dtype))


def plain_logprobs(s):
    c = s["case"]
    x = s["logits"].to(torch.float32) * c["scale"]
    d = x - x.amax(-1, keepdim=True)
    p = torch.exp(d)
    over = p.sum(-1)
    lse = torch.log(over)
    entropy = lse - (torch.where(p > 0, d, 0) * p).sum(-1) / over
    out = dict(logprob=torch.gather(d, 1, s["token"].long()[:, None])[:, 0] - lse, entropy=entropy)
    # larger first, of equal ones the lower index first: whole numbers in the order of the values, above the index
    bits = (s["logits"].to(torch.float32) + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64) * (1 << 20) + ((1 << 20) - 1 - torch.arange(c["v"], device=x.device))
    top = torch.topk(key, c["k"], dim=-1).indices
    found = torch.gather(d, 1, top)
    # a masked logit is no alternative
    out["top"] = torch.where(torch.isinf(found), -1, top).to(torch.int32)
    out["top_logprob"] = found - lse[:, None]
    return out


PLAIN = {"group": plain_group, "lora": plain_lora, "norm": plain_norm, "logprobs": plain_logprobs}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "group":
        return None
    s = prepare(case, seed)
    if op == "lora":
        y = s["y"].double()
        ids, ranks = torch.tensor(adapters(case), device=DEV), ranks_of(case)
        for l in range(case["l"]):
            rows = torch.nonzero(ids == l)[:, 0]
            r = ranks[l]
            y[rows, : case["n"]] += float(s["scale"][l]) * (s["x"][rows].double() @ s["a"][l, :r].double().T) @ s["b"][l, :, :r].double().T
        return y
    if op == "norm":
        def normed(v):
            if case["kind"] == "rms":
                return v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)
            var, mean = torch.var_mean(v, -1, correction=0, keepdim=True)
            return (v - mean) / torch.sqrt(var + EPS)

        sums, ys = [], []
        for rows in torch.arange(case["m"], device=DEV).split(2048):
            f = s["x"][rows].double()
            if case["post"]:
                f = normed(f) * s["post_weight"].double()
            if case["gate"] != "none":
                f = f * (s["gate"] if case["gate"] == "channel" else s["gate"][rows]).double()
            f = X_SCALE * f
            if case["residual"]:
                f = f + R_SCALE * s["residual"][rows].double()
            y = normed(f)
            y = y if s["weight"] is None else y * s["weight"].double()
            y = y if s["bias"] is None else y + s["bias"].double()
            sums.append(f)
            ys.append(y)
        return dict(s=torch.cat(sums), y=torch.cat(ys))
    out = dict(logprob=[], entropy=[], top_logprob=[])
    for x, token in zip(s["logits"].split(256), s["token"].split(256)):
        z = torch.log_softmax(x.double() * case["scale"], -1)
        out["logprob"].append(torch.gather(z, 1, token.long()[:, None])[:, 0])
        out["entropy"].append(torch.special.entr(torch.exp(z)).sum(-1))
        out["top_logprob"].append(torch.sort(z, -1, descending=True).values[:, : case["k"]])
    return dict({n: torch.cat(v) for n, v in out.items()}, top=None)
