"""The operators around the layers by their definitions, in float64, with bounds of what float32 may lose.

u = 2^-24 is half a float32 step of a value (relative). Each function returns (reference, allowance), where the
allowance bounds the float32 computation by the number of its roundings; the rounding to the output type (half a
step of the reference, out_half_step) is added by `check`."""
import math

import torch

U = 2.0 ** -24


def out_half_step(ref, dtype):
    """Half a step of ref in dtype (a subnormal's step is the smallest one)."""
    fi = torch.finfo(dtype)
    return ref.abs().clamp(min=fi.tiny) * (fi.eps / 2)


def check(got, ref, allow, what=""):
    assert got.shape == ref.shape, what
    g = got.double()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{what}: NaN at other places"
    inf = torch.isinf(ref)
    assert torch.equal(g[inf], ref[inf]), f"{what}: infinities at other places"
    allow = allow + out_half_step(ref, got.dtype) * (1 + 2.0 ** -10)      # (the reference may lie in the next binade)
    over = ((g - ref).abs() - allow)[fine]
    if over.numel():
        assert float(over.max()) <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} outside, by up to {float(over.max()):.3e}"


def group(adapter, L):
    ids = [int(i) for i in adapter]
    row = [m for l in range(L) for m in range(len(ids)) if ids[m] == l]
    offsets = [0]
    for l in range(L):
        offsets.append(offsets[-1] + sum(i == l for i in ids))
    return row + [-1] * (len(ids) - len(row)), offsets


def lora(y, x, a, b, adapter, rank, scale):
    """y [M][N], x [M][K], a [L][R][K], b [L][N][R]; adapter, rank and scale lists."""
    out, allow = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    K = x.shape[1]
    # Sums on the tensor cores: steps of 16 products, each at worst cut off instead of rounded (2 u of the absolute
    # sum), then up to 8 warps' and 8 blocks' parts. The middle values enter as 16-bit terms that hold 17 bits at least
    # where y is a 16-bit type, 22 where it is float32.
    terms = 2.0 ** -22 if y.dtype == torch.float32 or x.dtype == torch.float16 else 2.0 ** -17
    for l in sorted(set(adapter)):
        if not 0 <= l < a.shape[0]:
            continue
        r = min(max(rank[l], 0), a.shape[1]) if rank is not None else a.shape[1]
        rows = torch.tensor([m for m, i in enumerate(adapter) if i == l], device=y.device)
        al, bl, s = a[l, :r].double(), b[l, :, :r].double(), float(scale[l]) if scale is not None else 1.0
        h = x[rows].double() @ al.T
        out[rows] += s * (h @ bl.T)
        size = abs(s) * ((x[rows].double().abs() @ al.abs().T) @ bl.abs().T)
        n = K / 16 + 16 + 3 * (r / 16 + 1) + 4
        allow[rows] = size * (2 * U * n + terms) + U * out[rows].abs()
    return out, allow


def _stats(v, kind, eps, err):
    """Mean and factor of the norm in float64, and bounds of their errors where v is off by err: a sum of K values
    in up to 32 a thread, 5 + 32 joining steps (n roundings), then a product, a sum, and a root good to 2 u * 2."""
    n = 32 + 5 + 32 + 6
    mean = v.mean(-1, keepdim=True) if kind == 2 else torch.zeros_like(v[..., :1])
    e_mean = (n * U * v.abs().mean(-1, keepdim=True) + err.mean(-1, keepdim=True)) if kind == 2 else torch.zeros_like(mean)
    d = v - mean
    e_d = err + e_mean + U * (v.abs() + mean.abs())
    var = d.square().mean(-1, keepdim=True)
    inv = 1 / torch.sqrt(var + eps)
    e_var = n * U * var + (2 * d.abs() * e_d + e_d.square()).mean(-1, keepdim=True)
    e_inv = inv * (e_var * inv.square() / 2 * 1.5 + 4 * U)        # half the relative error of the square (1.5: second order)
    return d, inv, e_d, e_inv


def norm(x, kind, eps, x_scale, post, post_weight, gate, residual, r_scale, weight, bias):
    """(s, its allowance, y, its allowance)"""
    f, err = x.double(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    if post:
        d, inv, e_d, e_inv = _stats(f, kind, eps, err)
        w = post_weight.double() if post_weight is not None else 1.0
        f = d * inv * w
        err = (e_d * inv + d.abs() * e_inv) * (w.abs() if post_weight is not None else 1.0) + 3 * U * f.abs()
    if gate is not None:
        f = f * gate.double()
        err = err * gate.double().abs() + U * f.abs()
    f = f * x_scale
    err = err * abs(x_scale) + U * f.abs()
    if residual is not None:
        f = f + r_scale * residual.double()
        err = err + U * f.abs()
    d, inv, e_d, e_inv = _stats(f, kind, eps, err)
    y = d * inv
    e_y = e_d * inv + d.abs() * e_inv + 2 * U * y.abs()
    if weight is not None:
        y, e_y = y * weight.double(), e_y * weight.double().abs()
    if bias is not None:
        y = y + bias.double()
    return f, err, y, e_y + U * y.abs()


def logprobs(logits, scale, token, k):
    """dict of logprob, entropy, top, top_logprob, and `allow`, what they may be off by (absolute)."""
    x = logits.double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    T, V = x.shape
    out = dict(logprob=[], entropy=[], top=[], top_logprob=[], allow=[])
    for i in range(T):
        z, m = x[i], x[i].max()
        order = torch.sort(z, descending=True, stable=True)
        if m == -math.inf:
            lp, h, S = torch.full_like(z, -math.inf), 0.0, 1.0
        elif m == math.inf:
            c = int((z == m).sum())
            lp, h, S = torch.where(z == m, -math.log(c), -math.inf), math.log(c), float(c)
        else:
            d = (z - m) * scale
            p = torch.exp(d)
            S = float(p.sum())
            lp = d - math.log(S)
            h = math.log(S) - float((torch.where(p > 0, d, 0) * p).sum()) / S
        ids = [int(j) for j in order.indices[:k] if lp[j] > -math.inf]
        t = int(token[i]) if token is not None else -1
        out["logprob"].append(float(lp[t]) if 0 <= t < V else 0.0)
        out["entropy"].append(h)
        out["top"].append(ids + [-1] * (k - len(ids)))
        out["top_logprob"].append([float(lp[j]) for j in ids] + [-math.inf] * (k - len(ids)))
        # S: a thread's sum of V / 512 terms (a cluster's of fewer), two halves, 5 + 16 + 8 joining steps; each term's
        # 2^t is good to 2^-22, with t off by 2 u |t|, three times over (the thread's, block's and row's reference).
        # The terms with a large |t| weigh little: sum p |t| / S is at most ln V + 1.
        off = (V / 512 + 40) * U + 3 * (2.0 ** -22 + 2 * U * (math.log(V) + 1 + 8))
        out["allow"].append(off)
    return {n: torch.tensor(v, dtype=torch.int32 if n == "top" else torch.float64, device=logits.device) for n, v in out.items()}
