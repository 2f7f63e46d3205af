"""The bf16 base side in float64 on the CPU, from its definition, and the error each output may have.

Bounds count roundings: bf16 is off by at most 2^-8 of a value, an fp32 operation by 2^-24 (2^-23
where it may truncate)."""
import math

import torch

BF, D = torch.bfloat16, torch.float64
NEG = float("-inf")
GATED = ("silu_mul", "swiglu_clamp")


# ---------------------------------------------------------------- routing

def route(logits, topk, scoring="softmax", bias=None, n_group=1, topk_group=1, group_top=1,
          renormalize=True, scale=1.0):
    """(ids, weights) by the definition, a row at a time in Python's floats (float64)."""
    ids, weights = [], []
    b = None if bias is None else bias.double().tolist()
    for x in logits.double().tolist():
        E = len(x)
        live = [v == v and v > NEG for v in x]
        nan = any(v != v for v in x)
        m = max([v for v, ok in zip(x, live) if ok], default=0.0)

        def grow(v, ref):  # exp(v - ref), also where both are the same infinity
            return 1.0 if v == ref else math.exp(v - ref)
        if scoring == "softmax":
            e = [grow(v, m) if ok else 0.0 for v, ok in zip(x, live)]
            total = math.fsum(e)
            s = [v / total if total else 0.0 for v in e]
        else:
            s = [0.0 if not ok else 1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v, ok in zip(x, live)]
        if b is not None:
            key = [u + v for u, v in zip(s, b)]
            nan |= any(ok and k != k for ok, k in zip(live, key))
        else:
            key = list(s) if group_top == 2 else list(x)
        key = [k if ok and k == k else NEG for k, ok in zip(key, live)]
        size = E // n_group
        score = []
        for g in range(n_group):
            best = sorted(key[g * size:(g + 1) * size], reverse=True)[:group_top]
            score.append(sum(k for k in best if k > NEG) if best[0] > NEG else NEG)
        kept = sorted(range(n_group), key=lambda g: (-score[g], g))[:topk_group]
        left = [i for i in range(E) if i // size in kept and key[i] > NEG]
        picks = sorted(left, key=lambda i: (-key[i], i))[:topk]
        if renormalize and picks:
            top = max(x[i] for i in picks)
            if scoring == "softmax":
                w = [grow(x[i], top) for i in picks]
            else:  # exp(x) / (1 + exp(x)), all times exp(-c)
                c = min(top, 0.0)
                w = [1 / (1 + math.exp(-x[i])) if x[i] > 0 else grow(x[i], c) / (1 + math.exp(x[i]))
                     for i in picks]
            total = math.fsum(w)
            w = [v / total if total else 0.0 for v in w]
        else:
            w = [s[i] for i in picks]
        w = [float("nan") if nan else v * scale for v in w]
        fill = topk - len(picks)
        ids.append(picks + [-1] * fill)
        weights.append(w + [float("nan") if nan else 0.0] * fill)
    return (torch.tensor(ids, dtype=torch.int32).view(-1, topk),
            torch.tensor(weights, dtype=D).view(-1, topk))


def check_route(got, want, spread):
    """`spread`: the largest |x - reference| of an exponential among the picks.  Its argument is off by
    2^-24 of itself; then come the exponential (2^-22), up to 22 additions, a product and two quotients.
    Below 2^-126 fp32 may keep nothing."""
    ids, w = (t.cpu() for t in got)
    assert torch.equal(ids, want[0]), f"ids differ in {int((ids != want[0]).any(1).sum())} rows"
    tol = (spread + 4 + 22 + 3) * 2.0 ** -24 * want[1].abs() + 2.0 ** -126
    nan = torch.isnan(want[1])
    assert torch.equal(torch.isnan(w), nan)
    err = (w.to(D) - want[1]).abs()[~nan]
    assert torch.all(err <= tol[~nan]), f"weights: worst {(err / tol[~nan]).max():.3f} of the bound"


# ---------------------------------------------------------------- products

def sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def activate(z, act):
    if act is None:
        return z
    if act == "silu":
        return z * sigmoid(z)
    if act == "gelu_tanh":
        return z * sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    g, u = z.chunk(2, -1)
    if act == "silu_mul":
        return g * sigmoid(g) * u
    g, u = torch.clamp(g, max=7.0), torch.clamp(u, -7.0, 7.0)
    return g * sigmoid(1.702 * g) * (u + 1)


def activate_err(z, ez, act):
    """Error of the activation's output when z is known to ez, and fp32 computes it.

    z sigmoid(c z) has a slope within [-0.13, 1.13].  The hardware's exponential and reciprocal
    leave a sigmoid of v off by (3 + |v|) 2^-23 of itself; four more roundings; a sigmoid below
    2^-126 may be 0."""
    step = 2.0 ** -23

    def unit(v, ev, arg):
        return 1.13 * ev + (v * sigmoid(arg)).abs() * (5 + arg.abs()) * step + 2.0 ** -126 * v.abs()
    if act is None:
        return ez
    if act == "silu":
        return unit(z, ez, z)
    if act == "gelu_tanh":
        # the argument's own five roundings on top
        arg = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        return unit(z, ez, arg) + (z * sigmoid(arg)).abs() * 5 * step * arg.abs()
    g, u = z.chunk(2, -1)
    eg, eu = ez.chunk(2, -1)
    if act == "silu_mul":
        f, ef = g * sigmoid(g), unit(g, eg, g)
        return ef * (u.abs() + eu) + (f.abs() + ef) * eu + (f * u).abs() * step
    g, u = torch.clamp(g, max=7.0), torch.clamp(u, -7.0, 7.0)
    f, ef = g * sigmoid(1.702 * g), unit(g, eg, 1.702 * g)
    eu = eu + (u + 1).abs() * step
    return ef * ((u + 1).abs() + eu) + (f.abs() + ef) * eu + (f * (u + 1)).abs() * step


def product(x, w, bias=None, delta=None, act=None, residual=None, wt=None):
    """(y, its error before it is rounded) of x [M, K], w [N, K]: fp32 sums in any order are off by
    2^-23 a term of the sum over magnitudes at most."""
    x, w = x.to(D), w.reshape(-1, w.shape[-1]).to(D)
    K = x.shape[1]
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, mag = z + bias.to(D), mag + bias.to(D).abs()
    if wt is not None:
        z, mag = z * wt.to(D)[:, None], mag * wt.to(D).abs()[:, None]
    if delta is not None:
        z, mag = z + delta.to(D), mag + delta.to(D).abs()
    ez = (K + 4) * 2.0 ** -23 * mag
    y, ey = activate(z, act), activate_err(z, ez, act)
    if residual is not None:
        y = y + residual.to(D)
        ey = ey + 2.0 ** -23 * y.abs()
    return y, ey


def check(got, ref, err):
    """`got` (bf16 or fp32) against ref known to err: its own rounding on top."""
    half = {BF: 2.0 ** -8, torch.float32: 2.0 ** -24}[got.dtype]
    got = got.cpu().to(D)
    tol = half * (ref.abs() + err) + err + 2.0 ** -133
    off = (got - ref).abs()
    assert torch.all(off <= tol), f"worst {(off / tol).max():.3f} of the bound"


def whole(g, *shape, most=4):
    """Small whole numbers: a product's sums stay whole and below 2^24, so fp32 holds them exactly and
    a bf16 output is the exact value's rounding."""
    return torch.randint(-most, most + 1, shape, generator=g).to(BF)


def rows(g, M, K):
    return (torch.randn((M, K), generator=g) * (1 + 30 * (torch.rand(K, generator=g) < 0.01))).to(BF)


def weights(g, *shape):
    return (torch.randn(shape, generator=g) * shape[-1] ** -0.5).to(BF)


# ---------------------------------------------------------------- combine

def combine(y, wt=None, ids=None, E=0, residual=None):
    """(out, its error before it is rounded)."""
    f = torch.ones(y.shape[:2], dtype=D) if wt is None else wt.to(D)
    v = y.to(D) * f[:, :, None]
    if ids is not None:
        v = torch.where(((ids >= 0) & (ids < E))[:, :, None], v, torch.zeros_like(v))
    out, mag = v.sum(1), v.abs().sum(1)
    if residual is not None:
        out, mag = out + residual.to(D), mag + residual.to(D).abs()
    return out, (y.shape[1] + 1) * 2.0 ** -24 * mag
