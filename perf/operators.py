"""The 8-bit base side of a MoE-LoRA layer: cases, inputs, plain forms and work of its operators.

    rms_norm   residual addition + root-mean-square norm, e4m3 rows with one fp32 scale per
               block of 128 columns, and the bf16 rows that the LoRA side reads
    silu_mul   silu(gate) * up of a projection's two slices, e4m3 rows with scales and bf16 rows
    gemm       e4m3 x e4m3 product with a scale per (row, 128 of K) and per (128 columns, 128 of K)
    moe_gemm   the same product over routed (token, k) pairs, grouped by expert in the layout of
               the align step

Where `own` is false, `run` computes each in elementary torch operations in 32 bits; where it is
true it calls the library.
"""

import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
MIN_AMAX = 2.0 ** -40  # a block whose largest magnitude is below this is scaled as if it were this
BLOCK = 128


def _cdiv(a, b):
    return -(-a // b)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the norm before a 20b-like decode layer: 16 sequences, one token each
        dict(name="norm decode 16x2880", op="rms_norm", M=16, H=2880, residual=True),
        # a ragged chunk of a prompt, the first layer (nothing to add yet)
        dict(name="norm chunk 777x2048", op="rms_norm", M=777, H=2048, residual=False),
        # a large prefill batch
        dict(name="norm prefill 16384x4096", op="rms_norm", M=16384, H=4096, residual=True),
        # the activation between w13 and w2 of a 20b-like decode layer (16 tokens x top-4)
        dict(name="silu decode 64x2880", op="silu_mul", P=64, I=2880),
        # the same for a Qwen3-like prefill (8192 tokens x top-8)
        dict(name="silu prefill 65536x768", op="silu_mul", P=65536, I=768),
        # the qkv projection of one sequence's next token: the weights are all there is to read
        dict(name="gemm token 1x4096x3x4096", op="gemm", M=1, K=4096, Ns=4096, S=3),
        # a ragged chunk whose K ends inside a scale block
        dict(name="gemm chunk 333x2880x2880", op="gemm", M=333, K=2880, Ns=2880, S=1),
        # the qkv projection of a 4096-token prefill
        dict(name="gemm prefill 4096x4096x3x4096", op="gemm", M=4096, K=4096, Ns=4096, S=3),
        # 20b-like decode, gate and up projections of 16 tokens: every routed expert's weights
        dict(name="moe decode w13 20b", op="moe_gemm", M=16, K=2880, Ns=2880, S=2, E=32, topk=4,
             block_m=16, x_per_pair=False, mul=False, zipf=0.0, drop=0.0),
        # 120b-like decode, down projection of 8 tokens, routed weight applied
        dict(name="moe decode w2 120b", op="moe_gemm", M=8, K=2880, Ns=2880, S=1, E=128, topk=4,
             block_m=16, x_per_pair=True, mul=True, zipf=0.0, drop=0.0),
        # 120b-like prefill, down projection: 64 rows an expert on average
        dict(name="moe prefill w2 120b", op="moe_gemm", M=2048, K=2880, Ns=2880, S=1, E=128,
             topk=4, block_m=64, x_per_pair=True, mul=True, zipf=0.0, drop=0.0),
        # Qwen3-like prefill, gate and up projections, skewed routing, some pairs' experts on
        # another rank
        dict(name="moe prefill w13 qwen3", op="moe_gemm", M=8192, K=2048, Ns=768, S=2, E=128,
             topk=8, block_m=128, x_per_pair=False, mul=False, zipf=1.2, drop=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, step):
    """A multiple of `step`, its logarithm uniform in [lo, hi]."""
    return max(step, _log(rng, lo, hi) // step * step)


def draw(rng: random.Random):
    op = rng.choice(["rms_norm", "silu_mul", "gemm", "moe_gemm", "moe_gemm", "gemm"])
    if op == "rms_norm":
        return dict(op=op, M=_log(rng, 1, 16384), H=_mult(rng, 128, 4096, 8),
                    residual=rng.random() < 0.7)
    if op == "silu_mul":
        return dict(op=op, P=_log(rng, 1, 32768), I=_mult(rng, 64, 1536, 8))
    if op == "gemm":
        return dict(op=op, M=_log(rng, 1, 4096), K=_mult(rng, 256, 4096, 16),
                    Ns=_mult(rng, 256, 4096, 8), S=rng.choice([1, 2, 3]))
    E = rng.choice([8, 16, 32, 64, 128])
    topk = rng.choice([1, 2, 4, 8])
    M = _log(rng, 1, 4096)
    rows = M * topk / E
    block_m = 16 if rows <= 16 else rng.choice([16, 32]) if rows < 32 else rng.choice([32, 64, 128])
    return dict(op=op, M=M, K=_mult(rng, 256, 2880, 16), Ns=_mult(rng, 256, 1536, 8),
                S=rng.choice([1, 2]), E=E, topk=topk, block_m=block_m,
                x_per_pair=rng.random() < 0.5, mul=rng.random() < 0.5,
                zipf=rng.choice([0.0, 0.8, 1.2]), drop=rng.choice([0.0, 0.1]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _rows(g, M, K):
    """Activations as 8-bit rows: a few wide channels, as hidden states have."""
    v = _randn(g, M, K) * (1 + 8 * (torch.rand(K, device="cuda", generator=g) < 0.01))
    nb = _cdiv(K, BLOCK)
    b = torch.nn.functional.pad(v, (0, nb * BLOCK - K)).view(M, nb, BLOCK)
    s = b.abs().amax(2).clamp(min=MIN_AMAX) / F8_MAX
    q = (b / s[:, :, None]).reshape(M, nb * BLOCK)[:, :K].to(F8)
    return q.contiguous(), s.t().contiguous()  # [M, K], [nb, M]


def _weights(g, E, S, Ns, K):
    """Weights in 8 bits, a scale per 128 x 128 block of each slice."""
    nb, kb = _cdiv(Ns, BLOCK), _cdiv(K, BLOCK)
    q = torch.empty((E, S, Ns, K), dtype=F8, device="cuda")
    s = torch.empty((E, S, nb, kb), device="cuda")
    for e in range(E):
        v = torch.nn.functional.pad(_randn(g, S, Ns, K) * K ** -0.5,
                                    (0, kb * BLOCK - K, 0, nb * BLOCK - Ns))
        b = v.view(S, nb, BLOCK, kb, BLOCK)
        s[e] = b.abs().amax((2, 4)).clamp(min=MIN_AMAX) / F8_MAX
        b = b / s[e][:, :, None, :, None]
        q[e] = b.reshape(S, nb * BLOCK, kb * BLOCK)[:, :Ns, :K].to(F8)
    return q, s


def _route(g, M, topk, E, zipf, drop):
    """Distinct experts per token, popularity by Zipf's law; -1 where an expert is elsewhere."""
    pop = -zipf * torch.log(torch.arange(1, E + 1, device="cuda").float())
    pop = pop[torch.randperm(E, device="cuda", generator=g)]
    u = torch.rand((M, E), device="cuda", generator=g).clamp(1e-7, 1 - 1e-7)
    ids = torch.topk(pop - torch.log(-torch.log(u)), topk, dim=1).indices.to(torch.int32)
    gone = torch.rand((M, topk), device="cuda", generator=g) < drop
    return torch.where(gone, torch.full_like(ids, -1), ids).contiguous()


def _align(ids, E, block_m):
    """The align step's layout for one slot: pairs by expert, each group padded to block_m."""
    flat = ids.reshape(-1).long()
    numel = flat.numel()
    cap = _cdiv(numel + min(E, numel) * (block_m - 1), block_m) * block_m
    kept = (flat >= 0).nonzero().reshape(-1)
    e, order = torch.sort(flat[kept], stable=True)
    pairs = kept[order]
    count = torch.bincount(e, minlength=E)
    padded = (count + block_m - 1) // block_m * block_m
    start = torch.cumsum(padded, 0) - padded
    first = torch.cumsum(count, 0) - count
    at = start[e] + torch.arange(pairs.numel(), device="cuda") - first[e]
    srt = torch.full((1, cap), numel, dtype=torch.int32, device="cuda")
    srt[0, at] = pairs.int()
    eids = torch.zeros((1, cap // block_m), dtype=torch.int32, device="cuda")
    blk = torch.repeat_interleave(torch.arange(E, device="cuda"), padded // block_m)
    eids[0, :blk.numel()] = blk.int()
    return srt, eids, padded.sum().int().reshape(1), cap


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    bf = torch.bfloat16
    if c["op"] == "rms_norm":
        M, H = c["M"], c["H"]
        nb = _cdiv(H, BLOCK)
        return dict(case=c, x=_randn(g, M, H).to(bf),
                    residual=(4 * _randn(g, M, H)).to(bf) if c["residual"] else None,
                    weight=(1 + 0.2 * _randn(g, H)).to(bf), eps=1e-6,
                    y=torch.empty((M, H), dtype=bf, device="cuda"),
                    residual_out=torch.empty((M, H), dtype=bf, device="cuda") if c["residual"] else None,
                    q=torch.empty((M, H), dtype=F8, device="cuda"),
                    scales=torch.empty((nb, M), device="cuda"))
    if c["op"] == "silu_mul":
        P, I = c["P"], c["I"]
        return dict(case=c, y=(1.5 * _randn(g, P, 2 * I)).to(bf),
                    h=torch.empty((P, I), dtype=bf, device="cuda"),
                    q=torch.empty((P, I), dtype=F8, device="cuda"),
                    scales=torch.empty((_cdiv(I, BLOCK), P), device="cuda"))
    M, K, Ns, S = c["M"], c["K"], c["Ns"], c["S"]
    if c["op"] == "gemm":
        xq, xs = _rows(g, M, K)
        wq, ws = _weights(g, 1, S, Ns, K)
        return dict(case=c, xq=xq, xs=xs, wq=wq[0], ws=ws[0],
                    y=torch.empty((M, S * Ns), dtype=bf, device="cuda"))
    E, topk = c["E"], c["topk"]
    xq, xs = _rows(g, M * topk if c["x_per_pair"] else M, K)
    wq, ws = _weights(g, E, S, Ns, K)
    ids = _route(g, M, topk, E, c["zipf"], c["drop"])
    srt, eids, ntpp, cap = _align(ids, E, c["block_m"])
    w = torch.softmax(_randn(g, M, topk), 1)
    y = _randn(g, M, topk, S * Ns).to(bf)  # rows of pairs without an expert here stay as they are
    return dict(case=c, xq=xq, xs=xs, wq=wq, ws=ws, ids=ids, sorted=srt, eids=eids, ntpp=ntpp,
                cap=cap, w=w, y=y)


# ---------------------------------------------------------------- the library's calls

def _run_own(st):
    import moe_lora_adapter_amd as mla
    c = st["case"]
    if c["op"] == "rms_norm":
        out = mla.moe_lora_rms_norm_fp8(st["x"], st["weight"], eps=st["eps"],
                                        residual=st["residual"], residual_out=st["residual_out"],
                                        y=st["y"], out=mla.Fp8Rows(st["q"], st["scales"]))
        return dict(q=out.q, scales=out.scales, y=st["y"], residual=st["residual_out"])
    if c["op"] == "silu_mul":
        out = mla.moe_lora_silu_mul_fp8(st["y"], h=st["h"], out=mla.Fp8Rows(st["q"], st["scales"]))
        return dict(q=out.q, scales=out.scales, h=st["h"])
    x = mla.Fp8Rows(st["xq"], st["xs"])
    if c["op"] == "gemm":
        return mla.moe_lora_fp8_gemm(x, st["wq"], st["ws"], st["y"])
    al = mla.AlignOutput(st["sorted"], st["eids"], st["ntpp"], None, None, c["block_m"], st["cap"])
    return mla.moe_lora_fp8_moe_gemm(x, st["wq"], st["ws"], al, st["w"], st["y"],
                                     mul_routed_weight=c["mul"], x_per_pair=c["x_per_pair"])


# ---------------------------------------------------------------- plain forms

def _quantise(v):
    """fp32 [M, K] -> e4m3 [M, K] and fp32 scales [K / 128, M]."""
    M, K = v.shape
    nb = _cdiv(K, BLOCK)
    b = torch.nn.functional.pad(v, (0, nb * BLOCK - K)).view(M, nb, BLOCK)
    s = b.abs().amax(2).clamp(min=MIN_AMAX) / F8_MAX
    q = (b / s[:, :, None]).view(M, nb * BLOCK)[:, :K].to(F8)
    return q, s.t().contiguous()


def _widen_rows(q, s):
    return q.float() * s.t().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _widen_weights(q, s):
    s = s.repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :]
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _run_plain(st):
    c = st["case"]
    bf = torch.bfloat16
    if c["op"] == "rms_norm":
        f, kept = st["x"].float(), None
        if st["residual"] is not None:
            kept = (f + st["residual"].float()).to(bf)
            f = kept.float()
        v = f * torch.rsqrt((f * f).mean(1, keepdim=True) + st["eps"]) * st["weight"].float()
        q, s = _quantise(v)
        return dict(q=q, scales=s, y=v.to(bf), residual=kept)
    if c["op"] == "silu_mul":
        gate, up = st["y"].float().chunk(2, 1)
        v = gate / (1 + torch.exp(-gate)) * up
        q, s = _quantise(v)
        return dict(q=q, scales=s, h=v.to(bf))
    x = _widen_rows(st["xq"], st["xs"])
    K = c["K"]
    w = _widen_weights(st["wq"], st["ws"])
    if c["op"] == "gemm":
        return (x @ w.view(-1, K).t()).to(bf)
    numel, N = c["M"] * c["topk"], c["S"] * c["Ns"]
    pairs = st["sorted"][0].long().view(-1, c["block_m"])  # numel: padding
    pad = torch.where(pairs < numel, pairs, 0)
    rows = pad if c["x_per_pair"] else pad // c["topk"]
    w = w.view(c["E"], N, K)[st["eids"][0].long()]
    d = torch.bmm(w, x[rows].transpose(1, 2).contiguous()).transpose(1, 2)
    if c["mul"]:
        d = d * st["w"].view(-1)[pad][:, :, None]
    y = torch.empty((numel + 1, N), dtype=bf, device=d.device)
    y[:numel] = st["y"].view(numel, N)
    y[pairs.reshape(-1)] = d.reshape(-1, N).to(bf)
    return y[:numel].view(c["M"], c["topk"], N)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "rms_norm":
        n = c["M"] * c["H"]
        return dict(bytes=n * (9 if c["residual"] else 5) + 2 * c["H"] + 4 * c["M"] * _cdiv(c["H"], BLOCK),
                    flops=8 * n)
    if c["op"] == "silu_mul":
        n = c["P"] * c["I"]
        return dict(bytes=7 * n + 4 * c["P"] * _cdiv(c["I"], BLOCK), flops=8 * n)
    M, K, N = c["M"], c["K"], c["S"] * c["Ns"]
    kb = _cdiv(K, BLOCK)
    weights = N * K + 4 * c["S"] * _cdiv(c["Ns"], BLOCK) * kb
    if c["op"] == "gemm":
        return dict(bytes=weights + M * (K + 4 * kb + 2 * N), flops=2 * M * N * K)
    pairs = M * c["topk"] * (1 - c["drop"])
    rows = M * c["topk"] if c["x_per_pair"] else M
    # experts that some token reaches, for even routing
    reached = c["E"] * (1 - (1 - c["topk"] / c["E"]) ** M)
    return dict(bytes=reached * weights + rows * (K + 4 * kb) + pairs * (2 * N + 4),
                flops=2 * pairs * N * K)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The operators' definition in float64, a block or an expert at a time.  What is rounded to 8
    bits is given before that rounding; the stored residual's rounding is part of the definition."""
    st = prepare(case, seed)
    c, D = st["case"], torch.float64

    def rows64(v):
        cols, scl = [], []
        for k in range(0, v.shape[1], BLOCK):
            part = v[:, k:k + BLOCK]
            scl.append(torch.maximum(part.abs().max(1).values,
                                     torch.tensor(MIN_AMAX, dtype=D, device=v.device)) / F8_MAX)
            cols.append(part / scl[-1][:, None])
        return torch.cat(cols, 1), torch.stack(scl)

    if c["op"] == "rms_norm":
        f, kept = st["x"].to(D), None
        if st["residual"] is not None:
            kept = (f + st["residual"].to(D)).to(torch.bfloat16).to(D)
            f = kept
        rms = (f.square().sum(1) / c["H"] + st["eps"]).sqrt()
        v = f / rms[:, None] * st["weight"].to(D)
        q, s = rows64(v)
        return dict(q=q, scales=s, y=v, residual=kept)
    if c["op"] == "silu_mul":
        y = st["y"].to(D)
        v = y[:, :c["I"]] * torch.sigmoid(y[:, :c["I"]]) * y[:, c["I"]:]
        q, s = rows64(v)
        return dict(q=q, scales=s, h=v)
    K, Ns, S = c["K"], c["Ns"], c["S"]

    def product(xq, xs, wq, ws):
        """[m, K] rows, their scales [kb, m], one expert's weights -> [m, S * Ns]."""
        out = torch.zeros((xq.shape[0], S, _cdiv(Ns, BLOCK) * BLOCK), dtype=D, device=xq.device)
        for j in range(_cdiv(K, BLOCK)):
            xk = xq[:, j * BLOCK:(j + 1) * BLOCK].to(D) * xs[j].to(D)[:, None]
            wk = wq[:, :, j * BLOCK:(j + 1) * BLOCK].to(D)
            for s in range(S):
                col = ws[s, :, j].to(D)[:, None].expand(-1, BLOCK).reshape(-1)
                out[:, s, :Ns] += (xk @ wk[s].t()) * col[:Ns]
        return out[:, :, :Ns].reshape(-1, S * Ns)

    if c["op"] == "gemm":
        return product(st["xq"], st["xs"], st["wq"], st["ws"])
    y = st["y"].to(D).view(-1, S * Ns)
    flat = st["ids"].reshape(-1)
    for e in range(c["E"]):
        p = (flat == e).nonzero().reshape(-1)
        if p.numel():
            r = p if c["x_per_pair"] else p // c["topk"]
            d = product(st["xq"].view(torch.uint8)[r].view(F8), st["xs"][:, r], st["wq"][e], st["ws"][e])
            y[p] = d * st["w"].view(-1)[p].to(D)[:, None] if c["mul"] else d
    return y.view(c["M"], c["topk"], S * Ns)
