"""The bf16 products on the GPU against float64 on the CPU, dense and over the align step's blocks: the
sums exactly on whole numbers, the epilogue within its error, alone and as a layer runs them."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_lora_adapter_amd as mla  # noqa: E402
import base_reference as br  # noqa: E402
from gpu_helpers import DEV  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
ACTS = [None, "silu", "gelu_tanh", "silu_mul", "swiglu_clamp"]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def dev(t):
    return None if t is None else t.to(DEV)


def bits(t):
    return t.view(torch.int16 if t.dtype is BF else torch.int32)


# ---------------------------------------------------------------- dense

# (M, K, Ns, S): from one row and eight columns to many tiles of 128 x 128 whose last ones are short (sizes
# for every kernel and tile are in product_tiles.py)
SIZES = [(1, 8, 8, 1), (1, 2880, 264, 2), (2, 72, 2056, 2), (5, 136, 40, 1), (16, 2880, 128, 2),
         (17, 264, 104, 2), (33, 1032, 120, 1), (64, 2048, 384, 2), (100, 2880, 320, 1),
         (64, 4096, 2048, 2), (40, 520, 1032, 2), (129, 376, 136, 2), (333, 656, 520, 3),
         (333, 1336, 1032, 2), (513, 1160, 520, 2), (1000, 272, 1032, 1), (1000, 200, 1032, 2),
         (2049, 144, 520, 2), (2049, 136, 2056, 1), (4096, 136, 1032, 2), (2300, 200, 2056, 2),
         (300, 8328, 136, 1), (70, 64, 1000, 2), (1, 16400, 16, 2), (4111, 1032, 64, 2)]


@pytest.mark.parametrize("M,K,Ns,S", SIZES)
def test_whole_numbers_exactly(M, K, Ns, S):
    """Sums of whole numbers up to 16 K + 8 stay below 2^24 and are exact; so is a sum with the bias,
    the delta and the residual."""
    g = gen(M + K + Ns)
    x, w = br.whole(g, M, K), br.whole(g, S, Ns, K)
    b, d, r = br.whole(g, S * Ns), br.whole(g, M, S * Ns), br.whole(g, M, S * Ns)
    xd, wd = x.to(DEV), w.to(DEV)
    want = x.float() @ w.view(-1, K).float().t()
    y = mla.moe_lora_gemm(xd, wd, out_dtype=F32)
    assert y.dtype is F32 and torch.equal(y.cpu(), want)
    assert torch.equal(mla.moe_lora_gemm(xd, wd).cpu(), want.to(BF))
    y = mla.moe_lora_gemm(xd, wd, bias=dev(b), delta=dev(d), residual=dev(r))
    assert torch.equal(y.cpu(), (want + b.float() + d.float() + r.float()).to(BF))


@pytest.mark.parametrize("M,K,Ns,S", SIZES)
@pytest.mark.parametrize("act", ACTS)
def test_epilogue(M, K, Ns, S, act):
    if act in br.GATED and S != 2:
        S = 2
    g = gen(M * 3 + K + Ns)
    x, w = br.rows(g, M, K), br.weights(g, S, Ns, K)
    No = Ns if act in br.GATED else S * Ns
    full = (M + K) % 3  # which of the operands are there
    b = (2 * torch.randn(S * Ns, generator=g)).to(BF) if full != 1 else None
    d = torch.randn((M, S * Ns), generator=g).to(BF) if full != 2 else None
    r = (3 * torch.randn((M, No), generator=g)).to(BF) if full != 0 else None
    ref, err = br.product(x, w, b, d, act, r)
    kw = dict(bias=dev(b), delta=dev(d), residual=dev(r), activation=act)
    out = F32 if (M + Ns) % 2 else BF
    y = mla.moe_lora_gemm(x.to(DEV), w.to(DEV), out_dtype=out, **kw)
    br.check(y, ref, err)
    z = torch.full((M + 1, No), 7.0, dtype=out, device=DEV)
    mla.moe_lora_gemm(x.to(DEV), w.to(DEV), z[:M], **kw)
    assert torch.equal(bits(y), bits(z[:M])), "the same inputs, other bits"
    assert torch.all(z[M] == 7)


@pytest.mark.parametrize("M,K,Ns", [(3, 256, 96), (40, 520, 264), (700, 136, 1032), (2100, 72, 2056)])
def test_in_place(M, K, Ns):
    """y may be the delta, or the residual."""
    g = gen(M)
    x, w = br.rows(g, M, K).to(DEV), br.weights(g, 1, Ns, K).to(DEV)
    t = torch.randn((M, Ns), generator=g).to(BF).to(DEV)
    for name in ("delta", "residual"):
        want = mla.moe_lora_gemm(x, w, activation="silu", **{name: t})
        y = t.clone()
        assert torch.equal(mla.moe_lora_gemm(x, w, y, activation="silu", **{name: y}), want)
    w2 = br.weights(g, 2, Ns, K).to(DEV)
    want = mla.moe_lora_gemm(x, w2, activation="silu_mul", residual=t)
    y = t.clone()
    assert torch.equal(mla.moe_lora_gemm(x, w2, y, activation="silu_mul", residual=y), want)


@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(act):
    """One product of ones carries every value of z to the epilogue: zeros of both signs, tails on both
    sides, the clamps' edges, infinities and NaN."""
    v = torch.cat([torch.tensor([0.0, -0.0, 1e-30, -1e-30, 7.0, -7.0, 7.03125, -7.03125, 20.0, -20.0,
                                 80.0, -80.0, 87.0, -87.0, 90.0, -90.0, 300.0, -300.0, 1e4, -1e4,
                                 3e38, -3e38]), torch.linspace(-12, 12, 74)]).to(BF)
    odd = torch.tensor([float("nan"), float("inf"), float("-inf")]).to(BF)
    if act in br.GATED:  # every pair
        gate, up = (t.reshape(-1) for t in torch.meshgrid(v[:48], v[:48], indexing="ij"))
        z = torch.stack([gate, up])
    else:
        z = v.view(1, -1)
    S, Ns = z.shape
    zero = torch.zeros((1, 8), dtype=BF)
    w = torch.zeros((S, Ns, 8), dtype=BF)
    ref = br.activate(z.view(1, -1).double(), act)
    err = br.activate_err(z.view(1, -1).double(), torch.zeros((1, S * Ns), dtype=torch.float64), act)
    # what float64 takes past fp32's range is infinite there
    ref = torch.where(ref.abs() > torch.finfo(F32).max, torch.sign(ref) * float("inf"), ref)
    for out in (BF, F32):
        y = mla.moe_lora_gemm(zero.to(DEV), w.to(DEV), delta=z.reshape(1, -1).to(DEV), activation=act,
                              out_dtype=out)
        fine = ref.abs() < 3e38
        br.check(y.cpu()[fine], ref[fine], err[fine])
        assert torch.all(y.cpu()[~fine].double().abs() >= 3e38)
    z = odd.repeat(8)[:24].repeat(S).view(1, -1)
    y = mla.moe_lora_gemm(zero.to(DEV), torch.zeros((S, 24, 8), dtype=BF, device=DEV),
                          delta=z.to(DEV), activation=act).cpu()
    ref = br.activate(z.double(), act).to(BF)
    if act == "swiglu_clamp":  # -inf * 0
        assert torch.equal(torch.isnan(y), torch.isnan(ref))
    assert torch.equal(torch.isnan(y), torch.isnan(ref)) and torch.equal(torch.isinf(y), torch.isinf(ref))


@pytest.mark.parametrize("M,K,Ns", [(9, 264, 40), (50, 520, 1032), (600, 200, 1032), (2100, 136, 2056)])
def test_nan_stays_in_its_row_and_column(M, K, Ns):
    g = gen(M)
    x, w = br.rows(g, M, K), br.weights(g, 1, Ns, K)
    clean = mla.moe_lora_gemm(x.to(DEV), w.to(DEV)).cpu()
    x[M - 1, K - 1], x[M // 2, 0] = float("nan"), float("inf")
    w[0, Ns - 1, K // 2] = float("nan")
    y = mla.moe_lora_gemm(x.to(DEV), w.to(DEV)).cpu()
    assert torch.isnan(y[M - 1]).all() and torch.isnan(y[:, Ns - 1]).all()
    assert not torch.isfinite(y[M // 2]).any()
    keep = [m for m in range(M) if m not in (M - 1, M // 2)]
    assert torch.equal(y[keep][:, :Ns - 1], clean[keep][:, :Ns - 1])


def test_no_rows_another_stream_and_a_given_buffer():
    w = br.weights(gen(1), 2, 64, 128).to(DEV)
    x = br.rows(gen(2), 24, 128).to(DEV)
    assert mla.moe_lora_gemm(x[:0], w).shape == (0, 128)
    want = mla.moe_lora_gemm(x, w, activation="silu_mul")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = mla.moe_lora_gemm(x, w, activation="silu_mul", stream=s)
    s.synchronize()
    assert torch.equal(y, want)


def test_weights_of_nearly_two_gib():
    """Offsets near the limit: the last columns of a matrix of 2^30 - 2^13 elements, few rows and many."""
    K, Ns = 8192, (1 << 17) - 1 - 7
    w = torch.zeros((1, Ns, K), dtype=BF, device=DEV)
    g = gen(4)
    tail = br.whole(g, 40, K)
    w[0, -40:] = tail.to(DEV)
    for M in (3, 70, 300):
        x = br.whole(g, M, K)
        y = mla.moe_lora_gemm(x.to(DEV), w, out_dtype=F32)
        assert torch.equal(y[:, -40:].cpu(), x.float() @ tail.float().t())
        assert torch.all(y[:, :-40] == 0)
        del y


# ---------------------------------------------------------------- grouped

def _routed(g, M, topk, E, zipf=0.0, drop=0.0):
    p = -zipf * torch.log(torch.arange(1, E + 1).float())[torch.randperm(E, generator=g)]
    u = torch.rand((M, E), generator=g).clamp(1e-6, 1 - 1e-6)
    ids = torch.topk(p - torch.log(-torch.log(u)), topk, dim=1).indices.int()
    return torch.where(torch.rand((M, topk), generator=g) < drop, torch.full_like(ids, -1), ids)


def _align(ids, E, B):
    return mla.moe_lora_align(ids.to(DEV), torch.zeros(ids.shape[0], dtype=torch.int32, device=DEV), E, 1, B)


def _grouped(x, w, ids, bias, delta, act, wt, per_pair, before):
    """(y, err) of every pair; a pair without an expert keeps its row."""
    E, S, Ns, K = w.shape
    M, k = ids.shape
    flat = ids.reshape(-1)
    ref, err = before.double().reshape(M * k, -1).clone(), torch.zeros(before.shape, dtype=torch.float64).view(M * k, -1)
    for e in range(E):
        p = torch.nonzero(flat == e).reshape(-1)
        if p.numel():
            ref[p], err[p] = br.product(x[p if per_pair else p // k], w[e], None if bias is None else bias[e],
                                        None if delta is None else delta.view(M * k, -1)[p], act, None,
                                        None if wt is None else wt.reshape(-1)[p])
    return ref, err


# (M, topk, E, K, Ns, B, zipf, drop): blocks of few rows, tiles over several blocks, experts with
# none, one and most of the pairs
MOE = [(1, 1, 1, 8, 8, 16, 0, 0), (1, 4, 32, 264, 136, 16, 0, 0), (16, 4, 32, 2880, 200, 16, 0, 0),
       (8, 4, 128, 520, 264, 16, 0, 0.1), (33, 2, 8, 136, 72, 32, 1.2, 0.1), (100, 8, 16, 264, 264, 64, 0, 0),
       (300, 4, 8, 200, 264, 64, 0.8, 0.05), (513, 2, 4, 328, 520, 128, 1.2, 0.1), (700, 8, 64, 72, 136, 16, 1.2, 0),
       (1024, 4, 8, 136, 392, 128, 0, 0), (2000, 2, 4, 72, 1032, 64, 1.2, 0.2), (2500, 1, 2, 264, 264, 32, 0, 0),
       (64, 6, 6, 1032, 40, 16, 0, 0.5), (1500, 4, 16, 64, 264, 128, 2.0, 0.1)]


@pytest.mark.parametrize("M,topk,E,K,Ns,B,zipf,drop", MOE)
@pytest.mark.parametrize("per_pair", [False, True])
def test_moe_whole_numbers_exactly(M, topk, E, K, Ns, B, zipf, drop, per_pair):
    g = gen(M + K)
    S = 1 + (M + E) % 2
    ids = _routed(g, M, topk, E, zipf, drop)
    x, w = br.whole(g, M * topk if per_pair else M, K), br.whole(g, E, S, Ns, K)
    b, d = br.whole(g, E, S * Ns), br.whole(g, M, topk, S * Ns)
    wt = torch.randint(1, 5, (M, topk), generator=g).float()  # products with it are exact, too
    y = torch.full((M, topk, S * Ns), 3.0, dtype=BF, device=DEV)
    mla.moe_lora_moe_gemm(x.to(DEV), w.to(DEV), _align(ids, E, B), wt.to(DEV), y, mul_routed_weight=True,
                          x_per_pair=per_pair, bias=b.to(DEV), delta=d.to(DEV))
    want, _ = _grouped(x, w, ids, b, d, None, wt, per_pair, torch.full((M, topk, S * Ns), 3.0))
    assert torch.equal(y.cpu().view(M * topk, -1), want.float().to(BF))


@pytest.mark.parametrize("M,topk,E,K,Ns,B,zipf,drop", MOE)
@pytest.mark.parametrize("act", ACTS)
def test_moe_epilogue(M, topk, E, K, Ns, B, zipf, drop, act):
    g = gen(M * 5 + K)
    S, per_pair, mul = 2 if act in br.GATED else 1, M % 2 == 0, E % 3 != 1
    No = Ns if act in br.GATED else S * Ns
    ids = _routed(g, M, topk, E, zipf, drop)
    x, w = br.rows(g, M * topk if per_pair else M, K), br.weights(g, E, S, Ns, K)
    b = torch.randn((E, S * Ns), generator=g).to(BF) if K % 3 else None
    d = torch.randn((M, topk, S * Ns), generator=g).to(BF) if K % 5 else None
    wt = torch.softmax(torch.randn((M, topk), generator=g), 1)
    before = torch.randn((M, topk, No), generator=g).to(BF)
    al = _align(ids, E, B)

    def go():
        y = before.to(DEV)
        return mla.moe_lora_moe_gemm(x.to(DEV), w.to(DEV), al, wt.to(DEV), y, mul_routed_weight=mul,
                                     x_per_pair=per_pair, bias=dev(b), delta=dev(d), activation=act)
    y = go()
    ref, err = _grouped(x, w, ids, b, d, act, wt if mul else None, per_pair, before)
    br.check(y.view(M * topk, -1), ref, err)
    gone = ids.reshape(-1) < 0
    assert torch.equal(y.cpu().view(M * topk, -1)[gone], before.view(M * topk, -1)[gone])
    assert torch.equal(bits(y), bits(go())), "the same inputs, other bits"


@pytest.mark.parametrize("M,topk,E,K,Ns,B", [(16, 4, 8, 264, 136, 16), (400, 4, 4, 136, 264, 64),
                                             (1200, 4, 4, 72, 264, 128)])
def test_moe_passes_over_what_is_no_pair(M, topk, E, K, Ns, B):
    """Ids outside the pairs in the middle of a block, experts outside [0, E), and whatever stands behind
    the last block."""
    g = gen(M + 2)
    ids = _routed(g, M, topk, E)
    x, w = br.whole(g, M, K), br.whole(g, E, 1, Ns, K)
    al = _align(ids, E, B)
    n = int(al.num_tokens_post_padded[0])
    srt, eids = al.sorted_token_ids.cpu(), al.expert_ids.cpu()
    want, _ = _grouped(x, w, ids, None, None, None, None, False, torch.full((M, topk, Ns), 5.0))
    srt[0, n:] = torch.arange(al.cap - n)   # pairs behind the last block
    eids[0, n // B:] = 1
    junk = [-1, M * topk, 2 ** 31 - 1, -2 ** 31]
    at = torch.randperm(n, generator=g)[:n // 7]
    for j, i in enumerate(at.tolist()):
        p = int(srt[0, i])
        if p < M * topk:
            want[p] = 5.0
        srt[0, i] = junk[j % 4]
    for blk, e in ((0, E), (n // B - 1, -1)):
        for p in srt[0, blk * B:(blk + 1) * B].tolist():
            if 0 <= p < M * topk:
                want[p] = 5.0
        eids[0, blk] = e
    al = mla.AlignOutput(srt.to(DEV), eids.to(DEV), al.num_tokens_post_padded, None, None, B, al.cap)
    y = torch.full((M, topk, Ns), 5.0, dtype=BF, device=DEV)
    mla.moe_lora_moe_gemm(x.to(DEV), w.to(DEV), al, None, y, mul_routed_weight=False)
    assert torch.equal(y.cpu().view(M * topk, -1), want.float().to(BF))


def test_moe_delta_in_place_and_empty():
    g = gen(8)
    M, k, E, K, Ns = 40, 4, 8, 136, 264
    ids = _routed(g, M, k, E, drop=0.2)
    x, w = br.rows(g, M, K).to(DEV), br.weights(g, E, 1, Ns, K).to(DEV)
    al = _align(ids, E, 16)
    d = torch.randn((M, k, Ns), generator=g).to(BF).to(DEV)
    kw = dict(mul_routed_weight=False, activation="gelu_tanh")
    want = mla.moe_lora_moe_gemm(x, w, al, None, d.clone(), delta=d, **kw)
    y = d.clone()
    assert torch.equal(mla.moe_lora_moe_gemm(x, w, al, None, y, delta=y, **kw), want)
    none = _align(torch.full((M, k), -1, dtype=torch.int32), E, 16)
    y = d.clone()
    assert torch.equal(mla.moe_lora_moe_gemm(x, w, none, None, y, **kw), d)
    e = _align(torch.zeros((0, k), dtype=torch.int32), E, 16)
    mla.moe_lora_moe_gemm(x[:0], w, e, None, d[:0], **kw)


# ---------------------------------------------------------------- a layer

@pytest.mark.parametrize("M,E,topk,K,I,B,act", [(9, 32, 4, 264, 136, 16, "swiglu_clamp"),
                                                (300, 16, 4, 256, 264, 64, "silu_mul")])
def test_layer_with_adapters(M, E, topk, K, I, B, act):
    """Router's projection, routing, align, the adapters' delta, w13 with it and the activation, w2 with
    its adapters on top, and the combine, eager and from a captured graph on other inputs: each step's
    output against float64 of what that step was given."""
    g = gen(M + E)
    L, r, cap = 3, 16, 1
    gate, gb = br.weights(g, 1, E, K), torch.randn(E, generator=g).to(BF)
    w13, b13 = br.weights(g, E, 2, I, K), torch.randn((E, 2 * I), generator=g).to(BF)
    w2, b2 = br.weights(g, E, 1, K, I), torch.randn((E, K), generator=g).to(BF)
    a13, e13 = br.weights(g, 2, L, E, r, K), br.weights(g, 2, L, E, I, r)
    a2, e2 = br.weights(g, 1, L, E, r, I), br.weights(g, 1, L, E, K, r)
    mapping = torch.randint(-1, L, (M,), generator=g).int()
    xs = [br.rows(g, M, K) for _ in range(3)]
    t = {n: v.to(DEV) for n, v in dict(gate=gate, gb=gb, w13=w13, b13=b13, w2=w2, b2=b2, a13=a13, e13=e13,
                                       a2=a2, e2=e2, mapping=mapping, x=xs[0]).items()}
    zero = torch.zeros(M, dtype=torch.int32, device=DEV)
    al = mla.alloc_align_output(M, topk, E, L, 16, DEV)
    base = mla.alloc_align_output(M, topk, E, 1, B, DEV)
    ws = [torch.empty(max(16, mla.align_workspace_size(M, topk, E, n, b)), dtype=torch.uint8, device=DEV)
          for n, b in ((L, 16), (1, B))]
    o = {}

    def buf(name, *shape, dtype=BF):
        return o.setdefault(name, torch.zeros(shape, dtype=dtype, device=DEV))

    def layer():
        logits = mla.moe_lora_gemm(t["x"], t["gate"], buf("logits", M, E, dtype=F32), bias=t["gb"])
        ids, wt = mla.moe_lora_route(logits, topk, topk_ids=buf("ids", M, topk, dtype=torch.int32),
                                     topk_weights=buf("wt", M, topk, dtype=F32))
        mla.moe_lora_align(ids, zero, E, 1, B, out=base, workspace=ws[1])
        mla.moe_lora_align(ids, t["mapping"], E, L, 16, out=al, workspace=ws[0])
        d = buf("d13", M, topk, 2 * I)
        d.zero_()
        mla.fused_moe_lora(t["x"], t["a13"], t["e13"], al, None, d, mul_routed_weight=False, add_inputs=False)
        h = buf("h", M, topk, I)
        mla.moe_lora_moe_gemm(t["x"], t["w13"], base, None, h, mul_routed_weight=False, bias=t["b13"],
                              delta=d, activation=act)
        h = h.view(M * topk, I)
        y = buf("y", M, topk, K)
        mla.moe_lora_moe_gemm(h, t["w2"], base, wt, y, mul_routed_weight=True, x_per_pair=True, bias=t["b2"])
        buf("y0", M, topk, K).copy_(y)
        mla.fused_moe_lora(h, t["a2"], t["e2"], al, wt, y, mul_routed_weight=True, add_inputs=True, x_per_pair=True)
        mla.moe_lora_combine(y, buf("out", M, K), residual=t["x"])

    def check(x):
        v = {n: b.cpu() for n, b in o.items()}
        br.check(o["logits"], *br.product(x, gate, gb))
        br.check_route((v["ids"], v["wt"]), br.route(v["logits"], topk), 64.0)
        br.check(o["h"].view(M * topk, I), *_grouped(x, w13, v["ids"], b13, v["d13"], act, None, False, v["h"]))
        br.check(o["y0"].view(M * topk, K),
                 *_grouped(v["h"].view(M * topk, I), w2, v["ids"], b2, None, None, v["wt"], True, v["y0"]))
        br.check(o["out"], *br.combine(v["y"], residual=x))
        some = mapping >= 0
        assert not torch.equal(v["y"][some], v["y0"][some]) and torch.equal(v["y"][~some], v["y0"][~some])
        assert bool((v["d13"][some].abs().amax((1, 2)) > 0).all()) and not v["d13"][~some].any()

    layer()
    torch.cuda.synchronize()
    check(xs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for x in xs + xs[:1]:
        t["x"].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        check(x)
        kept = {n: b.clone() for n, b in o.items()}
        layer()
        torch.cuda.synchronize()
        for n in kept:
            assert torch.equal(kept[n], o[n]), n
