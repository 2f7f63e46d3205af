"""The 8-bit base side on the GPU against float64 on the CPU: the norm, the activation and the
e4m3 products, dense and over the align step's blocks, alone and as a layer runs them."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_lora_adapter_amd as mla  # noqa: E402
import fp8_reference as fr  # noqa: E402
import gpu_helpers as gh  # noqa: E402
import oracle  # noqa: E402

DEV, BF, D = gh.DEV, torch.bfloat16, torch.float64
NORM_REL = 2.0 ** -17  # at most 90 additions of a thread and the tree, halved by the root, 4 more
SILU_REL = 2.0 ** -16  # the exponential's argument: |x| 2^-24 for |x| < 90, and 6 more roundings


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- norm

@pytest.mark.parametrize("M,H", [(1, 8), (3, 120), (5, 136), (16, 2880), (9, 2048), (7, 4096),
                                 (65, 2056), (2, 8192), (3, 16384), (2, 16392), (1, 65536)])
@pytest.mark.parametrize("res", [False, True])
def test_rms_norm(M, H, res):
    g = gen(M * 7 + H + res)
    x, w = torch.randn((M, H), generator=g).to(BF), (1 + torch.randn(H, generator=g) / 4).to(BF)
    r = (3 * torch.randn((M, H), generator=g)).to(BF) if res else None
    h, v = fr.rms_norm(x, w, 1e-5, r)
    y = torch.empty((M, H), dtype=BF, device=DEV)
    ro = torch.empty((M, H), dtype=BF, device=DEV) if res else None
    out = mla.moe_lora_rms_norm_fp8(x.to(DEV), w.to(DEV), eps=1e-5, y=y, residual_out=ro,
                                    residual=r.to(DEV) if res else None)
    fr.check_rows(out.q, out.scales, v, NORM_REL)
    fr.check_bf16(y, v, NORM_REL * v.abs())
    if res:
        assert torch.equal(ro.cpu().to(D), h)


def test_rms_norm_in_place_residual_and_without_bf16_rows():
    g = gen(5)
    x, r = torch.randn((33, 2880), generator=g).to(BF), torch.randn((33, 2880), generator=g).to(BF)
    w = torch.ones(2880, dtype=BF)
    h, v = fr.rms_norm(x, w, 1e-6, r)
    rd, xd = r.to(DEV), x.to(DEV)
    out = mla.moe_lora_rms_norm_fp8(xd, w.to(DEV), residual=rd)
    assert torch.equal(rd.cpu().to(D), h) and torch.equal(xd.cpu(), x)
    fr.check_rows(out.q, out.scales, v, NORM_REL)
    out2 = mla.moe_lora_rms_norm_fp8(xd, w.to(DEV), residual=r.to(DEV), residual_out=xd)
    assert torch.equal(xd.cpu().to(D), h)
    assert torch.equal(out.q.view(torch.uint8), out2.q.view(torch.uint8))


def test_rms_norm_extreme_rows():
    """Zeros, values under the least scale, large values, and rows of NaN and infinity between
    ordinary ones, which stay as they are."""
    H = 400
    g = gen(6)
    x = torch.randn((8, H), generator=g).to(BF)
    x[0] = 0
    x[1] = x[1] * 2.0 ** -60
    x[2] = x[2] * 2.0 ** 30
    x[4, 17] = float("nan")
    x[6, 300] = float("inf")
    w = torch.ones(H, dtype=BF)
    out = mla.moe_lora_rms_norm_fp8(x.to(DEV), w.to(DEV), eps=1e-12)
    q, s = out.q.cpu().float(), out.scales.cpu()
    keep = [0, 1, 2, 3, 5, 7]
    _, v = fr.rms_norm(x[keep], w, 1e-12)
    fr.check_rows(out.q.cpu().view(torch.uint8)[keep].view(fr.F8), s[:, keep], v, NORM_REL)
    assert torch.all(q[0] == 0) and torch.isnan(q[4]).all() and torch.isnan(q[6, 300])


# ---------------------------------------------------------------- activation

@pytest.mark.parametrize("P,I", [(1, 8), (3, 120), (33, 136), (64, 2880), (1000, 768), (17, 1160)])
def test_silu_mul(P, I):
    y = (4 * torch.randn((P, 2 * I), generator=gen(P + I))).to(BF)
    y[0, :8] = torch.tensor([0.0, -0.0, 60.0, -60.0, 80.0, -80.0, 1e-30, -1e-30]).to(BF)
    v = fr.silu_mul(y)
    h = torch.empty((P, I), dtype=BF, device=DEV)
    out = mla.moe_lora_silu_mul_fp8(y.to(DEV), h=h)
    fr.check_rows(out.q, out.scales, v, SILU_REL)
    fr.check_bf16(h, v, SILU_REL * v.abs() + 2.0 ** -140)
    out2 = mla.moe_lora_silu_mul_fp8(y.to(DEV).view(P, 1, 2 * I))
    assert torch.equal(out.q.view(torch.uint8), out2.q.view(torch.uint8))


def test_silu_mul_nan_and_infinity():
    y = torch.ones((4, 2 * 256), dtype=BF)
    y[1, 5] = float("nan")
    y[2, 130] = float("inf")
    out = mla.moe_lora_silu_mul_fp8(y.to(DEV))
    q, s = out.q.cpu().float(), out.scales.cpu()
    assert torch.isnan(q[1, 5]) and int(torch.isnan(q).sum()) == 2
    assert torch.isinf(s[1, 2]) and torch.isnan(q[2, 130]) and int(torch.isinf(s).sum()) == 1
    assert torch.all(q[1, :5] == 448) and torch.all(q[3] == 448) and torch.all(q[2, 131:] == 0)


# ---------------------------------------------------------------- dense product

GEMM = [(1, 16, 8, 1), (1, 2880, 264, 2), (2, 128, 16, 1), (5, 144, 24, 3), (15, 400, 136, 1),
        (16, 4096, 256, 1), (17, 272, 200, 2), (31, 2880, 64, 1), (33, 1040, 120, 1),
        (64, 2048, 768, 1), (65, 256, 264, 1), (100, 2880, 320, 1), (128, 512, 512, 1),
        (129, 384, 136, 2), (257, 1168, 392, 1), (333, 656, 520, 3), (513, 2880, 264, 1),
        (1000, 272, 1032, 1), (2049, 144, 264, 1), (300, 8336, 136, 1), (4, 16400, 40, 1)]


def _gemm(M, K, Ns, S, seed):
    g = gen(seed)
    xq, xs = fr.rand_rows(g, M, K)
    wq, ws = fr.rand_weights(g, S, Ns, K)
    return xq, xs, wq, ws


def _rows(xq, xs):
    return mla.Fp8Rows(xq.to(DEV), xs.contiguous().to(DEV))


@pytest.mark.parametrize("M,K,Ns,S", GEMM)
def test_gemm(M, K, Ns, S):
    xq, xs, wq, ws = _gemm(M, K, Ns, S, M + K + Ns)
    ref, mag = fr.gemm(xq, xs, wq, ws)
    x = _rows(xq, xs)
    y = mla.moe_lora_fp8_gemm(x, wq.to(DEV), ws.to(DEV))
    fr.check_bf16(y, ref, fr.gemm_err(mag, K))
    z = torch.full_like(y, 7.0)
    mla.moe_lora_fp8_gemm(x, wq.to(DEV), ws.to(DEV), z)
    assert torch.equal(y.view(torch.int16), z.view(torch.int16)), "the same inputs, other bits"


@pytest.mark.parametrize("M,K,Ns,S", GEMM)
def test_gemm_whole_numbers_exactly(M, K, Ns, S):
    g = gen(M + K)
    xq, xs = fr.whole_rows(g, M, K)
    wq, ws = fr.whole_weights(g, S, Ns, K)
    ref, _ = fr.gemm(xq, xs, wq, ws)
    y = mla.moe_lora_fp8_gemm(_rows(xq, xs), wq.to(DEV), ws.to(DEV)).cpu()
    assert torch.equal(y, ref.float().to(BF))


# More tiles than the device holds at once, so that a workgroup takes several: tiles of 64 x 128 and
# larger, K of one block, of two and of more than the ring's stages, tiles that end in the last row
# and column.
MANY = [(4100, 64, 5000, 1), (4100, 144, 4104, 1), (5000, 400, 4304, 2), (3000, 272, 9000, 1),
        (4096, 1040, 8200, 1), (2000, 528, 4104, 1), (700, 400, 4200, 2), (1500, 128, 12304, 1),
        (65, 272, 40000, 1), (130, 656, 33000, 1), (64, 272, 70000, 1), (12000, 272, 264, 1),
        (40000, 144, 72, 1)]


def _wide(q, s):
    return q.float() * s.t().repeat_interleave(128, 1)[:, :q.shape[1]]


def _wide_w(q, s):
    s = s.repeat_interleave(128, -2)[..., :q.shape[-2], :]
    return q.float() * s.repeat_interleave(128, -1)[..., :q.shape[-1]]


@pytest.mark.parametrize("M,K,Ns,S", MANY)
def test_gemm_many_tiles_exactly(M, K, Ns, S):
    """Whole numbers again, where any order of fp32 additions is exact: torch's product on the GPU."""
    g = gen(M + Ns)
    xq, xs = fr.whole_rows(g, M, K)
    wq, ws = fr.whole_weights(g, S, Ns, K)
    x, w, sc = _rows(xq, xs), wq.to(DEV), ws.to(DEV)
    buf = torch.full((M * S * Ns + 65536,), 3.0, dtype=BF, device=DEV)
    y = mla.moe_lora_fp8_gemm(x, w, sc, buf[:M * S * Ns].view(M, S * Ns))
    want = (_wide(x.q, x.scales) @ _wide_w(w, sc).view(S * Ns, K).t().contiguous()).to(BF)
    assert torch.equal(y, want)
    assert bool((buf[M * S * Ns:] == 3.0).all())


@pytest.mark.parametrize("M", [3, 200, 700])
def test_gemm_nan_stays_in_its_row_and_column(M):
    xq, xs, wq, ws = _gemm(M, 656, 264, 1, M)
    ref, mag = fr.gemm(xq, xs, wq, ws)
    xq[1, 650] = float("nan")
    wq[0, 77, 3] = float("nan")
    y = mla.moe_lora_fp8_gemm(_rows(xq, xs), wq.to(DEV), ws.to(DEV)).cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 77]).all()
    rows, cols = torch.arange(M) != 1, torch.arange(264) != 77
    fr.check_bf16(y[rows][:, cols], ref[rows][:, cols], fr.gemm_err(mag, 656)[rows][:, cols])


@pytest.mark.parametrize("M,K,Ns", [(40, 272, 264), (3000, 272, 9000), (700, 144, 8200)])
def test_gemm_infinite_and_nan_scales_stay_in_their_rows(M, K, Ns):
    """Rows whose scale is infinite or NaN, also where a workgroup goes on to another tile."""
    g = gen(M)
    xq, xs = fr.whole_rows(g, M, K)
    wq, ws = fr.whole_weights(g, 1, Ns, K)
    bad = torch.arange(7, M, 31)
    xs[:, bad[::2]] = float("inf")
    xs[-1, bad[1::2]] = float("nan")
    x, w, sc = _rows(xq, xs), wq.to(DEV), ws.to(DEV)
    y = mla.moe_lora_fp8_gemm(x, w, sc)
    keep = torch.ones(M, dtype=torch.bool)
    keep[bad] = False
    keep = keep.to(DEV)
    want = (_wide(x.q, x.scales)[keep] @ _wide_w(w, sc).view(Ns, K).t().contiguous()).to(BF)
    assert torch.equal(y[keep], want)
    assert not bool(torch.isfinite(y[~keep]).any())


def test_gemm_leaves_what_is_behind_its_output():
    """The buffer goes on behind y: nothing is written there, at sizes that end inside a tile."""
    for M, Ns in ((5, 40), (70, 264), (300, 392)):
        xq, xs, wq, ws = _gemm(M, 272, Ns, 1, M)
        buf = torch.full((M * Ns + 4096,), 3.0, dtype=BF, device=DEV)
        mla.moe_lora_fp8_gemm(_rows(xq, xs), wq.to(DEV), ws.to(DEV), buf[:M * Ns].view(M, Ns))
        assert bool((buf[M * Ns:] == 3.0).all())


# ---------------------------------------------------------------- grouped product

MOE = [  # M, topk, K, Ns, S, E, block_m, x_per_pair, mul, kind
    (1, 1, 128, 16, 1, 1, 16, False, False, "uniform"),
    (1, 4, 2880, 136, 2, 32, 16, False, True, "uniform"),
    (16, 4, 400, 264, 2, 32, 16, False, False, "uniform"),
    (8, 4, 2880, 120, 1, 128, 16, True, True, "uniform"),
    (40, 2, 272, 72, 1, 4, 16, True, True, "invalid"),
    (50, 3, 144, 200, 2, 5, 32, False, True, "invalid"),
    (100, 2, 656, 264, 1, 3, 32, True, False, "uniform"),
    (33, 8, 384, 264, 2, 16, 64, False, False, "uniform"),
    (128, 2, 656, 392, 1, 3, 64, True, True, "invalid"),
    (300, 4, 272, 136, 2, 8, 64, False, True, "one"),
    (257, 2, 512, 264, 1, 2, 128, True, True, "uniform"),
    (500, 4, 1168, 200, 2, 7, 128, False, False, "invalid"),
    (64, 8, 144, 264, 1, 128, 128, True, True, "uniform"),
    (90, 2, 256, 264, 1, 4, 128, False, True, "twice"),
    (20, 2, 256, 40, 1, 8, 16, False, False, "none"),
    (200, 1, 8336, 72, 1, 3, 64, False, False, "uniform"),
]


def _routing(rng, M, topk, E, kind):
    if kind == "none":
        return np.full((M, topk), -1, np.int32)
    if kind == "one":
        return np.full((M, topk), E - 1, np.int32)
    ids = rng.integers(-1, E + 1, (M, topk)) if kind == "invalid" else rng.integers(0, E, (M, topk))
    if kind == "twice":  # a token that names an expert twice has two rows
        ids[:, 1] = ids[:, 0]
    return ids.astype(np.int32)


def _moe(M, topk, K, Ns, S, E, B, per_pair, mul, kind):
    rng, g = np.random.default_rng(M * topk + K + E), gen(M + K + E)
    ids = _routing(rng, M, topk, E, kind)
    xq, xs = fr.rand_rows(g, M * topk if per_pair else M, K)
    wq, ws = fr.rand_weights(g, E, S, Ns, K)
    tw = torch.rand((M, topk), generator=g)
    y0 = torch.randn((M, topk, S * Ns), generator=g).to(BF)
    return ids, xq, xs, wq, ws, tw, y0


def _base_align(ids, E, B):
    return mla.moe_lora_align(gh.i32_dev(ids), torch.zeros(ids.shape[0], dtype=torch.int32, device=DEV),
                              E, 1, B)


def _check_moe(y, y0, ids, xq, xs, wq, ws, tw, per_pair, mul, skip=()):
    K, N, topk = wq.shape[-1], y0.shape[-1], ids.shape[1]
    got, left = y.cpu().view(-1, N), np.ones(ids.size, bool)
    for e, p in fr.pairs_of(ids, wq.shape[0]).items():
        if e in skip:
            continue
        r = p if per_pair else p // topk
        ref, mag = fr.gemm(xq.view(torch.uint8)[r].view(fr.F8), xs[:, r], wq[e], ws[e])
        if mul:
            f = tw.view(-1)[p].to(D)[:, None]
            ref, mag = ref * f, mag * f
        fr.check_bf16(got[p], ref, fr.gemm_err(mag, K) + mag * 2.0 ** -24)
        left[p] = False
    assert torch.equal(got[left].view(torch.int16), y0.view(-1, N)[left].view(torch.int16))


@pytest.mark.parametrize("case", MOE)
def test_moe_gemm(case):
    M, topk, K, Ns, S, E, B, per_pair, mul, kind = case
    ids, xq, xs, wq, ws, tw, y0 = _moe(*case)
    al = _base_align(ids, E, B)
    y, x = y0.to(DEV), _rows(xq, xs)
    args = dict(mul_routed_weight=mul, x_per_pair=per_pair)
    mla.moe_lora_fp8_moe_gemm(x, wq.to(DEV), ws.to(DEV), al, tw.to(DEV) if mul else None, y, **args)
    _check_moe(y, y0, ids, xq, xs, wq, ws, tw, per_pair, mul)
    z = y0.to(DEV)
    mla.moe_lora_fp8_moe_gemm(x, wq.to(DEV), ws.to(DEV), al, tw.to(DEV), z, **args)
    assert torch.equal(y.view(torch.int16), z.view(torch.int16)), "the same inputs, other bits"


@pytest.mark.parametrize("case", MOE)
def test_moe_gemm_whole_numbers_exactly(case):
    M, topk, K, Ns, S, E, B, per_pair, mul, kind = case
    ids = _routing(np.random.default_rng(M + E), M, topk, E, kind)
    g = gen(M + topk)
    xq, xs = fr.whole_rows(g, M * topk if per_pair else M, K)
    wq, ws = fr.whole_weights(g, E, S, Ns, K)
    tw = 2.0 ** torch.randint(-2, 3, (M, topk), generator=g).float()
    y = torch.full((M, topk, S * Ns), 5.0, dtype=BF, device=DEV)
    mla.moe_lora_fp8_moe_gemm(_rows(xq, xs), wq.to(DEV), ws.to(DEV), _base_align(ids, E, B),
                              tw.to(DEV), y, mul_routed_weight=mul, x_per_pair=per_pair)
    want = torch.full((M * topk, S * Ns), 5.0, dtype=BF)
    for e, p in fr.pairs_of(ids, E).items():
        r = p if per_pair else p // topk
        ref, _ = fr.gemm(xq.view(torch.uint8)[r].view(fr.F8), xs[:, r], wq[e], ws[e])
        want[p] = ((ref * tw.view(-1)[p].to(D)[:, None]) if mul else ref).float().to(BF)
    assert torch.equal(y.cpu().view(-1, S * Ns), want)


@pytest.mark.parametrize("M,topk,K,Ns,S,E,B,kind", [
    (3000, 4, 272, 392, 2, 16, 16, "invalid"), (3000, 2, 144, 2200, 1, 40, 64, "uniform"),
    (9000, 4, 64, 520, 1, 40, 128, "uniform"), (6000, 4, 400, 136, 2, 64, 32, "invalid"),
    (2500, 8, 272, 1032, 1, 128, 128, "uniform"), (140000, 2, 16, 8, 1, 3, 16, "invalid"),
    (150000, 2, 48, 24, 1, 600, 16, "uniform")])
def test_moe_gemm_many_tiles_exactly(M, topk, K, Ns, S, E, B, kind):
    """Tiles of several align blocks, more of them than the device holds at once; the last two have
    more blocks than one launch takes."""
    ids = _routing(np.random.default_rng(M + E), M, topk, E, kind)
    g = gen(M + topk)
    xq, xs = fr.whole_rows(g, M, K)
    wq, ws = fr.whole_weights(g, E, S, Ns, K)
    tw = 2.0 ** torch.randint(-2, 3, (M, topk), generator=g).float()
    x, w, sc, dw = _rows(xq, xs), wq.to(DEV), ws.to(DEV), tw.to(DEV)
    y = torch.full((M, topk, S * Ns), 5.0, dtype=BF, device=DEV)
    mla.moe_lora_fp8_moe_gemm(x, w, sc, _base_align(ids, E, B), dw, y, mul_routed_weight=True)
    xw, want = _wide(x.q, x.scales), torch.full((M * topk, S * Ns), 5.0, dtype=BF, device=DEV)
    flat, wt = gh.i32_dev(ids).view(-1), dw.view(-1)
    for e in range(E):
        p = (flat == e).nonzero().view(-1)
        d = xw[p // topk] @ _wide_w(w[e], sc[e]).view(S * Ns, K).t().contiguous()
        want[p] = (d * wt[p][:, None]).to(BF)
    assert torch.equal(y.view(M * topk, S * Ns), want)


def test_rms_norm_more_rows_than_a_grid_axis():
    M, H = (1 << 26) + 5, 8
    x = torch.ones((M, H), dtype=BF, device=DEV)
    x[-1] = 2.0
    out = mla.moe_lora_rms_norm_fp8(x, torch.ones(H, dtype=BF, device=DEV), eps=0.0)
    assert bool((out.q.view(torch.uint8) == 0x7e).all())  # 448, the largest of its block
    assert bool(((out.scales - 1 / 448).abs() < 1e-8).all())


@pytest.mark.parametrize("B", [16, 64, 128])
def test_moe_gemm_passes_over_ids_outside_their_range(B):
    case = (120, 2, 272, 136, 1, 4, B, True, True, "uniform")
    ids, xq, xs, wq, ws, tw, y0 = _moe(*case)
    al = _base_align(ids, 4, B)
    n = int(al.num_tokens_post_padded.item()) // B
    al.expert_ids[0, :n][al.expert_ids[0, :n] == 2] = 4
    al.expert_ids[0, :n][al.expert_ids[0, :n] == 1] = -3
    y = y0.to(DEV)
    mla.moe_lora_fp8_moe_gemm(_rows(xq, xs), wq.to(DEV), ws.to(DEV), al, tw.to(DEV), y,
                              mul_routed_weight=True, x_per_pair=True)
    _check_moe(y, y0, ids, xq, xs, wq, ws, tw, True, True, skip=(1, 2))


def test_empty_calls():
    E = dict(device=DEV)
    w = torch.zeros((2, 1, 16, 32), dtype=fr.F8, **E)
    ws = torch.ones((2, 1, 1, 1), **E)
    x = mla.alloc_fp8_rows(0, 32, DEV)
    assert mla.moe_lora_fp8_gemm(x, w[0], ws[0]).shape == (0, 16)
    al = _base_align(np.zeros((0, 2), np.int32), 2, 16)
    y = torch.empty((0, 2, 16), dtype=BF, **E)
    mla.moe_lora_fp8_moe_gemm(x, w, ws, al, None, y, mul_routed_weight=False)
    out = mla.moe_lora_rms_norm_fp8(torch.empty((0, 16), dtype=BF, **E), torch.ones(16, dtype=BF, **E))
    assert out.q.shape == (0, 16)
    assert mla.moe_lora_silu_mul_fp8(torch.empty((0, 16), dtype=BF, **E)).q.shape == (0, 8)


# ---------------------------------------------------------------- a layer

class Layer:
    """One layer's base side in 8 bits with adapters on both projections."""

    def __init__(self, M, seed, H=272, I=144, E=6, topk=2, L=2, r=8, B=16):
        g, rng = gen(seed), np.random.default_rng(seed)
        self.M, self.H, self.I, self.E, self.topk, self.L, self.B = M, H, I, E, topk, L, B
        self.x = torch.randn((M, H), generator=g).to(BF)
        self.res = torch.randn((M, H), generator=g).to(BF)
        self.g = (1 + torch.randn(H, generator=g) / 8).to(BF)
        self.ids = np.stack([rng.permutation(E)[:topk] for _ in range(M)]).astype(np.int32)
        self.map = rng.integers(-1, L, M).astype(np.int32)
        self.tw = torch.softmax(torch.randn((M, topk), generator=g), 1)
        self.w13, self.s13 = fr.rand_weights(g, E, 2, I, H)
        self.w2, self.s2 = fr.rand_weights(g, E, 1, H, I)
        self.s13 *= 0.02 / self.s13.mean() / H ** 0.5
        self.s2 *= 0.02 / self.s2.mean() / I ** 0.5
        b = lambda *s: (torch.randn(s, generator=g) / s[-1] ** 0.5).to(BF)  # noqa: E731
        self.a13, self.b13 = b(2, L, E, r, H), b(2, L, E, I, r)
        self.a2, self.b2 = b(1, L, E, r, I), b(1, L, E, H, r)
        for n in ("x", "res", "g", "tw", "w13", "s13", "w2", "s2", "a13", "b13", "a2", "b2"):
            setattr(self, "d_" + n, getattr(self, n).to(DEV))
        self.d_ids, self.d_map = gh.i32_dev(self.ids), gh.i32_dev(self.map)
        self.zero = torch.zeros(M, dtype=torch.int32, device=DEV)
        e = lambda *s: torch.empty(s, dtype=BF, device=DEV)  # noqa: E731
        self.ro, self.hid, self.h = e(M, H), e(M, H), e(M * topk, I)
        self.y, self.y2 = e(M, topk, 2 * I), e(M, topk, H)
        self.x8, self.h8 = mla.alloc_fp8_rows(M, H, DEV), mla.alloc_fp8_rows(M * topk, I, DEV)
        self.al = mla.alloc_align_output(M, topk, E, L, B, DEV)
        self.base = mla.alloc_align_output(M, topk, E, 1, B, DEV)

    def run(self):
        mla.moe_lora_align(self.d_ids, self.zero, self.E, 1, self.B, out=self.base)
        mla.moe_lora_align(self.d_ids, self.d_map, self.E, self.L, self.B, out=self.al)
        mla.moe_lora_rms_norm_fp8(self.d_x, self.d_g, residual=self.d_res, residual_out=self.ro,
                                  y=self.hid, out=self.x8)
        mla.moe_lora_fp8_moe_gemm(self.x8, self.d_w13, self.d_s13, self.base, None, self.y,
                                  mul_routed_weight=False)
        mla.fused_moe_lora(self.hid, self.d_a13, self.d_b13, self.al, None, self.y,
                           mul_routed_weight=False, add_inputs=True)
        mla.moe_lora_silu_mul_fp8(self.y, h=self.h, out=self.h8)
        mla.moe_lora_fp8_moe_gemm(self.h8, self.d_w2, self.d_s2, self.base, self.d_tw, self.y2,
                                  mul_routed_weight=True, x_per_pair=True)
        mla.fused_moe_lora(self.h, self.d_a2, self.d_b2, self.al, self.d_tw, self.y2,
                           mul_routed_weight=True, add_inputs=True, x_per_pair=True)
        return self.y2


@pytest.mark.parametrize("M,B", [(1, 16), (16, 16), (150, 64)])
def test_layer_step_by_step(M, B):
    """norm, w13, adapters, activation, w2, adapters: each step's output against float64 on the
    step's own inputs, in one run."""
    la = Layer(M, 40 + M, B=B)
    orc = oracle.load()
    la.run()
    y2 = la.y2.cpu()
    h, v = fr.rms_norm(la.x, la.g, 1e-6, la.res)
    assert torch.equal(la.ro.cpu().to(D), h)
    fr.check_rows(la.x8.q, la.x8.scales, v, NORM_REL)
    fr.check_bf16(la.hid, v, NORM_REL * v.abs())
    # each projection and its adapters: the product's error, its rounding to bf16 before the adapters
    # add to it, and their own tolerance; the adapters' delta in float64 from the oracle
    bits = lambda t: t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)  # noqa: E731

    def check(y, x8, w, s, x, a, b, per_pair, mul):
        K, N = w.shape[-1], y.shape[-1]
        xq, xs = x8.q.cpu(), x8.scales.cpu()
        base = torch.zeros((M * la.topk, N), dtype=D)
        tol = torch.zeros((M * la.topk, N), dtype=D)
        for e, p in fr.pairs_of(la.ids, la.E).items():
            r = p if per_pair else p // la.topk
            f = la.tw.view(-1)[p].to(D)[:, None] if mul else 1.0
            ref, mag = fr.gemm(xq.view(torch.uint8)[r].view(fr.F8), xs[:, r], w[e], s[e])
            base[p], err = ref * f, fr.gemm_err(mag * f, K) + mag * f * 2.0 ** -24
            tol[p] = 2.0 ** -8 * (base[p].abs() + err) + err
        delta = orc.fused(bits(x), bits(a), bits(b), la.ids, la.map, la.tw.numpy(),
                          np.zeros(base.shape, np.uint16), mul, False, x_per_pair=per_pair)
        ref = base + torch.from_numpy(delta)
        err = (y.cpu().to(D).view(M * la.topk, N) - ref).abs()
        assert bool((err <= tol + gh.TOL * (1 + ref.abs())).all())

    check(la.y, la.x8, la.w13, la.s13, la.hid, la.a13, la.b13, False, False)
    v2 = fr.silu_mul(la.y.cpu().view(M * la.topk, -1))
    fr.check_rows(la.h8.q, la.h8.scales, v2, SILU_REL)
    check(y2, la.h8, la.w2, la.s2, la.h, la.a2, la.b2, True, True)


def test_layer_captured_and_replayed_with_eager_work_between():
    la = Layer(16, 77)
    want = la.run().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        la.run()
    other = Layer(24, 78)
    for i in range(4):
        la.y.fill_(float(i))
        la.y2.fill_(float(i))
        graph.replay()
        other.run()
        torch.cuda.synchronize()
        assert torch.equal(la.y2.view(torch.int16), want.view(torch.int16)), f"replay {i}"


def test_two_calls_on_two_streams():
    a, b = Layer(16, 80), Layer(150, 81, B=64)
    wa, wb = a.run().clone(), b.run().clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a.y2.zero_(), b.y2.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        a.run()
    with torch.cuda.stream(s2):
        b.run()
    torch.cuda.synchronize()
    assert torch.equal(a.y2.view(torch.int16), wa.view(torch.int16))
    assert torch.equal(b.y2.view(torch.int16), wb.view(torch.int16))


def test_stream_argument():
    xq, xs, wq, ws = _gemm(20, 272, 136, 1, 3)
    s = torch.cuda.Stream()
    x, w, sc = _rows(xq, xs), wq.to(DEV), ws.to(DEV)
    want = mla.moe_lora_fp8_gemm(x, w, sc)
    torch.cuda.synchronize()
    y = torch.zeros_like(want)
    s.wait_stream(torch.cuda.current_stream())
    mla.moe_lora_fp8_gemm(x, w, sc, y, stream=s)
    s.synchronize()
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))


# Enough weights for each of the tiles, and the 64-column rows kernel, at odd sizes: the same list's
# columns as MOE.
MOE_WIDE = [
    (1040, 1, 2192, 1032, 1, 4, 64, False, True, "invalid"),
    (400, 4, 2064, 520, 1, 4, 16, True, False, "uniform"),
    (700, 2, 1168, 520, 2, 7, 32, False, True, "twice"),
    (60, 8, 400, 1288, 2, 20, 32, False, False, "uniform"),
    (700, 2, 1168, 520, 2, 7, 128, True, True, "invalid"),
    (600, 2, 1040, 776, 2, 4, 128, False, False, "twice"),
    (1000, 4, 784, 1544, 1, 3, 32, False, True, "invalid"),
    (1000, 2, 656, 1032, 2, 3, 128, True, True, "uniform"),
    (800, 2, 656, 1032, 2, 4, 64, False, True, "one"),
    (70, 2, 784, 456, 2, 16, 64, False, True, "invalid"),
    (300, 4, 528, 776, 1, 48, 16, True, False, "uniform"),
    (90, 2, 272, 2056, 1, 8, 128, False, True, "one"),
    (250, 2, 144, 1080, 1, 16, 64, False, True, "invalid"),
    (3, 2, 1328, 1304, 2, 64, 64, False, True, "uniform"),
]


@pytest.mark.parametrize("case", MOE_WIDE)
def test_moe_gemm_wide(case):
    test_moe_gemm(case)


@pytest.mark.parametrize("case", MOE_WIDE)
def test_moe_gemm_wide_whole_numbers_exactly(case):
    test_moe_gemm_whole_numbers_exactly(case)


@pytest.mark.parametrize("M,K,Ns,B", [(60, 272, 136, 16), (120, 400, 1288, 64), (800, 784, 1544, 32),
                                      (800, 784, 1544, 128)])
def test_moe_gemm_reads_no_meaning_behind_the_last_block(M, K, Ns, B):
    """Whatever the align outputs hold behind num_tokens_post_padded, and experts out of range."""
    case = (M, 2, K, Ns, 1, 4, B, True, True, "uniform")
    ids, xq, xs, wq, ws, tw, y0 = _moe(*case)
    al = _base_align(ids, 4, B)
    n = int(al.num_tokens_post_padded.item())
    al.sorted_token_ids.view(-1)[n:] = 0
    al.expert_ids.view(-1)[n // B:] = 3
    al.expert_ids[0, :n // B][al.expert_ids[0, :n // B] == 2] = -1
    y = y0.to(DEV)
    mla.moe_lora_fp8_moe_gemm(_rows(xq, xs), wq.to(DEV), ws.to(DEV), al, tw.to(DEV), y,
                              mul_routed_weight=True, x_per_pair=True)
    _check_moe(y, y0, ids, xq, xs, wq, ws, tw, True, True, skip=(2,))


# Enough columns for the tiles, and for 32 columns a workgroup, at odd sizes: the same list's columns
# as GEMM.
GEMM_WIDE = [(3, 272, 6040, 2), (16, 144, 5000, 1), (90, 656, 4104, 1), (70, 1168, 2056, 2),
             (300, 1168, 2056, 1), (200, 2192, 4104, 1), (500, 784, 4104, 1), (520, 1296, 4104, 1),
             (1000, 1040, 5128, 1), (777, 2064, 3592, 1)]


@pytest.mark.parametrize("M,K,Ns,S", GEMM_WIDE)
def test_gemm_wide(M, K, Ns, S):
    test_gemm(M, K, Ns, S)


@pytest.mark.parametrize("M,K,Ns,S", GEMM_WIDE)
def test_gemm_wide_whole_numbers_exactly(M, K, Ns, S):
    test_gemm_whole_numbers_exactly(M, K, Ns, S)


@pytest.mark.parametrize("M,K,Ns", [(16, 144, 5000), (90, 656, 4104), (500, 784, 4104), (1000, 1040, 5128)])
def test_gemm_wide_nan_stays_in_its_row_and_column(M, K, Ns):
    xq, xs, wq, ws = _gemm(M, K, Ns, 1, M)
    ref, mag = fr.gemm(xq, xs, wq, ws)
    xq[M - 2, K - 6] = float("nan")
    wq[0, Ns - 3, 3] = float("nan")
    y = mla.moe_lora_fp8_gemm(_rows(xq, xs), wq.to(DEV), ws.to(DEV)).cpu()
    assert torch.isnan(y[M - 2]).all() and torch.isnan(y[:, Ns - 3]).all()
    rows, cols = torch.arange(M) != M - 2, torch.arange(Ns) != Ns - 3
    fr.check_bf16(y[rows][:, cols], ref[rows][:, cols], fr.gemm_err(mag, K)[rows][:, cols])


def test_gemm_many_rows_of_few_columns():
    """Straight from memory at many rows: the scales' offsets, and K of many blocks."""
    test_gemm_whole_numbers_exactly(5512, 352, 24, 1)
    test_gemm_whole_numbers_exactly(1463, 4016, 40, 1)


# 32 x 32 tiles, whose stages hold four blocks of K: K that ends inside a stage and inside a block.
GEMM_PARTS = [(60, 4112, 4040, 1), (97, 6160, 1032, 2), (40, 5008, 3592, 1), (130, 3600, 1544, 1),
              (1040, 4240, 200, 1), (20, 8336, 7000, 1), (33, 2576, 3528, 1), (64, 6032, 1032, 3)]


@pytest.mark.parametrize("M,K,Ns,S", GEMM_PARTS)
def test_gemm_parts(M, K, Ns, S):
    test_gemm(M, K, Ns, S)


@pytest.mark.parametrize("M,K,Ns,S", GEMM_PARTS)
def test_gemm_parts_whole_numbers_exactly(M, K, Ns, S):
    test_gemm_whole_numbers_exactly(M, K, Ns, S)


@pytest.mark.parametrize("M,K,Ns", [(3, 272, 264), (60, 4112, 4040), (33, 2576, 3528), (300, 1168, 2056)])
def test_gemm_infinite_scales_of_columns_stay_there(M, K, Ns):
    """The scale behind a column block's last one is the next block's first."""
    g = gen(M)
    xq, xs = fr.whole_rows(g, M, K)
    wq, ws = fr.whole_weights(g, 1, Ns, K)
    ws[0, 1, 0] = float("inf")
    ws[0, -1, 0] = float("nan")
    y = mla.moe_lora_fp8_gemm(_rows(xq, xs), wq.to(DEV), ws.to(DEV)).cpu()
    keep = torch.ones(Ns, dtype=torch.bool)
    keep[128:256] = keep[(Ns - 1) // 128 * 128:] = False
    ws[~torch.isfinite(ws)] = 1.0
    ref, _ = fr.gemm(xq, xs, wq, ws)
    assert torch.equal(y[:, keep], ref[:, keep].float().to(BF))
    assert not bool(torch.isfinite(y[:, ~keep]).any())
