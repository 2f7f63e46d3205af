"""The bf16 base side past 32-bit offsets, over many rows at once, and on two streams together."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_lora_adapter_amd as mla  # noqa: E402
import base_reference as br  # noqa: E402
from gpu_helpers import DEV  # noqa: E402

BF, D, NEG = torch.bfloat16, torch.float64, float("-inf")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def plain_route(x, bias, topk, sigmoid, n_group=1, topk_group=1, group_top=1):
    """Picks and renormalised weights in float64, all rows at once."""
    x = x.to(D)
    s = br.sigmoid(x) if sigmoid else torch.softmax(x, 1)
    key = s if bias is None else s + bias.to(D)
    key = torch.where(x == NEG, x, key)
    if n_group > 1:
        g = torch.sort(key.view(len(x), n_group, -1), dim=2, descending=True).values[:, :, :group_top]
        order = torch.sort(g.sum(2), dim=1, descending=True, stable=True).indices[:, :topk_group]
        kept = torch.zeros((len(x), n_group), dtype=torch.bool).scatter_(1, order, True)
        key = key.masked_fill(~kept.repeat_interleave(x.shape[1] // n_group, 1), NEG)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :topk]
    w = s.gather(1, ids)
    return ids.int(), w / w.sum(1, keepdim=True)


@pytest.mark.parametrize("E,topk,groups", [(64, 8, None), (256, 8, (8, 4, 2)), (60, 4, (5, 2, 2)), (100, 16, None)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_many_rows_by_score(E, topk, groups, sigmoid):
    """A wavefront takes several rows at once; a fifth of them have keys that fp32 cannot tell apart,
    next to rows that it can."""
    M = 20011
    g = gen(E + topk)
    x = 2 * torch.randn((M, E), generator=g)
    near = torch.rand(M, generator=g) < 0.2
    x[near] = 18 + torch.randint(0, 40, (int(near.sum()), E), generator=g).float() / 8 if sigmoid else \
        1 + torch.randint(0, 40, (int(near.sum()), E), generator=g).float() * 2.0 ** -20
    b = torch.where(torch.rand(E, generator=g) < 0.5, 0.0, 0.25)
    kw = {} if groups is None else dict(n_group=groups[0], topk_group=groups[1], group_top=groups[2])
    ids, w = mla.moe_lora_route(x.to(DEV), topk, scoring="sigmoid" if sigmoid else "softmax", bias=b.to(DEV), **kw)
    br.check_route((ids, w), plain_route(x, b, topk, sigmoid, **kw), 32.0)


def test_route_past_32_bit_offsets():
    M, E = (1 << 21) + 300, 1024
    x = torch.empty((M, E), dtype=BF, device=DEV).normal_()
    ids, w = mla.moe_lora_route(x, 2)
    for rows in (slice(0, 64), slice(M // 2, M // 2 + 64), slice(M - 64, M)):
        br.check_route((ids[rows], w[rows]), br.route(x[rows].cpu(), 2), 16.0)


def test_gemm_past_32_bit_offsets():
    M, N, K = 66001, 33000, 64
    x = torch.randint(-4, 5, (M, K), device=DEV).to(BF)
    w = torch.randint(-4, 5, (1, N, K), device=DEV).to(BF)
    y = torch.ones((M, N), dtype=BF, device=DEV)
    mla.moe_lora_gemm(x, w, y, residual=y)
    for r in (slice(0, 40), slice(M // 2, M // 2 + 40), slice(M - 300, M)):
        want = x[r].cpu().float() @ w[0].cpu().float().t() + 1
        assert torch.equal(y[r].cpu(), want.to(BF))


@pytest.mark.parametrize("topk,N", [(2, 32768)])
def test_moe_gemm_past_32_bit_offsets(topk, N):
    M, K, E = 33500, 16, 2
    g = gen(3)
    ids = torch.randint(0, E, (M, topk), generator=g, dtype=torch.int32)
    x = torch.randint(-4, 5, (M, K), generator=g).to(BF)
    w = torch.randint(-4, 5, (E, 1, N, K), generator=g).to(BF)
    al = mla.moe_lora_align(ids.to(DEV), torch.zeros(M, dtype=torch.int32, device=DEV), E, 1, 128)
    y = torch.empty((M, topk, N), dtype=BF, device=DEV)
    mla.moe_lora_moe_gemm(x.to(DEV), w.to(DEV), al, None, y, mul_routed_weight=False)
    for m in (0, 1, M // 2, M - 2, M - 1):
        for k in range(topk):
            want = x[m].float() @ w[int(ids[m, k]), 0].float().t()
            assert torch.equal(y[m, k].cpu(), want.to(BF))


def test_combine_past_32_bit_offsets():
    M, topk, N = 40003, 8, 8192
    y = torch.empty((M, topk, N), dtype=BF, device=DEV).normal_()
    out = mla.moe_lora_combine(y)
    for r in (slice(0, 8), slice(M // 2, M // 2 + 8), slice(M - 8, M)):
        br.check(out[r], *br.combine(y[r].cpu()))


def test_two_streams_at_once():
    """No call shares anything with another: the same work on two streams together, on different inputs,
    gives what each gives alone."""
    g = gen(4)
    M, E, topk, K, I, B = 200, 16, 4, 256, 136, 32
    w13, w2 = br.weights(g, E, 2, I, K).to(DEV), br.weights(g, E, 1, K, I).to(DEV)
    gate = br.weights(g, 1, E, K).to(DEV)
    xs = [br.rows(g, M, K).to(DEV) for _ in range(2)]
    zero = torch.zeros(M, dtype=torch.int32, device=DEV)

    def layer(x):
        ids, wt = mla.moe_lora_route(mla.moe_lora_gemm(x, gate, out_dtype=torch.float32), topk)
        al = mla.moe_lora_align(ids, zero, E, 1, B)
        h = torch.zeros((M, topk, I), dtype=BF, device=DEV)
        mla.moe_lora_moe_gemm(x, w13, al, None, h, mul_routed_weight=False, activation="silu_mul")
        y = torch.zeros((M, topk, K), dtype=BF, device=DEV)
        mla.moe_lora_moe_gemm(h.view(M * topk, I), w2, al, wt, y, mul_routed_weight=True, x_per_pair=True)
        return mla.moe_lora_combine(y, residual=x)

    want = [layer(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = []
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(layer(x))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("E", [8, 256])
def test_every_row_undecided(E):
    """More rows than the wavefronts take at once, all with equal scores: fp32 decides none of them."""
    M, topk = (2_500_000, 4) if E == 8 else (1_200_000, 8)
    g = torch.Generator(device=DEV).manual_seed(E)
    x = torch.randint(0, 2, (M, E), generator=g, device=DEV).to(torch.bfloat16)
    ids, w = mla.moe_lora_route(x, topk, scoring="sigmoid", bias=torch.zeros(E, device=DEV))
    # the ones first, each kind in ascending order
    at = torch.arange(E, device=DEV)
    want = torch.topk((1 - x.long()) * E + at, topk, dim=1, largest=False, sorted=True).values
    assert torch.equal(ids.long(), want % E)
    s = torch.sigmoid((want < E).double())
    # (the exponential, two quotients and up to 8 additions: below 32 half steps)
    assert torch.allclose(w.double(), s / s.sum(1, keepdim=True), rtol=2 ** -19, atol=0)
