"""Every kernel of the bf16 products at sizes that leave its last tiles short, against float64: exactly
on whole numbers, with each activation, operand and output type, in place, and around NaN."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_lora_adapter_amd as mla  # noqa: E402
import base_reference as br  # noqa: E402
import product_tiles as pt  # noqa: E402
from gpu_helpers import DEV  # noqa: E402

BF, F32, D = torch.bfloat16, torch.float32, torch.float64


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def whole(g, *shape):
    """Whole numbers up to 4: a sum of K products, the bias, the delta and the residual stays below 16 K
    + 12 < 2^24, and fp32 holds it exactly."""
    return torch.randint(-4, 5, shape, generator=g, device=DEV).to(BF)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def rows(g, M, K):
    return (normal(g, M, K) * (1 + 30 * (torch.rand(K, generator=g, device=DEV) < 0.01))).to(BF)


def weights(g, *shape):
    return (normal(g, *shape) * shape[-1] ** -0.5).to(BF)


def close(got, ref, err):
    """As base_reference.check, on the device."""
    half = {BF: 2.0 ** -8, F32: 2.0 ** -24}[got.dtype]
    tol = half * (ref.abs() + err) + err + 2.0 ** -133
    off = (got.to(D) - ref).abs()
    assert torch.all(off <= tol), f"worst {float((off / tol).max()):.3f} of the bound"


def same_bits(a, b):
    kind = torch.int16 if a.dtype is BF else torch.int32
    return torch.equal(a.view(kind), b.view(kind))


def acts(gated):
    return pt.GATED if gated else pt.UNGATED


# ---------------------------------------------------------------- dense

@pytest.mark.parametrize("kernel,gated,size", **pt.flat(pt.DENSE, False))
def test_dense_whole_numbers_exactly(kernel, gated, size):
    M, K, Ns, S = size
    assert mla.gemm_kernel_name(*size) == kernel
    g = gen(M + K + Ns)
    x, w = whole(g, M, K), whole(g, S, Ns, K)
    b, d, r = whole(g, S * Ns), whole(g, M, S * Ns), whole(g, M, S * Ns)
    want = x.to(D) @ w.view(-1, K).to(D).t()
    assert torch.equal(mla.moe_lora_gemm(x, w, out_dtype=F32), want.to(F32))
    assert torch.equal(mla.moe_lora_gemm(x, w), want.to(BF))
    want = want + b.to(D) + d.to(D) + r.to(D)
    assert torch.equal(mla.moe_lora_gemm(x, w, bias=b, delta=d, residual=r, out_dtype=F32), want.to(F32))
    assert torch.equal(mla.moe_lora_gemm(x, w, bias=b, delta=d, residual=r), want.to(BF))


@pytest.mark.parametrize("kernel,gated,size", **pt.flat(pt.DENSE))
def test_dense_epilogue(kernel, gated, size):
    """Each activation with all operands into either type, and with every other choice of operands."""
    M, K, Ns, S = size
    g = gen(M * 3 + K + Ns)
    No = Ns if gated else S * Ns
    x, w = rows(g, M, K), weights(g, S, Ns, K)
    b, d = (2 * normal(g, S * Ns)).to(BF), normal(g, M, S * Ns).to(BF)
    r = (3 * normal(g, M, No)).to(BF)
    for n, act in enumerate(acts(gated)):
        assert mla.gemm_kernel_name(*size, act) == kernel
        for keep in (7, (n + M) % 7):
            kw = dict(bias=b if keep & 1 else None, delta=d if keep & 2 else None, residual=r if keep & 4 else None)
            ref, err = br.product(x, w, act=act, **kw)
            for out in (BF, F32):
                y = torch.full((M + 1, No), 7.0, dtype=out, device=DEV)
                mla.moe_lora_gemm(x, w, y[:M], activation=act, **kw)
                close(y[:M], ref, err)
                assert torch.all(y[M] == 7), "the row behind the last"
                assert same_bits(y[:M], mla.moe_lora_gemm(x, w, activation=act, out_dtype=out, **kw))


@pytest.mark.parametrize("kernel,gated,size", **pt.flat(pt.DENSE))
def test_dense_in_place(kernel, gated, size):
    """y may be the residual, and, ungated, the delta."""
    M, K, Ns, S = size
    g = gen(M + 1)
    x, w = rows(g, M, K), weights(g, S, Ns, K)
    t = normal(g, M, Ns if gated else S * Ns).to(BF)
    for act in acts(gated):
        for name in ("residual",) if gated else ("residual", "delta"):
            want = mla.moe_lora_gemm(x, w, activation=act, **{name: t})
            y = t.clone()
            mla.moe_lora_gemm(x, w, y, activation=act, **{name: y})
            assert same_bits(y, want)


@pytest.mark.parametrize("kernel,gated,size", **pt.flat(pt.DENSE))
def test_dense_nan_stays_in_its_row_and_column(kernel, gated, size):
    M, K, Ns, S = size
    act = "silu_mul" if gated else None
    g = gen(M + 2)
    x, w = rows(g, M, K), weights(g, S, Ns, K)
    clean = mla.moe_lora_gemm(x, w, activation=act)
    x[M - 1, K - 1] = float("nan")
    w[S - 1, Ns - 1, K // 2] = float("nan")
    y = mla.moe_lora_gemm(x, w, activation=act)
    assert torch.isnan(y[M - 1]).all() and torch.isnan(y[:, -1]).all()
    assert same_bits(y[:M - 1, :-1].contiguous(), clean[:M - 1, :-1].contiguous())


# ---------------------------------------------------------------- grouped

def routed(g, M, topk, E, skew):
    """Distinct experts of every token, a few of them popular, some pairs without one."""
    p = -skew * torch.log(torch.arange(1, E + 1, device=DEV).float())
    u = torch.rand((M, E), generator=g, device=DEV).clamp(1e-6, 1 - 1e-6)
    ids = torch.topk(p - torch.log(-torch.log(u)), topk, dim=1).indices.int()
    return torch.where(torch.rand((M, topk), generator=g, device=DEV) < 0.05, torch.full_like(ids, -1), ids)


def align(ids, E, B):
    return mla.moe_lora_align(ids.contiguous(), torch.zeros(ids.shape[0], dtype=torch.int32, device=DEV), E, 1, B)


def expected(x, w, ids, b, d, act, wt, per_pair, before):
    """(y, its error) of every pair; one without an expert keeps its row."""
    E, topk = w.shape[0], ids.shape[1]
    pairs = ids.reshape(-1)
    ref = before.to(D).view(pairs.numel(), -1).clone()
    err = torch.zeros_like(ref)
    for e in range(E):
        p = (pairs == e).nonzero().view(-1)
        if p.numel():
            ref[p], err[p] = br.product(x[p if per_pair else p // topk], w[e], None if b is None else b[e],
                                        None if d is None else d.view(pairs.numel(), -1)[p], act, None,
                                        None if wt is None else wt.view(-1)[p])
    return ref, err


@pytest.mark.parametrize("kernel,gated,size", **pt.flat(pt.GROUPED))
@pytest.mark.parametrize("skew", [0.0, 1.2])
def test_grouped(kernel, gated, size, skew):
    M, topk, E, K, Ns, S, B = size
    No = Ns if gated else S * Ns
    for n, act in enumerate(acts(gated)):
        per_pair, mul = bool((M + n) % 2), bool((M + n) % 3)
        assert mla.moe_gemm_kernel_name(M, topk, K, Ns, S, E, B, per_pair, act) == kernel
        g = gen(M + K + n)
        ids = routed(g, M, topk, E, skew)
        al = align(ids, E, B)
        x, w = rows(g, M * topk if per_pair else M, K), weights(g, E, S, Ns, K)
        b, d = normal(g, E, S * Ns).to(BF), normal(g, M, topk, S * Ns).to(BF)
        wt = torch.softmax(normal(g, M, topk), 1)
        before = normal(g, M, topk, No).to(BF)
        for keep in (3, n):
            kw = dict(bias=b if keep & 1 else None, delta=d if keep & 2 else None)
            y = before.clone()
            mla.moe_lora_moe_gemm(x, w, al, wt, y, mul_routed_weight=mul, x_per_pair=per_pair, activation=act, **kw)
            ref, err = expected(x, w, ids, kw["bias"], kw["delta"], act, wt if mul else None, per_pair, before)
            close(y.view(M * topk, No), ref, err)
            gone = ids.reshape(-1) < 0
            assert same_bits(y.view(M * topk, No)[gone], before.view(M * topk, No)[gone])
            again = before.clone()
            mla.moe_lora_moe_gemm(x, w, al, wt, again, mul_routed_weight=mul, x_per_pair=per_pair, activation=act, **kw)
            assert same_bits(y, again)


@pytest.mark.parametrize("kernel,gated,size", **pt.flat(pt.GROUPED, False))
def test_grouped_whole_numbers_exactly(kernel, gated, size):
    M, topk, E, K, Ns, S, B = size
    assert mla.moe_gemm_kernel_name(M, topk, K, Ns, S, E, B) == kernel
    g = gen(M + K)
    ids = routed(g, M, topk, E, 0.8)
    x, w = whole(g, M, K), whole(g, E, S, Ns, K)
    b, d = whole(g, E, S * Ns), whole(g, M, topk, S * Ns)
    wt = torch.randint(1, 5, (M, topk), generator=g, device=DEV).float()
    y = torch.full((M, topk, S * Ns), 3.0, dtype=BF, device=DEV)
    want, _ = expected(x, w, ids, b, d, None, wt, False, y)
    mla.moe_lora_moe_gemm(x, w, align(ids, E, B), wt, y, mul_routed_weight=True, bias=b, delta=d)
    assert torch.equal(y.view(M * topk, -1), want.to(BF))


@pytest.mark.parametrize("act,S,Ns,mul", [(None, 1, 72, True), (None, 2, 264, False), ("silu_mul", 2, 136, True)])
def test_grouped_over_two_launches(act, S, Ns, mul):
    """More align blocks than one launch of the tiles takes (16384), with an expert's run across the
    border: the second launch's blocks, biases and weights are its own."""
    M, topk, E, K, B = 150001, 2, 3, 72, 16
    assert "tile" in mla.moe_gemm_kernel_name(M, topk, K, Ns, S, E, B, False, act)
    g = gen(Ns)
    ids = torch.randint(0, E, (M, topk), generator=g, device=DEV, dtype=torch.int32)
    al = align(ids, E, B)
    blocks, eids = int(al.num_tokens_post_padded[0]) // B, al.expert_ids[0]
    assert blocks > 16384 + 1000 and int(eids[16383]) == int(eids[16384])
    x, w, b = whole(g, M, K), whole(g, E, S, Ns, K), whole(g, E, S * Ns)
    wt = torch.randint(1, 5, (M, topk), generator=g, device=DEV).float()
    No = Ns if act else S * Ns
    y = torch.full((M, topk, No), 3.0, dtype=BF, device=DEV)
    want, err = expected(x, w, ids, b, None, act, wt if mul else None, False, y)
    mla.moe_lora_moe_gemm(x, w, al, wt, y, mul_routed_weight=mul, bias=b, activation=act)
    if act:
        close(y.view(M * topk, No), want, err)
    else:
        assert torch.equal(y.view(M * topk, No), want.to(BF))


@pytest.mark.parametrize("M,Ns,S,act", [(1, 8, 1, None), (5, 136, 2, "silu_mul"), (70, 264, 1, None), (300, 504, 1, None)])
def test_longest_k(M, Ns, S, act):
    """K of 2^21, the most: rows of 4 MiB, and columns behind the last one at offsets towards 4 GiB.  Sums
    of zeros and ones of either sign stay below 2^24."""
    K = 1 << 21
    g = gen(M)
    x = torch.randint(-1, 2, (M, K), generator=g, device=DEV, dtype=torch.int8).to(BF)
    w = torch.randint(-1, 2, (S, Ns, K), generator=g, device=DEV, dtype=torch.int8).to(BF)
    y = mla.moe_lora_gemm(x, w, out_dtype=F32)
    want = torch.zeros((M, S * Ns), dtype=D, device=DEV)
    for k in range(0, K, 1 << 16):
        want += x[:, k:k + (1 << 16)].to(D) @ w.view(-1, K)[:, k:k + (1 << 16)].to(D).t()
    assert torch.equal(y, want.to(F32))
    if act:
        z = mla.moe_lora_gemm(x, w, activation=act, out_dtype=F32)
        close(z, br.activate(want, act), br.activate_err(want, torch.zeros_like(want), act))
