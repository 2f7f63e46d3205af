"""The 8-bit base side where its definition decides: roundings on exact ties, the largest launches,
buffers of other streams, and ids outside their range."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_lora_adapter_amd as mla  # noqa: E402
import fp8_reference as fr  # noqa: E402
import gpu_helpers as gh  # noqa: E402

DEV, BF = gh.DEV, torch.bfloat16


# ---------------------------------------------------------------- rounding
# Inputs whose fp32 value is known to the last bit, so that the scales and the e4m3 values follow
# from the definition exactly: scale = max(2^-40, largest) / 448, q = e4m3(value / scale), the two
# quotients rounded to fp32.  bf16 values over a bf16 maximum meet ties between two e4m3 values;
# a product with the reciprocal breaks some of them the other way.

def _rows_exactly(out, v):
    """Returns in how many places the reciprocal's product would differ."""
    K = v.shape[1]
    s = torch.stack([v[:, k:k + 128].abs().max(1).values.clamp(min=fr.MIN_AMAX) / fr.F8_MAX
                     for k in range(0, K, 128)])
    wide = s.t().repeat_interleave(128, 1)[:, :K]
    q = (v / wide).to(fr.F8).view(torch.uint8)
    assert torch.equal(out.scales.cpu(), s)
    assert torch.equal(out.q.cpu().view(torch.uint8), q)
    return int((q != (v * (1.0 / wide)).to(fr.F8).view(torch.uint8)).sum())


@pytest.mark.parametrize("H,weights", [(1024, 16), (2048, 2), (4096, 2), (8192, 2), (65528, 1)])
def test_rms_norm_rounds_the_quotient(H, weights):
    """x = +-2 in every place: the mean of the squares is 4 and the norm +-1 times the weight."""
    g, differ = torch.Generator().manual_seed(H), 0
    for _ in range(weights):
        x = (2.0 * (2 * torch.randint(0, 2, (5, H), generator=g) - 1)).to(BF)
        w = torch.randn(H, generator=g).to(BF)
        out = mla.moe_lora_rms_norm_fp8(x.to(DEV), w.to(DEV), eps=0.0)
        differ += _rows_exactly(out, x.float() * 0.5 * w.float())
    assert differ > 0, "the case does not tell the two apart"


@pytest.mark.parametrize("P,I", [(300, 136), (64, 1160), (33, 2880)])
def test_silu_mul_rounds_the_quotient(P, I):
    """silu(64) is 64 in fp32."""
    u = torch.randn((P, I), generator=torch.Generator().manual_seed(I)).to(BF)
    y = torch.cat([torch.full_like(u, 64.0), u], 1)
    differ = _rows_exactly(mla.moe_lora_silu_mul_fp8(y.to(DEV)), 64.0 * u.float())
    assert differ > 0, "the case does not tell the two apart"


# ---------------------------------------------------------------- launches

@pytest.mark.parametrize("M,K,Ns,S", [(1, 16, 8, 1 << 23), (300, 512, 8, 1 << 20)])
def test_gemm_more_slices_than_one_launch_of_few_rows_takes(M, K, Ns, S):
    """2^23 workgroups of 512 threads are 2^32 threads, which no launch has.  Whole numbers, every
    sum a multiple of 1/4 below 2^15: exact in fp32 in any order."""
    g = torch.Generator(device=DEV).manual_seed(S)
    whole = lambda *s: torch.randint(-4, 5, s, device=DEV, generator=g).float()  # noqa: E731
    x, w = whole(M, K), torch.empty((S, Ns, K), dtype=fr.F8, device=DEV)
    step = S // 16
    for i in range(0, S, step):
        w[i:i + step] = whole(step, Ns, K).to(fr.F8)
    xs = 2.0 ** torch.randint(-1, 2, (fr.blocks(K), M), device=DEV, generator=g).float()
    ws = 2.0 ** torch.randint(-1, 2, (S, 1, fr.blocks(K)), device=DEV, generator=g).float()
    y = mla.moe_lora_fp8_gemm(mla.Fp8Rows(x.to(fr.F8), xs), w, ws)
    wide = x * xs.t().repeat_interleave(128, 1)[:, :K]
    for i in range(0, S, step):
        wf = w[i:i + step].float() * ws[i:i + step].repeat_interleave(128, 2)[:, :, :K]
        want = (wide @ wf.view(step * Ns, K).t().contiguous()).to(BF)
        assert torch.equal(y[:, i * Ns:(i + step) * Ns], want)


# ---------------------------------------------------------------- streams

def _stream_of(t):
    """The stream that the allocator gave a tensor's memory to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


def test_buffers_of_a_call_on_a_given_stream_are_that_streams():
    """A buffer that a call allocates is taken from the stream that the call writes it on: memory
    that work of the current stream may still be using, or is given next, is another."""
    g = torch.Generator().manual_seed(9)
    xb, w = torch.randn((40, 272), generator=g).to(BF).to(DEV), torch.ones(272, dtype=BF, device=DEV)
    wq, ws = fr.rand_weights(g, 1, 136, 272)
    wq, ws = wq.to(DEV), ws.to(DEV)
    want = mla.moe_lora_rms_norm_fp8(xb, w)
    want_h = mla.moe_lora_silu_mul_fp8(xb)
    want_y = mla.moe_lora_fp8_gemm(want, wq, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    n = mla.moe_lora_rms_norm_fp8(xb, w, stream=s)
    h = mla.moe_lora_silu_mul_fp8(xb, stream=s)
    y = mla.moe_lora_fp8_gemm(n, wq, ws, stream=s)
    s.synchronize()
    for t in (n.q, n.scales, h.q, h.scales, y):
        assert _stream_of(t) == s.cuda_stream
    for a, b in ((n.q, want.q), (h.q, want_h.q)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(n.scales, want.scales) and torch.equal(h.scales, want_h.scales)
    assert torch.equal(y.view(torch.int16), want_y.view(torch.int16))
    assert torch.cuda.current_stream() != s


# ---------------------------------------------------------------- ids outside their range

def _mask(ids, B, used, kind):
    """`ids` (one slot's sorted pairs) with some taken out, wherever in a block they stand."""
    at = torch.arange(used)
    gone = {"first of a block": at % B == 0,
            "first of 16": at % 16 == 0,
            "first 16 of a block": at % B < 16,
            "all but the last of 16": at % 16 != 15,
            "every third": at % 3 == 1,
            "all but the last of a block": at % B != B - 1}[kind]
    out = ids.clone()
    bad = torch.tensor([-1, 1 << 30, -(1 << 31)], dtype=torch.int32)
    out[:used][gone] = bad[torch.arange(int(gone.sum())) % 3]
    return out


KINDS = ["first of a block", "first of 16", "first 16 of a block", "all but the last of 16",
         "every third", "all but the last of a block"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,topk,K,Ns,S,E,B,per_pair", [
    (60, 2, 272, 136, 1, 4, 16, False),        # few rows, 32 columns
    (200, 2, 272, 136, 1, 16, 128, True),      # the same, pieces of a block in turn
    (600, 1, 144, 72, 1, 3, 64, False),        # the same, several of them at once
    (90, 2, 272, 2056, 1, 8, 128, False),      # few rows, 64 columns
    (400, 8, 272, 1288, 1, 64, 16, False),     # tiles of 64 rows
    (700, 2, 1168, 520, 2, 7, 32, True),
    (700, 2, 1168, 520, 2, 7, 128, True),      # tiles of 128 rows
    (1000, 4, 784, 1544, 1, 3, 32, False),
    (900, 8, 64, 1544, 1, 64, 128, False),     # tiles of 256 rows
    (2500, 4, 128, 1032, 1, 64, 64, True)])
def test_moe_gemm_passes_over_pairs_outside_their_range(M, topk, K, Ns, S, E, B, per_pair, kind):
    """Ids that are no pair's, anywhere in a block: the others' rows are computed, and no more."""
    rng, g = np.random.default_rng(M + K), torch.Generator().manual_seed(M)
    ids = rng.integers(0, E, (M, topk)).astype(np.int32)
    xq, xs = fr.whole_rows(g, M * topk if per_pair else M, K)
    wq, ws = fr.whole_weights(g, E, S, Ns, K)
    tw = 2.0 ** torch.randint(-2, 3, (M, topk), generator=g).float()
    al = mla.moe_lora_align(gh.i32_dev(ids), torch.zeros(M, dtype=torch.int32, device=DEV), E, 1, B)
    used = int(al.num_tokens_post_padded.item())
    kept = _mask(al.sorted_token_ids[0].cpu(), B, used, kind)
    al.sorted_token_ids[0].copy_(kept)
    x, w, sc, dw = mla.Fp8Rows(xq.to(DEV), xs.to(DEV)), wq.to(DEV), ws.to(DEV), tw.to(DEV)
    y = torch.full((M, topk, S * Ns), 5.0, dtype=BF, device=DEV)
    mla.moe_lora_fp8_moe_gemm(x, w, sc, al, dw, y, mul_routed_weight=True, x_per_pair=per_pair)
    want = torch.full((M * topk, S * Ns), 5.0, dtype=BF, device=DEV)
    xw = fr.widen_rows(xq, xs).float().to(DEV)
    left = kept[:used]
    left = left[(left >= 0) & (left < M * topk)].long().to(DEV)
    flat, wt = gh.i32_dev(ids).view(-1), dw.view(-1)
    for e in range(E):
        p = left[flat[left] == e]
        if p.numel():
            d = xw[p if per_pair else p // topk] @ fr.widen_weights(wq[e], ws[e]).float().view(
                S * Ns, K).to(DEV).t().contiguous()
            want[p] = (d * wt[p][:, None]).to(BF)
    assert torch.equal(y.view(M * topk, S * Ns), want)
