"""The 8-bit base side where its definition decides: roundings on exact ties, the largest launches,
buffers of other streams, and ids outside their range."""
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
