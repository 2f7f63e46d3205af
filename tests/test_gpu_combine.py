"""The combine on the GPU against float64."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_lora_adapter_amd as mla  # noqa: E402
import base_reference as br  # noqa: E402
from gpu_helpers import DEV  # noqa: E402

BF = torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def dev(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("M,topk,N", [(1, 1, 8), (3, 2, 24), (16, 4, 2880), (7, 8, 2048), (333, 6, 136),
                                      (65, 3, 1032), (2, 33, 64), (1000, 5, 8), (5, 64, 40)])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("ids", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_combine(M, topk, N, weights, ids, residual):
    g = gen(M + topk + N)
    y = torch.randn((M, topk, N), generator=g).to(BF)
    w = torch.rand((M, topk), generator=g) if weights else None
    i = torch.randint(-2, 12, (M, topk), generator=g, dtype=torch.int32) if ids else None
    r = (3 * torch.randn((M, N), generator=g)).to(BF) if residual else None
    out, err = br.combine(y, w, i, 10, r)
    kw = dict(topk_weights=dev(w), topk_ids=dev(i), E=10)
    got = mla.moe_lora_combine(y.to(DEV), residual=dev(r), **kw)
    br.check(got, out, err)
    if residual:  # onto the residual itself
        rd = dev(r)
        again = mla.moe_lora_combine(y.to(DEV), rd, residual=rd, **kw)
        assert again is rd and torch.equal(rd, got)


def test_left_out_pairs_are_not_read():
    """Rows that no product wrote may hold anything: NaN there reaches nothing, and a token without an
    expert here is its residual, or zero."""
    g = gen(1)
    y = torch.randn((6, 3, 64), generator=g).to(BF)
    ids = torch.tensor([[0, 1, 2], [-1, 1, 9], [-1, -1, -1], [8, 7, 6], [0, -1, 2 ** 31 - 1],
                        [-2 ** 31, 3, 4]], dtype=torch.int32)
    clean = y.clone()
    y[(ids < 0) | (ids >= 8)] = float("nan")
    r = torch.randn((6, 64), generator=g).to(BF)
    for res in (None, r):
        out, err = br.combine(clean, None, ids, 8, res)
        got = mla.moe_lora_combine(y.to(DEV), topk_ids=ids.to(DEV), E=8, residual=dev(res))
        br.check(got, out, err)
        assert torch.equal(got[2].cpu(), torch.zeros(64, dtype=BF) if res is None else res[2])
    y = clean.clone()
    y[3, 0, 5] = float("nan")
    got = mla.moe_lora_combine(y.to(DEV)).cpu()
    assert torch.isnan(got[3, 5]) and int(torch.isnan(got).sum()) == 1


def test_out_given_on_another_stream_and_no_rows():
    y = torch.ones((5, 2, 16), dtype=BF, device=DEV)
    out = torch.full((6, 16), 9.0, dtype=BF, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    mla.moe_lora_combine(y, out[:5], stream=s)
    s.synchronize()
    assert torch.all(out[:5] == 2) and torch.all(out[5] == 9)
    assert mla.moe_lora_combine(y[:0]).shape == (0, 16)
