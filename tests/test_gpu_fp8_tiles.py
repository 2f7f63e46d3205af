"""The e4m3 products' tiles where a workgroup takes several, in each size of the dense and the
grouped kernel that the lists of test_gpu_fp8.py give one tile a workgroup at most: pair lists and
weights used again, loads of the next tile behind the last one's, stores left in flight."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_lora_adapter_amd as mla  # noqa: E402
import fp8_reference as fr  # noqa: E402
import gpu_helpers as gh  # noqa: E402
import test_gpu_fp8 as base  # noqa: E402

DEV, BF = gh.DEV, torch.bfloat16


# Whole numbers, where any order of fp32 additions is exact.  64 x 64 tiles: 2 on each of 256 CUs
# at once.
@pytest.mark.parametrize("M,K,Ns,S", [(60000, 528, 64, 1), (70001, 128, 40, 1), (50005, 272, 64, 1),
                                      (18000, 656, 56, 4)])
def test_gemm_64x64_tiles_in_turn(M, K, Ns, S):
    base.test_gemm_many_tiles_exactly(M, K, Ns, S)


def _routing(rng, M, topk, E, kind):
    if kind == "skewed":  # an expert's share falls with its number; one takes several tiles' rows
        p = 1.0 / np.arange(1, E + 1)
        return rng.choice(E, (M, topk), p=p / p.sum()).astype(np.int32)
    return base._routing(rng, M, topk, E, kind)


# More tiles than the device holds at once (256): the tiles of 64 rows (three stages) and of 128
# rows (two), K of one block, of two, of the stages and of more, even, skewed and invalid routing.
@pytest.mark.parametrize("M,topk,K,Ns,S,E,B,kind", [
    (400, 8, 272, 1288, 1, 64, 16, "uniform"),
    (1200, 4, 400, 776, 1, 64, 32, "uniform"),
    (400, 8, 144, 1288, 1, 64, 64, "invalid"),
    (400, 8, 656, 1288, 1, 64, 16, "skewed"),
    (300, 8, 128, 2568, 1, 48, 64, "invalid"),
    (300, 8, 112, 2568, 1, 48, 32, "skewed"),
    (2048, 4, 272, 1032, 2, 64, 64, "uniform"),
    (1024, 4, 528, 1032, 2, 64, 16, "uniform"),
    (1024, 8, 128, 1288, 1, 128, 16, "invalid"),
    (1024, 8, 64, 1288, 1, 128, 128, "skewed"),
    (2048, 4, 400, 1032, 2, 64, 32, "skewed")])
@pytest.mark.parametrize("per_pair", [False, True])
def test_moe_gemm_tiles_in_turn(M, topk, K, Ns, S, E, B, kind, per_pair):
    ids = _routing(np.random.default_rng(M + E), M, topk, E, kind)
    g = torch.Generator().manual_seed(M + topk)
    xq, xs = fr.whole_rows(g, M * topk if per_pair else M, K)
    wq, ws = fr.whole_weights(g, E, S, Ns, K)
    tw = 2.0 ** torch.randint(-2, 3, (M, topk), generator=g).float()
    x, w, sc, dw = mla.Fp8Rows(xq.to(DEV), xs.to(DEV)), wq.to(DEV), ws.to(DEV), tw.to(DEV)
    y = torch.full((M, topk, S * Ns), 5.0, dtype=BF, device=DEV)
    mla.moe_lora_fp8_moe_gemm(x, w, sc, base._base_align(ids, E, B), dw, y, mul_routed_weight=True,
                              x_per_pair=per_pair)
    xw, want = base._wide(x.q, x.scales), torch.full((M * topk, S * Ns), 5.0, dtype=BF, device=DEV)
    flat, wt = gh.i32_dev(ids).view(-1), dw.view(-1)
    for e in range(E):
        p = (flat == e).nonzero().view(-1)
        d = xw[p if per_pair else p // topk] @ base._wide_w(w[e], sc[e]).view(S * Ns, K).t().contiguous()
        want[p] = (d * wt[p][:, None]).to(BF)
    assert torch.equal(y.view(M * topk, S * Ns), want)
