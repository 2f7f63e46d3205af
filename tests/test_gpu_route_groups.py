"""Groups whose best two keys nearly cancel: the sum is small and each key's rounding is not, and which
groups stay is still what float64 says."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_lora_adapter_amd as mla  # noqa: E402
import base_reference as br  # noqa: E402
from gpu_helpers import DEV  # noqa: E402

D, NEG = torch.float64, float("-inf")
# groups of whole lanes (E 4, 16, 32, 256, 512, 1024) and such whose keys go through LDS
SHAPES = [(4, 2, 1), (16, 4, 2), (256, 8, 4), (512, 16, 3), (60, 5, 2), (96, 4, 1), (21, 7, 3), (1024, 64, 9)]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def settled(x, b, scoring, G, Gk):
    """Rows whose group sums at the cut, and whose keys unless logit and bias are equal, lie further apart
    than float64's own roundings: an exponential, a sum and two additions at the size of the keys."""
    x = x.to(D)
    s = br.sigmoid(x) if scoring == "sigmoid" else torch.softmax(x, 1)
    key = torch.where(x == NEG, x, s + b.to(D))
    best = torch.sort(key.view(len(x), G, -1), dim=2, descending=True).values[:, :, :2]
    score = torch.where(best == NEG, torch.zeros_like(best), best).sum(2)
    size = torch.where(score > -1e8, best.abs().nan_to_num(posinf=0.0).sum(2), 0.0).amax(1)
    score = torch.sort(score, dim=1, descending=True).values
    step = 64 * 2.0 ** -52
    v, at = torch.sort(key, dim=1, descending=True)
    xs, bs = x.gather(1, at), b[at]
    same = (xs[:, 1:] == xs[:, :-1]) & (bs[:, 1:] == bs[:, :-1])
    apart = (v[:, :-1] - v[:, 1:] > step * (1 + v[:, 1:].abs())) | same | (v[:, 1:] < -1e8)
    return apart.all(1) & (score[:, Gk - 1] - score[:, Gk] > step * (1 + size))


def run(x, b, topk, scoring, G, Gk):
    keep = settled(x, b, scoring, G, Gk)
    assert int(keep.sum()) >= len(x) // 2
    x = x[keep]
    kw = dict(scoring=scoring, n_group=G, topk_group=Gk, group_top=2)
    want = br.route(x, topk, bias=b, **kw)
    live = x[torch.isfinite(x)]
    br.check_route(mla.moe_lora_route(x.to(DEV), topk, bias=b.to(DEV), **kw), want,
                   float(live.max() - live.min() + live.abs().max()))


@pytest.mark.parametrize("E,G,Gk", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B", [8.0, 16.0, 64.0, 1e3, 1e4, 1e5])
def test_opposite_biases(E, G, Gk, scoring, B):
    """One expert of every other group has bias B and one -B; of each, two experts are left.  The logits
    are about as close as keys of that size are in fp32."""
    size = E // G
    g = gen(E + G + int(B))
    x = 0.5 + torch.randn((400, E), generator=g) * min(1.0, B * 2.0 ** -20)
    b = torch.zeros(E)
    for j in range(0, G, 2):
        b[j * size] = B
        b[j * size + size - 1] = -B
        x[:, j * size + 1:(j + 1) * size - 1] = NEG
        x[:, (j + 1) * size + 2:(j + 2) * size] = NEG
    run(x, b, min(2 * Gk, 8), scoring, G, Gk)


@pytest.mark.parametrize("E,G,Gk", [(16, 4, 2), (256, 8, 4), (60, 5, 2), (96, 4, 1), (21, 7, 3)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("at", ["first", "last"])
def test_one_such_group_among_others(E, G, Gk, scoring, at):
    """Only one group's sum is uncertain, by more than lies between the others: it may belong on the
    other side of the cut though the two groups next to the cut are certain."""
    size = E // G
    j = 0 if at == "first" else G - 1
    g = gen(E + G)
    x = torch.randn((400, E), generator=g)
    b = 0.1 * torch.randn(E, generator=g)
    b[j * size:(j + 1) * size] = -1e9
    b[j * size], b[j * size + 1] = 4e6, -4e6
    run(x, b, min(2 * Gk, 8), scoring, G, Gk)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_experts_taken_out_by_a_far_bias(scoring):
    """Biases of -1e9 in every group, and all over one group."""
    E, G = 64, 8
    g = gen(5)
    x = torch.randn((400, E), generator=g)
    b = 0.1 * torch.randn(E, generator=g)
    b[::3] = -1e9
    b[24:32] = -1e9
    run(x, b, 8, scoring, G, 4)


def test_named_example():
    """Sums of 1.00002 and 1.00001, in fp32 1.0 and 1.00001."""
    x = torch.tensor([[8e-5, 0.0, 2e-5, 2e-5]])
    b = torch.tensor([1000.0, -1000.0, 0.0, 0.0])
    ids, _ = mla.moe_lora_route(x.to(DEV), 2, scoring="sigmoid", bias=b.to(DEV), n_group=2, group_top=2)
    assert ids.cpu().tolist() == [[0, 1]]
