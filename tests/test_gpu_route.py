"""Routing on the GPU against the definition in float64: picks are equal, weights within fp32."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_lora_adapter_amd as mla  # noqa: E402
import base_reference as br  # noqa: E402
from gpu_helpers import DEV  # noqa: E402

BF, NEG = torch.bfloat16, float("-inf")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def both(x, topk, bias=None, spread=None, **kw):
    want = br.route(x, topk, bias=bias, **kw)
    got = mla.moe_lora_route(x.to(DEV), topk, bias=None if bias is None else bias.to(DEV), **kw)
    live = x.float()[torch.isfinite(x.float())]
    if spread is None:
        spread = float(live.max() - live.min()) + float(live.abs().max()) if live.numel() else 0.0
    br.check_route(got, want, spread)
    return got


SIZES = [(1, 1, 1), (3, 2, 2), (16, 32, 4), (5, 63, 8), (7, 64, 6), (9, 65, 3), (33, 127, 8),
         (130, 128, 8), (17, 129, 1), (6, 200, 10), (65, 256, 8), (5, 257, 8), (4, 512, 64),
         (3, 513, 7), (2, 1000, 33), (3, 1024, 64), (2, 64, 64), (2, 24, 24)]


@pytest.mark.parametrize("M,E,topk", SIZES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_sizes(M, E, topk, scoring, bias, dtype):
    g = gen(M + 3 * E + topk)
    x = (2 * torch.randn((M, E), generator=g)).to(dtype)
    b = 0.3 * torch.randn(E, generator=g) if bias else None
    both(x, topk, b, scoring=scoring)
    both(x, topk, b, scoring=scoring, renormalize=False, scale=2.5)


@pytest.mark.parametrize("E,G,Gk,topk", [(32, 4, 2, 4), (256, 8, 4, 8), (60, 5, 3, 7), (24, 8, 1, 3),
                                         (128, 64, 9, 8), (126, 63, 62, 8), (15, 3, 3, 15), (12, 1, 1, 4),
                                         (1024, 16, 5, 32), (160, 8, 3, 6), (96, 3, 1, 8)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_groups(E, G, Gk, topk, top, scoring, bias):
    if top == 2 and G == 1:
        top = 1
    g = gen(E + G + topk)
    x = 2 * torch.randn((37, E), generator=g)
    x[torch.rand((37, E), generator=g) < 0.1] = NEG
    b = 0.3 * torch.randn(E, generator=g) if bias else None
    both(x, topk, b, scoring=scoring, n_group=G, topk_group=Gk, group_top=top, scale=2.5)


@pytest.mark.parametrize("E", [8, 64, 100, 256, 700])
@pytest.mark.parametrize("kw", [dict(), dict(scoring="sigmoid"), dict(bias=True),
                                dict(bias=True, scoring="sigmoid"), dict(group=True),
                                dict(group=True, scoring="sigmoid", bias=True)])
def test_ties_go_to_the_lowest_index(E, kw):
    """Few distinct logits, zeros of both signs among them, and few distinct biases."""
    kw = dict(kw)
    g = gen(E)
    x = torch.randint(-1, 2, (40, E), generator=g).float()
    x[:, 1::3] *= -0.0
    x[0] = 0.0
    x[1] = -0.0
    b = torch.randint(0, 2, (E,), generator=g).float() / 4 if kw.pop("bias", False) else None
    if kw.pop("group", False):
        kw.update(n_group=4, topk_group=2, group_top=2)
    for t in (torch.float32, BF):
        both(x.to(t), 4, b, **kw)


@pytest.mark.parametrize("E", [8, 100, 256])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_masked_rows(E, scoring, bias, renormalize):
    """Rows with nothing, one, and fewer than topk experts left; the type's lowest value is no mask."""
    g = gen(E + 1)
    x = torch.randn((9, E), generator=g)
    x[0] = NEG
    x[1] = NEG
    x[1, E - 1] = 0.5
    x[2, 3:] = NEG
    x[3, :E - 4] = NEG
    x[4] = torch.finfo(torch.float32).min
    x[5, 1:] = torch.finfo(torch.float32).min
    x[6] = -3e4
    b = 0.1 * torch.randn(E, generator=g) if bias else None
    if bias:
        b[E // 2] = NEG
    ids, w = both(x, 6, b, scoring=scoring, renormalize=renormalize, spread=128.0)
    assert torch.all(ids[0] == -1) and torch.all(w[0] == 0)
    assert ids[1].tolist() == [E - 1] + [-1] * 5
    both(x[:4].to(BF), 6, b, scoring=scoring, renormalize=renormalize, n_group=4, topk_group=1 if E > 20 else 3)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_nan_and_infinity(scoring, bias):
    """NaN is never picked and shows in its row's weights alone; +infinity comes first."""
    g = gen(3)
    x = torch.randn((8, 48), generator=g)
    x[1, 5] = float("nan")
    x[3] = float("nan")
    x[4, 7] = float("inf")
    x[5, 7] = x[5, 40] = float("inf")
    b = 0.1 * torch.randn(48, generator=g) if bias else None
    for r in (True, False):
        ids, w = both(x, 4, b, scoring=scoring, renormalize=r)
        assert torch.all(ids[3] == -1) and torch.isnan(w[3]).all() and torch.isnan(w[1]).all()
        assert 5 not in ids[1].tolist()
    if bias:
        b[9] = float("nan")
        both(x, 4, b, scoring=scoring)
        b[9] = float("inf")
        ids, _ = both(x[:3], 4, b, scoring=scoring)
        assert ids[0, 0] == 9
        x[0, 9] = NEG
        ids, _ = both(x[:1], 4, b, scoring=scoring)
        assert 9 not in ids[0].tolist()


def test_scores_decide_as_in_fp64():
    """Scores that round to the same fp32 value and differ in fp64: the larger one wins, not the lower
    index, for picks and for groups; far outweighed scores still order experts of equal bias."""
    x = torch.full((4, 32), 20.0)
    x[0, 11], x[0, 29] = 20.5, 21.0       # sigmoid: 1 - 2e-9, 1 - 1e-9
    x[1] = torch.linspace(18, 22, 32)
    x[2] = torch.linspace(22, 18, 32)
    b = torch.zeros(32)
    ids, _ = both(x, 3, b, scoring="sigmoid")
    assert ids[0].tolist() == [29, 11, 0] and ids[1].tolist() == [31, 30, 29]
    ids, _ = both(x, 3, b, scoring="sigmoid", n_group=4, topk_group=2, group_top=2)
    assert ids[0].tolist() == [29, 11, 8]
    big = torch.full((32,), 1e6)
    ids, _ = both(x[1:3] - 18, 5, big, scoring="sigmoid")
    assert ids[0].tolist() == [31, 30, 29, 28, 27] and ids[1].tolist() == [0, 1, 2, 3, 4]
    both(x - 18, 5, big, scoring="softmax")
    # logits next to each other
    y = 1 + torch.arange(64).float()[torch.randperm(64, generator=gen(1))] * 2.0 ** -23
    for kw in (dict(), dict(bias=torch.zeros(64))):
        both(y[None], 8, **kw)
        both(y[None], 8, scoring="sigmoid", **kw)


@pytest.mark.parametrize("E,G", [(16, 4), (24, 4), (256, 8), (512, 16), (96, 4)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_groups_whose_sums_leave_fp32(E, G, scoring):
    """Biases of the type's lowest and largest values: two of them are beyond fp32, and such a group is
    still one with experts, ahead of the empty ones around it and in its place among the others."""
    n, big = E // G, torch.finfo(torch.float32).max
    kw = dict(scoring=scoring, n_group=G, group_top=2)
    x = torch.randn((8, E), generator=gen(E))
    x[:, :n] = x[:, 4 * n:] = NEG
    b = torch.zeros(E)
    b[n:3 * n] = -big
    both(x, min(3 * n, 64), b, topk_group=3, **kw)
    both(x, 2 * n, b, topk_group=2, **kw)  # groups 3 and 1
    b[2 * n + 1:3 * n] = -big / 2  # two of them are in range: groups 3 and 2
    both(x, 2 * n, b, topk_group=2, **kw)
    b[n:2 * n], b[2 * n:3 * n] = big / 1.5, big  # groups 2 and 1
    both(x, 2 * n, b, topk_group=2, **kw)
    both(x, 2, b, topk_group=1, **kw)


def test_weights_of_far_picks_do_not_underflow():
    """Picks that a bias chose far below the row's largest logit are renormalised among themselves."""
    x = torch.zeros((2, 16))
    x[:, 4:8] = torch.tensor([-200.0, -201.0, -202.0, -203.0])
    b = torch.zeros(16)
    b[4:8] = 10.0
    for scoring in ("softmax", "sigmoid"):
        ids, w = both(x, 4, b, scoring=scoring, spread=4.0)
        assert sorted(ids[0].tolist()) == [4, 5, 6, 7] and abs(float(w[0].sum()) - 1) < 1e-6


def test_outputs_given_stream_and_sizes():
    g = gen(9)
    x = torch.randn((70, 96), generator=g)
    want = br.route(x, 5)
    ids = torch.full((71, 5), 77, dtype=torch.int32, device=DEV)
    w = torch.full((71, 5), 7.0, device=DEV)
    s = torch.cuda.Stream()
    xd = x.to(DEV)
    torch.cuda.synchronize()
    got = mla.moe_lora_route(xd, 5, topk_ids=ids[:70], topk_weights=w[:70], stream=s)
    s.synchronize()
    br.check_route(got, want, 16.0)
    assert torch.all(ids[70] == 77) and torch.all(w[70] == 7)
    e = mla.moe_lora_route(xd[:0], 5)
    assert e[0].shape == (0, 5) and e[1].shape == (0, 5)


def test_many_rows():
    """More rows than any one pass of small tests: every row is routed, the same as by itself."""
    x = torch.randn((30011, 40), generator=gen(10))
    xd = x.to(DEV)
    ids, w = mla.moe_lora_route(xd, 4)
    top = torch.sort(xd, dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), top.indices[:, :4])
    ref = torch.softmax(top.values[:, :4].double(), 1)
    assert torch.all((w.double() - ref).abs() <= 2.0 ** -19 * ref)


def test_captured_with_align():
    """Routing and align in one captured graph, replayed on other logits."""
    g = gen(11)
    E, M, k, B = 32, 48, 4, 16
    xs = [torch.randn((M, E), generator=g) for _ in range(3)]
    xs[1][10:20] = NEG
    x = xs[0].to(DEV)
    zero = torch.zeros(M, dtype=torch.int32, device=DEV)
    ids = torch.empty((M, k), dtype=torch.int32, device=DEV)
    w = torch.empty((M, k), device=DEV)
    out = mla.alloc_align_output(M, k, E, 1, B, DEV)

    def step():
        mla.moe_lora_route(x, k, topk_ids=ids, topk_weights=w)
        mla.moe_lora_align(ids, zero, E, 1, B, out=out)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in xs + xs:
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = br.route(v, k)
        br.check_route((ids, w), want, 16.0)
        n = int(out.num_tokens_post_padded[0])
        held = out.sorted_token_ids[0, :n].cpu()
        pairs = torch.nonzero(want[0].reshape(-1) >= 0).reshape(-1)
        assert torch.equal(torch.sort(held[held < M * k]).values.long(), pairs)
