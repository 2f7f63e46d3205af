"""The README's bf16 layer, run as it stands there: tokens without an adapter, pairs without an expert,
and buffers that hold NaN beforehand."""
import os
import re

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_lora_adapter_amd as mla  # noqa: E402
import base_reference as br  # noqa: E402
from gpu_helpers import DEV  # noqa: E402
from test_gpu_products import _grouped  # noqa: E402

BF = torch.bfloat16


def block():
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        found = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "moe_lora_route" in b]
    assert len(found) == 1
    return found[0]


@pytest.mark.parametrize("M,live", [(11, 64), (300, 64), (40, 6)])
def test_bf16_layer(M, live):
    """`live`: experts that the balance bias leaves."""
    g = torch.Generator().manual_seed(M + live)
    E, topk, K, I, L, r = 64, 8, 264, 136, 3, 16
    x, gate = br.rows(g, M, K), br.weights(g, 1, E, K)
    gate_bias, b13_bias = torch.randn(E, generator=g).to(BF), torch.randn((E, 2 * I), generator=g).to(BF)
    balance = 0.1 * torch.randn(E, generator=g)
    balance[live:] = float("-inf")
    w13, w2 = br.weights(g, E, 2, I, K), br.weights(g, E, 1, K, I)
    mapping = torch.randint(-1, L, (M,), generator=g).int()
    host = dict(x=x, gate=gate, gate_bias=gate_bias, balance=balance, b13_bias=b13_bias, w13=w13, w2=w2,
                token_lora_mapping=mapping, one_slot=torch.zeros(M, dtype=torch.int32),
                a13=br.weights(g, 2, L, E, r, K), b13=br.weights(g, 2, L, E, I, r), a2=br.weights(g, 1, L, E, r, I),
                b2=br.weights(g, 1, L, E, K, r), residual=torch.randn((M, K), generator=g).to(BF),
                d13=torch.full((M, topk, 2 * I), float("nan"), dtype=BF),
                h=torch.full((M, topk, I), float("nan"), dtype=BF),
                y=torch.full((M, topk, K), float("nan"), dtype=BF))
    env = dict({n: t.to(DEV) for n, t in host.items()}, mla=mla, torch=torch, M=M, E=E, topk=topk, K=K, I=I, L=L)
    exec(block(), env)
    ids, wt = env["ids"].cpu(), env["weights"].cpu()
    br.check_route((ids, wt), br.route(env["logits"].cpu(), topk, "sigmoid", balance, 8, 4, 2, True, 2.5), 64.0)
    assert bool((ids < 0).any()) == (live < topk)
    d, h, y = env["d13"].cpu(), env["h"], env["y"].cpu()
    plain = mapping < 0
    assert plain.any() and not d[plain].any()
    here = (ids >= 0).view(-1)
    ref, err = _grouped(x, w13, ids, b13_bias, d, "silu_mul", None, False, torch.zeros((M, topk, I)))
    br.check(h[here.to(DEV)], ref[here], err[here])
    ref, err = _grouped(h.cpu(), w2, ids, None, None, None, wt, True, torch.zeros((M, topk, K)))
    sure = here & plain.repeat_interleave(topk)
    br.check(y.view(M * topk, K)[sure], ref[sure], err[sure])
    other = here & ~sure
    assert torch.isfinite(y.view(M * topk, K)[other].float()).all()
    assert not torch.equal(y.view(M * topk, K)[other], ref[other].to(BF))
    br.check(env["out"], *br.combine(torch.where(here.view(M, topk, 1), y, torch.zeros_like(y)), None, ids, E,
                                     host["residual"]))
