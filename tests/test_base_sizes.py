"""Sizes of 2^31 and more are refused by the bf16 base side's binding and not cut to the 32 bits that the
entry points take (no GPU needed: the tensors have sizes and no memory)."""
import pytest
import torch

import moe_lora_adapter_amd as mla

BF = torch.bfloat16
BIG = 2 ** 32 + 64   # 64 in 32 bits


def meta(*s, dtype=BF):
    return torch.empty(s, dtype=dtype, device="meta")


def align():
    cap = mla.align_capacity(3, 2, 4, 16)
    i32 = torch.int32
    return mla.AlignOutput(meta(1, cap, dtype=i32), meta(1, cap // 16, dtype=i32), meta(1, dtype=i32), None, None, 16, cap)


def moe(K=64, Ns=16, E=4, S=2, topk=2):
    return mla.moe_lora_moe_gemm(meta(3, K), meta(E, S, Ns, K), align(), None, meta(3, topk, S * Ns),
                                 mul_routed_weight=False)


CALLS = {
    "route E": lambda: mla.moe_lora_route(meta(2, BIG), 2),
    "route topk": lambda: mla.moe_lora_route(meta(2, 64), BIG),
    "route n_group": lambda: mla.moe_lora_route(meta(2, 64), 2, n_group=2 ** 32 + 4),
    "route topk_group": lambda: mla.moe_lora_route(meta(2, 64), 2, n_group=4, topk_group=2 ** 32 + 2),
    "route group_top": lambda: mla.moe_lora_route(meta(2, 64), 2, n_group=4, group_top=2 ** 32 + 2),
    "gemm K": lambda: mla.moe_lora_gemm(meta(3, BIG), meta(1, 16, BIG)),
    "gemm Ns": lambda: mla.moe_lora_gemm(meta(3, 64), meta(1, BIG, 64)),
    "gemm S": lambda: mla.moe_lora_gemm(meta(3, 64), meta(BIG, 16, 64)),
    "moe K": lambda: moe(K=BIG), "moe Ns": lambda: moe(Ns=BIG), "moe E": lambda: moe(E=BIG),
    "moe S": lambda: moe(S=BIG), "moe topk": lambda: moe(topk=BIG),
    "combine N": lambda: mla.moe_lora_combine(meta(3, 2, BIG)),
    "combine topk": lambda: mla.moe_lora_combine(meta(3, BIG, 64)),
    "combine E": lambda: mla.moe_lora_combine(meta(3, 2, 64), topk_ids=meta(3, 2, dtype=torch.int32), E=BIG),
    "combine N 2^31": lambda: mla.moe_lora_combine(meta(3, 2, 2 ** 31)),
}


@pytest.mark.parametrize("name", CALLS)
def test_refused(name):
    with pytest.raises(mla.MoeLoraError) as e:
        CALLS[name]()
    assert e.value.status == mla.ERR_UNSUPPORTED
