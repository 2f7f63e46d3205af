"""Refusals of the bf16 base side's entry points, on the host: every bad argument is answered before
any HIP call, through the C ABI and through the binding (no GPU needed)."""
import ctypes

import pytest
import torch

import moe_lora_adapter_amd as mla

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)
OFF2 = ctypes.c_void_p(4098)
OFF8 = ctypes.c_void_p(4104)
INV, UNS = mla.ERR_INVALID, mla.ERR_UNSUPPORTED
BF = torch.bfloat16


def route(**kw):
    a = dict(logits=P, bf16=0, bias=None, M=4, E=64, topk=4, scoring=0, n_group=1, topk_group=1,
             group_top=1, renorm=1, scale=1.0, ids=P, weights=P)
    a.update(kw)
    return mla.lib().moe_lora_route(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INV), (dict(ids=None), INV), (dict(weights=None), INV), (dict(M=-1), INV),
    (dict(E=0), INV), (dict(topk=0), INV), (dict(topk=65), INV), (dict(bf16=2), INV),
    (dict(scoring=2), INV), (dict(scoring=-1), INV), (dict(renorm=2), INV),
    (dict(n_group=0), INV), (dict(n_group=3), INV), (dict(topk_group=2), INV),
    (dict(topk_group=0), INV), (dict(n_group=8, topk_group=9), INV), (dict(group_top=3), INV),
    (dict(group_top=2), INV), (dict(n_group=64, group_top=2), INV), (dict(group_top=0), INV),
    (dict(n_group=32, topk_group=1), INV), (dict(scale=float("inf")), INV),
    (dict(scale=float("nan")), INV), (dict(logits=OFF2), INV), (dict(logits=ODD, bf16=1), INV),
    (dict(bias=OFF2), INV), (dict(ids=OFF2), INV), (dict(weights=OFF2), INV),
    (dict(E=1025), UNS), (dict(E=128, topk=65), UNS), (dict(E=130, n_group=65, topk_group=65), UNS),
    (dict(M=1 << 29), UNS), (dict(M=0, logits=None, ids=None, weights=None), mla.OK),
])
def test_route(kw, status):
    assert route(**kw) == status


def gemm(**kw):
    a = dict(x=P, w=P, bias=None, delta=None, residual=None, M=4, K=64, Ns=64, S=1, act=0, y32=0, y=P)
    a.update(kw)
    return mla.lib().moe_lora_gemm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(M=-1), INV),
    (dict(K=0), INV), (dict(K=60), INV), (dict(K=-8), INV), (dict(Ns=0), INV), (dict(Ns=12), INV),
    (dict(S=0), INV), (dict(act=5), INV), (dict(act=-1), INV), (dict(act=3), INV),
    (dict(act=4, S=3), INV), (dict(y32=2), INV), (dict(x=OFF8), INV), (dict(w=OFF8), INV),
    (dict(bias=OFF8), INV), (dict(delta=OFF8), INV), (dict(residual=OFF8), INV), (dict(y=OFF8), INV),
    (dict(K=(1 << 21) + 8), UNS), (dict(Ns=1 << 20, K=1 << 10), UNS),
    (dict(Ns=1 << 20, S=1 << 11, K=8), UNS), (dict(M=1 << 31), UNS), (dict(M=1 << 30, Ns=512), UNS),
    (dict(M=0, x=None, y=None), mla.OK),
])
def test_gemm(kw, status):
    assert gemm(**kw) == status


def moe(**kw):
    a = dict(x=P, per_pair=0, w=P, bias=None, delta=None, sorted=P, eids=P, ntpp=P, tw=P, mul=1, M=4,
             topk=2, K=64, Ns=64, S=1, E=4, B=16, act=0, y=P)
    a.update(kw)
    return mla.lib().moe_lora_moe_gemm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(sorted=None), INV), (dict(eids=None), INV),
    (dict(ntpp=None), INV), (dict(tw=None), INV), (dict(y=None), INV), (dict(per_pair=2), INV),
    (dict(mul=-1), INV), (dict(M=-1), INV), (dict(topk=0), INV), (dict(E=0), INV), (dict(K=20), INV),
    (dict(Ns=4), INV), (dict(S=0), INV), (dict(act=7), INV), (dict(act=3), INV),
    (dict(x=OFF8), INV), (dict(w=OFF8), INV), (dict(bias=OFF8), INV), (dict(delta=OFF8), INV),
    (dict(y=OFF8), INV), (dict(E=1025), UNS), (dict(B=8), UNS), (dict(B=256), UNS),
    (dict(M=1 << 20, K=1 << 10), UNS), (dict(Ns=1 << 20, K=1 << 10), UNS),
    (dict(M=1024, topk=1, E=1024, B=128, Ns=8, S=1 << 19, K=8), UNS),
    (dict(M=0, x=None, y=None, sorted=None), mla.OK),
])
def test_moe_gemm(kw, status):
    assert moe(**kw) == status


def combine(**kw):
    a = dict(y=P, tw=None, ids=None, E=0, residual=None, M=4, topk=2, N=64, out=P)
    a.update(kw)
    return mla.lib().moe_lora_combine(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), INV), (dict(out=None), INV), (dict(M=-1), INV), (dict(topk=0), INV),
    (dict(N=0), INV), (dict(N=12), INV), (dict(ids=P), INV), (dict(ids=OFF2, E=4), INV),
    (dict(tw=OFF2), INV), (dict(y=OFF8), INV), (dict(residual=OFF8), INV), (dict(out=OFF8), INV),
    (dict(M=1 << 30), UNS), (dict(M=1 << 20, N=1 << 14), UNS), (dict(M=0, y=None, out=None), mla.OK),
])
def test_combine(kw, status):
    assert combine(**kw) == status


def bf(*s):
    return torch.zeros(s, dtype=BF)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


f32 = torch.zeros


def test_route_binding_refuses_before_calling():
    go = mla.moe_lora_route
    with pytest.raises(TypeError):
        go(torch.zeros((2, 8), dtype=torch.float64), 2)
    with pytest.raises(TypeError):
        go([[1.0, 2.0]], 1)
    for bad in (f32(8), f32(2, 16)[:, ::2], bf(2, 16)[:, ::2]):
        with pytest.raises(ValueError):
            go(bad, 2)
    with pytest.raises(ValueError):
        go(f32(2, 8), 2, scoring="tanh")
    with pytest.raises(ValueError):
        go(f32(2, 8), 2, bias=f32(7))
    with pytest.raises(TypeError):
        go(f32(2, 8), 2, bias=bf(8))
    with pytest.raises(TypeError):
        go(f32(2, 8), 2, topk_ids=torch.zeros((2, 2), dtype=torch.int64))
    with pytest.raises(ValueError):
        go(f32(2, 8), 2, topk_weights=f32(2, 3))
    with pytest.raises(mla.MoeLoraError):
        go(f32(2, 8), -1)


def test_gemm_binding_refuses_before_calling():
    go = mla.moe_lora_gemm
    x, w = bf(3, 64), bf(2, 16, 64)
    with pytest.raises(TypeError):
        go(x, f32(2, 16, 64))
    with pytest.raises(TypeError):
        go(f32(3, 64), w)
    for bad in (bf(3, 72), bf(6, 64)[::2], bf(3, 64, 1)):
        with pytest.raises(ValueError):
            go(bad, w)
    with pytest.raises(ValueError):
        go(x, bf(16, 64))
    with pytest.raises(ValueError, match="activation"):
        go(x, w, activation="relu")
    for kw in (dict(bias=bf(16)), dict(delta=bf(3, 16)), dict(residual=bf(3, 16)),
               dict(activation="silu_mul", residual=bf(3, 32)), dict(y=bf(3, 16)),
               dict(activation="silu_mul", y=bf(3, 32))):
        with pytest.raises(ValueError):
            go(x, w, **kw)
    for kw in (dict(bias=f32(32)), dict(y=torch.zeros((3, 32), dtype=torch.float16)),
               dict(y=bf(3, 32), out_dtype=torch.float32), dict(out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            go(x, w, **kw)


def _align(M, topk, E, B):
    cap = mla.align_capacity(M, topk, E, B)
    return mla.AlignOutput(i32(1, cap), i32(1, cap // B), i32(1), None, None, B, cap)


def test_moe_gemm_binding_refuses_before_calling():
    al = _align(3, 2, 4, 16)

    def go(x=bf(3, 64), w=bf(4, 2, 16, 64), al=al, tw=None, y=bf(3, 2, 32), mul=False, **kw):
        return mla.moe_lora_moe_gemm(x, w, al, tw, y, mul_routed_weight=mul, **kw)
    for kw in (dict(y=bf(3, 2, 16)), dict(x=bf(6, 64)), dict(x_per_pair=True), dict(w=bf(2, 16, 64)),
               dict(bias=bf(32)), dict(bias=bf(4, 16)), dict(delta=bf(6, 32)), dict(tw=f32(3, 3)),
               dict(activation="silu_mul"), dict(activation="gelu"), dict(al=_align(4, 2, 4, 16)),
               dict(y=bf(3, 2, 64)[:, :, ::2])):
        with pytest.raises(ValueError):
            go(**kw)
    for kw in (dict(y=f32(3, 2, 32)), dict(tw=bf(3, 2)), dict(x=f32(3, 64))):
        with pytest.raises(TypeError):
            go(**kw)


def test_combine_binding_refuses_before_calling():
    go = mla.moe_lora_combine
    y = bf(3, 2, 16)
    for kw in (dict(out=bf(3, 8)), dict(residual=bf(2, 16)), dict(topk_weights=f32(3, 1)),
               dict(topk_ids=i32(3, 2)), dict(topk_ids=i32(3, 1), E=4)):
        with pytest.raises(ValueError):
            go(y, **kw)
    with pytest.raises(ValueError):
        go(bf(3, 16))
    with pytest.raises(TypeError):
        go(f32(3, 2, 16))
    with pytest.raises(TypeError):
        go(y, topk_weights=bf(3, 2))


def test_nothing_runs_on_host_memory():
    al = _align(3, 2, 4, 16)
    for call in (lambda: mla.moe_lora_route(f32(2, 8), 2),
                 lambda: mla.moe_lora_gemm(bf(3, 64), bf(2, 16, 64)),
                 lambda: mla.moe_lora_moe_gemm(bf(3, 64), bf(4, 2, 16, 64), al, None, bf(3, 2, 32),
                                               mul_routed_weight=False),
                 lambda: mla.moe_lora_combine(bf(3, 2, 16))):
        with pytest.raises(ValueError, match="GPU"):
            call()
