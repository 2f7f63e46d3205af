"""Refusals of the 8-bit entry points, on the host: every bad argument is answered before any HIP
call, through the C ABI and through the binding (no GPU needed)."""
import ctypes

import pytest
import torch

import moe_lora_adapter_amd as mla

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4098)
OFF4 = ctypes.c_void_p(4100)
INV, UNS = mla.ERR_INVALID, mla.ERR_UNSUPPORTED
F8, BF = torch.float8_e4m3fn, torch.bfloat16


def norm(**kw):
    a = dict(x=P, residual=None, weight=P, M=4, H=64, eps=1e-6, residual_out=None, y=None, q=P,
             scales=P)
    a.update(kw)
    return mla.lib().moe_lora_rms_norm_fp8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(weight=None), INV), (dict(q=None), INV), (dict(scales=None), INV),
    (dict(M=-1), INV), (dict(H=0), INV), (dict(H=60), INV), (dict(H=-8), INV),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(residual=P), INV), (dict(residual_out=P), INV),
    (dict(x=OFF4), INV), (dict(weight=OFF4), INV), (dict(q=OFF4), INV), (dict(y=OFF4), INV),
    (dict(residual=OFF4, residual_out=P), INV), (dict(scales=ODD), INV),
    (dict(H=mla.RMS_NORM_MAX_WIDTH + 8), UNS), (dict(M=1 << 31), UNS),
    (dict(M=0, x=None, q=None, scales=None), mla.OK),
])
def test_norm(kw, status):
    assert norm(**kw) == status


def silu(**kw):
    a = dict(y=P, P=4, I=64, h=None, q=P, scales=P)
    a.update(kw)
    return mla.lib().moe_lora_silu_mul_fp8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), INV), (dict(q=None), INV), (dict(scales=None), INV), (dict(P=-1), INV),
    (dict(I=0), INV), (dict(I=12), INV), (dict(y=OFF4), INV), (dict(h=OFF4), INV),
    (dict(q=OFF4), INV), (dict(scales=ODD), INV), (dict(I=1 << 30), UNS), (dict(P=1 << 31), UNS),
    (dict(P=0, y=None, q=None, scales=None), mla.OK),
])
def test_silu(kw, status):
    assert silu(**kw) == status


def gemm(**kw):
    a = dict(x=P, xs=P, w=P, ws=P, M=4, K=128, Ns=64, S=1, y=P)
    a.update(kw)
    return mla.lib().moe_lora_fp8_gemm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(xs=None), INV), (dict(w=None), INV), (dict(ws=None), INV),
    (dict(y=None), INV), (dict(M=-1), INV), (dict(K=0), INV), (dict(K=120), INV),
    (dict(Ns=0), INV), (dict(Ns=12), INV), (dict(S=0), INV), (dict(x=OFF4), INV),
    (dict(w=OFF4), INV), (dict(y=OFF4), INV), (dict(xs=ODD), INV), (dict(ws=ODD), INV),
    (dict(Ns=1 << 20, K=1 << 11), UNS), (dict(Ns=1 << 20, S=1 << 11), UNS), (dict(M=1 << 31), UNS),
    (dict(M=1 << 24, K=1 << 14), UNS), (dict(M=0, x=None, y=None), mla.OK),
])
def test_gemm(kw, status):
    assert gemm(**kw) == status


def moe(**kw):
    a = dict(x=P, xs=P, per_pair=0, w=P, ws=P, sorted=P, eids=P, ntpp=P, tw=P, mul=1, M=4, topk=2,
             K=128, Ns=64, S=1, E=4, B=16, y=P)
    a.update(kw)
    return mla.lib().moe_lora_fp8_moe_gemm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(xs=None), INV), (dict(w=None), INV), (dict(ws=None), INV),
    (dict(sorted=None), INV), (dict(eids=None), INV), (dict(ntpp=None), INV), (dict(tw=None), INV),
    (dict(y=None), INV), (dict(per_pair=2), INV), (dict(mul=-1), INV), (dict(M=-1), INV),
    (dict(topk=0), INV), (dict(E=0), INV), (dict(K=24), INV), (dict(Ns=4), INV), (dict(S=0), INV),
    (dict(x=OFF4), INV), (dict(w=OFF4), INV), (dict(y=OFF4), INV), (dict(xs=ODD), INV),
    (dict(E=1025), UNS), (dict(B=8), UNS), (dict(B=256), UNS), (dict(M=1 << 20, K=1 << 12), UNS),
    (dict(Ns=1 << 20, K=1 << 11), UNS), (dict(M=0, x=None, y=None, sorted=None), mla.OK),
])
def test_moe_gemm(kw, status):
    assert moe(**kw) == status


def test_binding_refuses_before_calling():
    bf = lambda *s: torch.zeros(s, dtype=BF)  # noqa: E731
    f8 = lambda *s: torch.zeros(s, dtype=F8)  # noqa: E731
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    with pytest.raises(TypeError):
        mla.moe_lora_rms_norm_fp8(f32(2, 16), bf(16))
    with pytest.raises(ValueError):
        mla.moe_lora_rms_norm_fp8(bf(2, 16), bf(8))
    with pytest.raises(ValueError):
        mla.moe_lora_rms_norm_fp8(bf(2, 32)[:, ::2], bf(16))
    with pytest.raises(ValueError):
        mla.moe_lora_rms_norm_fp8(bf(2, 16), bf(16), residual_out=bf(2, 16))
    with pytest.raises(ValueError):
        mla.moe_lora_rms_norm_fp8(bf(2, 16), bf(16), out=mla.Fp8Rows(f8(2, 16), f32(2, 1)))
    with pytest.raises(TypeError):
        mla.moe_lora_rms_norm_fp8(bf(2, 16), bf(16), out=mla.Fp8Rows(torch.zeros((2, 16)), f32(1, 2)))
    with pytest.raises(ValueError):
        mla.moe_lora_silu_mul_fp8(bf(2, 17))
    with pytest.raises(ValueError):
        mla.moe_lora_silu_mul_fp8(bf(2, 32), h=bf(2, 8))
    x = mla.Fp8Rows(f8(3, 144), f32(2, 3))
    with pytest.raises(ValueError):
        mla.moe_lora_fp8_gemm(x, f8(1, 8, 128), f32(1, 1, 1))
    with pytest.raises(ValueError):
        mla.moe_lora_fp8_gemm(x, f8(1, 136, 144), f32(1, 1, 2))
    with pytest.raises(TypeError):
        mla.moe_lora_fp8_gemm(x, bf(1, 136, 144), f32(1, 2, 2))
    with pytest.raises(ValueError):
        mla.moe_lora_fp8_gemm(x, f8(1, 136, 144), f32(1, 2, 2), bf(3, 128))
    cap = mla.align_capacity(3, 2, 4, 16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    al = mla.AlignOutput(i32(1, cap), i32(1, cap // 16), i32(1), None, None, 16, cap)
    go = lambda x, al, y, w=f8(4, 1, 8, 144), **kw: mla.moe_lora_fp8_moe_gemm(  # noqa: E731
        x, w, f32(4, 1, 1, 2), al, None, y, mul_routed_weight=False, **kw)
    with pytest.raises(ValueError):
        go(x, al, bf(3, 2, 16))
    with pytest.raises(ValueError):
        go(x, al, bf(3, 2, 8), x_per_pair=True)
    with pytest.raises(ValueError):
        go(x, mla.AlignOutput(i32(2, cap), i32(2, cap // 16), i32(2), None, None, 16, cap), bf(3, 2, 8))
    with pytest.raises(ValueError):
        go(x, mla.AlignOutput(i32(1, 16), i32(1, 1), i32(1), None, None, 16, 16), bf(3, 2, 8))
    # what is left is the device: nothing runs on host memory
    for call in (lambda: go(x, al, bf(3, 2, 8)),
                 lambda: mla.moe_lora_fp8_gemm(x, f8(1, 136, 144), f32(1, 2, 2)),
                 lambda: mla.moe_lora_silu_mul_fp8(bf(2, 32)),
                 lambda: mla.moe_lora_rms_norm_fp8(bf(2, 16), bf(16))):
        with pytest.raises(ValueError, match="GPU"):
            call()
