"""The names of the bf16 products' kernels, and that the sizes the GPU tests run reach every one of them
(no GPU needed: without one the sizes are judged for 256 compute units)."""
import random

import pytest

import moe_lora_adapter_amd as mla
import product_tiles as pt


def acts(gated):
    return pt.GATED if gated else pt.UNGATED


@pytest.mark.parametrize("kernel,gated,size", **pt.flat(pt.DENSE))
def test_dense_size_reaches_its_kernel(kernel, gated, size):
    assert {mla.gemm_kernel_name(*size, act) for act in acts(gated)} == {kernel}


@pytest.mark.parametrize("kernel,gated,size", **pt.flat(pt.GROUPED))
def test_grouped_size_reaches_its_kernel(kernel, gated, size):
    M, topk, E, K, Ns, S, B = size
    assert {mla.moe_gemm_kernel_name(M, topk, K, Ns, S, E, B, pairs, act)
            for act in acts(gated) for pairs in (False, True)} == {kernel}


def test_no_other_kernel_over_random_sizes():
    """Whatever the dispatch takes has sizes in the tables."""
    rng = random.Random(1)

    def some(lo, hi, step=1):
        return max(step, int(lo * (hi / lo) ** rng.random()) // step * step)
    for _ in range(20000):
        gated = rng.random() < 0.5
        act, S = rng.choice(acts(gated)), 2 if gated else rng.choice([1, 2, 3])
        M, K, Ns = some(1, 70000), some(8, 9000, 8), some(8, 9000, 8)
        assert (mla.gemm_kernel_name(M, K, Ns, S, act), gated) in pt.DENSE
        topk, E, B = rng.choice([1, 2, 4, 8]), some(1, 256), rng.choice([16, 32, 64, 128])
        name = mla.moe_gemm_kernel_name(M, topk, K, Ns, S, E, B, False, act)
        assert (name, gated) in pt.GROUPED


def test_names_of_refused_sizes():
    lib = mla.lib()
    assert lib.moe_lora_gemm_kernel_name(4, 64, 64, 1, 0) == b"gemm_rows_kernel 16x16"
    for M, K, Ns, S, act in ((0, 64, 64, 1, 0), (-1, 64, 64, 1, 0), (4, 60, 64, 1, 0), (4, 64, 64, 1, 3),
                             (4, 64, 64, 1, 5), (1 << 31, 64, 64, 1, 0), (4, (1 << 21) + 8, 64, 1, 0)):
        assert lib.moe_lora_gemm_kernel_name(M, K, Ns, S, act) is None
    good = dict(M=4, topk=2, K=64, Ns=64, S=1, E=4, B=16, pairs=0, act=0)
    assert lib.moe_lora_moe_gemm_kernel_name(*good.values()) == b"gemm_rows_kernel 16x32"
    for bad in (dict(M=0), dict(M=-1), dict(topk=0), dict(K=20), dict(S=0), dict(E=0), dict(E=1025), dict(B=8),
                dict(pairs=2), dict(act=3), dict(M=1 << 20, K=1 << 10)):
        assert lib.moe_lora_moe_gemm_kernel_name(*dict(good, **bad).values()) is None
    for bad in (lambda: mla.gemm_kernel_name(0, 64, 64, 1), lambda: mla.moe_gemm_kernel_name(4, 2, 20, 64, 1, 4, 16)):
        with pytest.raises(mla.MoeLoraError):
            bad()
    with pytest.raises(ValueError, match="activation"):
        mla.gemm_kernel_name(4, 64, 64, 1, "relu")
