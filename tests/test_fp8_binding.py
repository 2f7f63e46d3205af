"""The 8-bit calls' way to the current stream, and the largest products (no GPU needed)."""
import ctypes
from types import SimpleNamespace

import moe_lora_adapter_amd as mla


def _torch(device, **names):
    return SimpleNamespace(_C=SimpleNamespace(_cuda_getDevice=lambda: device, **names))


def test_direct_takes_the_current_stream_of_the_current_device():
    raw = dict(_cuda_getCurrentRawStream=lambda d: 1000 + d)
    assert mla._direct(_torch(1, **raw), 1, None) == 1001
    assert mla._direct(_torch(0, **raw), 1, None) is None  # another device is current
    assert mla._direct(_torch(1, **raw), 1, object()) is None  # a stream was given
    assert mla._direct(_torch(1, **raw), -1, None) is None  # host memory


def test_direct_does_without_the_names_that_are_not_public():
    assert mla._direct(_torch(0), 0, None) is None
    assert mla._direct(SimpleNamespace(_C=SimpleNamespace()), 0, None) is None


def test_products_of_too_many_tiles_are_refused():
    """2^31 tiles of 16 x 16 and more, dense and over every block's rows; no call reaches a device."""
    P = ctypes.c_void_p(4096)
    dense = lambda M, S: mla.lib().moe_lora_fp8_gemm(P, P, P, P, M, 16, 8, S, P, None)  # noqa: E731
    assert dense(16 << 13, 1 << 18) == mla.ERR_UNSUPPORTED
    assert dense(1 << 28, 1 << 7) == mla.ERR_UNSUPPORTED
    # 1024 experts, a pair each in blocks of 128: 8192 tiles of rows
    grouped = lambda S: mla.lib().moe_lora_fp8_moe_gemm(  # noqa: E731
        P, P, 0, P, P, P, P, P, P, 1, 1024, 1, 16, 8, S, 1024, 128, P, None)
    assert grouped(1 << 18) == mla.ERR_UNSUPPORTED
    assert grouped(1 << 20) == mla.ERR_UNSUPPORTED
