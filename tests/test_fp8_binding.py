"""The 8-bit calls' way to the current stream (no GPU needed)."""
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
