"""Buffers that the adapters' calls allocate themselves: outputs and workspaces are taken from the
stream that the call writes them on."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_lora_adapter_amd as mla  # noqa: E402
from moe_lora_adapter_amd import synth  # noqa: E402
import gpu_helpers as gh  # noqa: E402


class Taken:
    """torch.empty, noting the stream that is current at each call."""

    def __init__(self, monkeypatch):
        self.streams, real = [], torch.empty

        def empty(*a, **kw):
            self.streams.append(torch.cuda.current_stream())
            return real(*a, **kw)
        monkeypatch.setattr(torch, "empty", empty)


def test_align_with_outputs_and_workspace_of_its_own(monkeypatch):
    s = synth.shape("align_stress")
    c = synth.draw(s, with_tensors=False)
    ids, mapping = gh.i32_dev(c.topk_ids), gh.i32_dev(c.token_lora_mapping)
    assert mla.align_workspace_size(s.M, s.topk, s.E, s.L, s.block_m) > 0
    want = gh.align_to_host(mla.moe_lora_align(ids, mapping, s.E, s.L, s.block_m))
    torch.cuda.synchronize()
    side, taken = torch.cuda.Stream(), Taken(monkeypatch)
    out = mla.moe_lora_align(ids, mapping, s.E, s.L, s.block_m, stream=side)
    assert taken.streams and all(t == side for t in taken.streams)
    side.synchronize()
    gh.assert_align_equal(gh.align_to_host(out), want, s.block_m)


def test_fused_calls_with_buffers_of_their_own(monkeypatch):
    d = gh.DeviceCase(synth.draw(synth.shape("tiny")))
    s = d.s
    al, args = d.align(), dict(mul_routed_weight=s.mul, add_inputs=s.add, x_per_pair=s.x_per_pair)
    both = dict(args, E=s.E, L=s.L, block_m=s.block_m)
    y, z = d.y_in.clone(), d.y_in.clone()
    mla.fused_moe_lora_two_kernel(d.x, d.a, d.b, al, d.w, y, **args)
    mla.fused_moe_lora_with_align(d.topk_ids, d.mapping, d.x, d.a, d.b, d.w, z, **both)
    y2, z2 = d.y_in.clone(), d.y_in.clone()
    torch.cuda.synchronize()
    side, taken = torch.cuda.Stream(), Taken(monkeypatch)
    mla.fused_moe_lora_two_kernel(d.x, d.a, d.b, al, d.w, y2, stream=side, **args)
    assert len(taken.streams) == 1
    mla.fused_moe_lora_with_align(d.topk_ids, d.mapping, d.x, d.a, d.b, d.w, z2, stream=side, **both)
    assert len(taken.streams) > 1 and all(t == side for t in taken.streams)
    side.synchronize()
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
    assert torch.equal(z.view(torch.int16), z2.view(torch.int16))
