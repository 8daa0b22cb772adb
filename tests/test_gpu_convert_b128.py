"""The offline checkpoint converter with the 128-block FP8 format: safetensors
in, E4M3 bytes and fp32 scales per 128 x 128 block out, the same as the plain
quantizer's, other tensors unchanged; and the layer on the converted weight
equal to the layer on the weight itself."""

import numpy as np
import pytest
import torch

from mxfp8_block_scaled_amd import api, convert, synth
from tests import b128_ref as ref


def test_unknown_format_is_refused(tmp_path):
    with pytest.raises(ValueError, match="fmt"):
        convert.convert(str(tmp_path / "in"), str(tmp_path / "out"), fmt="fp8")


@pytest.mark.gpu
def test_convert_b128(tmp_path):
    from safetensors import safe_open
    from safetensors.torch import load_file, save_file
    g = torch.Generator().manual_seed(43)
    tensors = {
        "a.weight": synth.randn_bf16((200, 272), 0.02, g),
        "a.bias": synth.randn_bf16((200,), 0.1, g),
        "b.weight": synth.scale_stress(synth.randn_bf16((64, 512), 0.02, g), seed=3),
        "c.weight": synth.randn_bf16((8, 40), 1.0, g),           # K % 16 == 8: copied
        "d.weight": torch.zeros(3, 16, dtype=torch.bfloat16),
        "e.weight": torch.randn(16, 16, generator=g),            # fp32: copied
    }
    src, dst = str(tmp_path / "in.safetensors"), str(tmp_path / "out.safetensors")
    save_file(tensors, src)
    names = convert.convert(src, dst, fmt="fp8-b128", device="cuda:0")
    assert sorted(names) == ["a.weight", "b.weight", "d.weight"]
    out = load_file(dst)
    with safe_open(dst, framework="pt") as f:
        assert f.metadata()["mx_format"] == "fp8-b128"
    for name in names:
        q, s, _ = ref.quantize(tensors[name].double().numpy(), rows=128)
        assert np.array_equal(ref.decode(out[name + ".qdata"]), q), name
        assert out[name + ".scale"].dtype == torch.float32
        assert np.array_equal(out[name + ".scale"].double().numpy(), np.exp2(s.astype(np.float64) - 127)), name
    for name in ("a.bias", "c.weight", "e.weight"):
        assert torch.equal(out[name], tensors[name])
    x = synth.randn_bf16((33, 272), 1.0, g).cuda()
    w = api.prepare_weight_b128(out["a.weight.qdata"].cuda(), out["a.weight.scale"].cuda())
    direct, _ = api.prepare_weight_b128_bf16(tensors["a.weight"].cuda(), transposed=False)
    assert torch.equal(api.linear(x, w), api.linear(x, direct))
