"""What the sources have to keep to where a run cannot show it (no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "whisper_audio_encoder_gb300", "csrc")
# kernels that may start while the kernel before them still writes, and what of their inputs nothing writes on the device
# while they run: weights and biases
EARLY = {"prefix_attention.cu": (), "prefix_attention.cuh": (), "prefix_attention_tc.cu": (), "cache_evict.cu": (),
         "decode_attention.cu": (), "layernorm.cu": ("g4 ", "b4 ", "g2 ", "b2 "),
         # (k_dec_embed, which reads tok, pos and the tables e and pp, starts after what is before it)
         "decode_step.cu": ("reinterpret_cast<const float4 *>(p.ln_g", "reinterpret_cast<const float4 *>(p.ln_b", "bp ", "tok ", "e ",
                            "pp ")}


@pytest.mark.parametrize("name", EARLY)
def test_early_kernels_read_what_others_write_by_ordinary_loads(name):
    """__ldg is ld.global.nc, which PTX allows only for data that stays as it is for the kernel's whole life."""
    with open(os.path.join(CSRC, name)) as f:
        source = re.sub(r"//[^\n]*", "", f.read())
    found = re.findall(r"__ldg\(([^;]*);", source)
    assert [x for x in found if not x.startswith(EARLY[name])] == []


def test_layernorm_s_rows_may_be_written_meanwhile():
    """(a const __restrict__ parameter is read by ld.global.nc without being asked to)"""
    with open(os.path.join(CSRC, "layernorm.cu")) as f:
        assert not re.search(r"const float \*__restrict__ x\b", f.read())
