"""What the sources have to keep to where a run cannot show it (no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "whisper_audio_encoder_gb300", "csrc")
# kernels that may start while the kernel before them still writes, and what of their inputs nothing writes on the device
# while they run: weights and biases
EARLY = {"prefix_attention.cu": (), "prefix_attention.cuh": (), "prefix_attention_tc.cu": (), "cache_evict.cu": ()}


@pytest.mark.parametrize("name", EARLY)
def test_early_kernels_read_what_others_write_by_ordinary_loads(name):
    """__ldg is ld.global.nc, which PTX allows only for data that stays as it is for the kernel's whole life."""
    with open(os.path.join(CSRC, name)) as f:
        source = re.sub(r"//[^\n]*", "", f.read())
    found = re.findall(r"__ldg\(([^;]*);", source)
    assert [x for x in found if not x.startswith(EARLY[name])] == []
