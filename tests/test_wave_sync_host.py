"""Lanes of a wave that exchange values through LDS order their accesses by wave_sync(), whose
fences keep the compiler from moving one lane's load past another's store; the barrier builtin
alone is modelled as touching no memory."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "state_space_model_ssd_amd", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".hip", ".h")))


@pytest.mark.parametrize("name", SOURCES)
def test_wave_barriers_come_with_fences(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    text = re.sub(r'__builtin_amdgcn_fence\(__ATOMIC_RELEASE, "wavefront"\);\s*'
                  r"__builtin_amdgcn_wave_barrier\(\);\s*"
                  r'__builtin_amdgcn_fence\(__ATOMIC_ACQUIRE, "wavefront"\);', "", text)
    assert "__builtin_amdgcn_wave_barrier" not in text
