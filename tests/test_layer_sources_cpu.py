"""The layer operators' headers hold nothing that no kernel calls."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "error_compensated_bit_echo_amd", "csrc")


@pytest.mark.parametrize("header", ["echo_elem.h", "echo_slab.h"])
def test_every_helper_has_a_caller(header):
    sources = {}
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            sources[name] = re.sub(r"//[^\n]*", "", f.read())
    defined = re.findall(r"^(?:__device__ __forceinline__|constexpr int)[^;{=]*?(\w+)\s*(?:\(|=)", sources[header], re.M)
    assert len(defined) >= 5
    everything = "\n".join(sources.values())
    once = [n for n in dict.fromkeys(defined) if len(re.findall(rf"\b{n}\b", everything)) <= defined.count(n)]
    assert not once, f"no caller: {once}"
