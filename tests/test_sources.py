"""What the compiler does not check in the CUDA sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "cascade_paged_attention_gb300", "csrc")
VECTOR_BYTES = {"float2": 8, "uint2": 8, "int2": 8, "float4": 16, "uint4": 16, "int4": 16}
ELEMENT_BYTES = {"long long": 8, "uint64_t": 8, "int64_t": 8, "double": 8}


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_shared_arrays_read_as_vectors_are_aligned(name):
    """A shared array has the alignment of its elements unless it is given more; one that is
    read or written as vectors needs theirs."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__shared__\s+(?:__align__\((\d+)\)\s+)?((?:long long|[\w:]+))\s+([^;=()]+);",
                         text):
        given = int(m.group(1) or 0) or ELEMENT_BYTES.get(m.group(2), 4)
        for var in re.findall(r"(\w+)\s*(?:\[[^\]]*\])+", m.group(3)):
            for c in re.finditer(r"reinterpret_cast<(?:const\s+)?(\w+)\s*\*>\(\s*&?" + var + r"\b", text):
                need = VECTOR_BYTES.get(c.group(1), 1)
                assert given >= need, f"{var}: {given}-byte aligned, read as {c.group(1)}"


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_a_block_that_gave_up_waits_for_its_copies_and_products(name):
    """The waits of a kernel return at once when its block has given up one of them; what is in flight
    then is waited for by mbar_drain()."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", lambda m: m.group(0) if "in flight when" in m.group(0) else "", f.read())
    for m in re.finditer(r"\bwait_warp\(&ctrl->mma_done|\bmbar_wait\(&ctrl->(?:mma_done|merge_full)", text):
        assert "mbar_drain(&ctrl->" in text[m.end():m.end() + 350], text[m.start():m.end()]
    for m in re.finditer(r"in flight when", text):
        block = text[m.end():m.end() + 700]
        assert "wait" in block and "mbar_drain(&" in block
    loads = len(re.findall(r"\b(?:tma_load_[23]d|bulk_load)\(smem", text))
    assert loads == 0 or "mbar_drain(&" in text
