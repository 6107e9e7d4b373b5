"""What test_kernel_waits.py holds of the attention's assembly, of the attention over caches held in 4 bits
and of what the two share: nothing is computed in a statement, as the compiler keeps the distance
of its own vector instructions to a matrix product's result and not that of a statement's."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_compression_anchor_amd", "csrc")


def words(text):
    """The instructions in a source's statements of assembly, and how many statements there are."""
    statements = re.findall(r"\b(?:asm|__asm|__asm__)\b(?:\s+(?:volatile|__volatile__))?\s*\(\s*((?:\"[^\"]*\"\s*)*)", text)
    lines = [line for s in statements for line in re.split(r"\\n|\\t|;", "".join(re.findall(r'"([^"]*)"', s)))]
    return [line.split()[0] for line in lines if line.strip()], len(statements)


@pytest.mark.parametrize("name,least", [("cg_quant_attention.hip", 10), ("cg_attention.h", 2), ("cg_quant.hip", 0)])
def test_nothing_is_computed_in_assembly(name, least):
    with open(os.path.join(CSRC, name)) as f:
        found, statements = words(f.read())
    assert statements >= least
    assert set(found) <= {"s_mov_b32", "s_nop", "global_load_lds_dwordx4", "s_waitcnt"}, found
    assert ("global_load_lds_dwordx4" in found) == (name == "cg_quant_attention.hip")


def test_a_vector_instruction_would_be_seen():
    found, n = words('asm volatile("s_nop 0\\n\\tv_max3_f32 %0, %1, %2, %3" : "=v"(x) : "v"(a), "v"(b), "v"(c));'
                     'asm("v_exp_f32 %0, %1" : "=v"(y) : "v"(z)); asm volatile("" : "+v"(x));')
    assert n == 3 and found == ["s_nop", "v_max3_f32", "v_exp_f32"]
