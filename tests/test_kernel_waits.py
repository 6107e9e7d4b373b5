"""Wait states that gfx950 leaves to whoever writes the instructions.  The compiler
keeps them between its own instructions but does not look inside inline assembly, so
they are checked in the library as it was built:
  - one between a scalar write of m0 and a load into LDS, whose address m0 is;
  - five between a vector instruction that writes a scalar register and a memory
    instruction that takes the register as an address or offset."""
import os
import re
import shutil
import subprocess

import pytest

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """The instructions of every kernel and device function, [(mnemonic, operands)] each."""
    import kv_cache_compression_anchor_amd as cg
    if not os.path.exists(cg.LIB_PATH):
        from kv_cache_compression_anchor_amd import build
        build.build()
    where = tmp_path_factory.mktemp("code")
    lib = shutil.copy(cg.LIB_PATH, where / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, cwd=where, stdout=subprocess.DEVNULL)
    functions = {}
    for part in sorted(p for p in os.listdir(where) if "gfx950" in p):
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", "--no-show-raw-insn", str(where / part)], check=True,
                              capture_output=True, text=True).stdout
        body = None
        for line in text.splitlines():
            head = re.match(r"[0-9a-f]+ <(.+)>:", line)
            if head:
                body = functions.setdefault(head.group(1), [])
            elif body is not None and line.startswith("\t"):
                word, _, rest = line.split("//")[0].strip().partition(" ")
                body.append((word, [x.strip() for x in rest.split(",")] if rest else []))
    return functions


def registers(operand):
    """Scalar registers that an operand names."""
    m = re.fullmatch(r"s(\d+)|s\[(\d+):(\d+)\]|(vcc|m0)", operand.split(" ")[0])
    if not m:
        return set()
    if m.group(4):
        return {m.group(4)}
    a, b = (int(m.group(1)),) * 2 if m.group(1) else (int(m.group(2)), int(m.group(3)))
    return {f"s{i}" for i in range(a, b + 1)}


def states(word, operands):
    return int(operands[0], 0) + 1 if word == "s_nop" else 1


MEMORY = re.compile(r"(global|buffer|scratch|flat)_")


def test_there_is_code_to_check(code):
    assert any("k_attention" in name for name in code)
    assert any(word.startswith("global_load_lds") for body in code.values() for word, _ in body)


def test_loads_into_lds_wait_for_their_address(code):
    short = []
    for name, body in code.items():
        for (word, ops), (after, rest) in zip(body, body[1:]):
            into_lds = "_load_lds" in after or (MEMORY.match(after) and any(x.split(" ")[-1] == "lds" for x in rest))
            if into_lds and word.startswith("s_") and ops and ops[0] == "m0":
                short.append(name)
    assert not short, (len(short), sorted(set(short))[:3])


def test_addresses_wait_for_vector_writes(code):
    short = []
    for name, body in code.items():
        since = {}  # register: wait states since a vector instruction wrote it
        for word, ops in body:
            if MEMORY.match(word):
                short += [(name, word, ops) for x in ops for r in registers(x) if since.get(r, 9) < 5]
            if word in ("s_branch", "s_endpgm", "s_setpc_b64"):
                since = {}
                continue
            since = {r: n + states(word, ops) for r, n in since.items() if n < 9}
            if word.startswith("v_"):
                since |= {r: 0 for x in ops[:2 if "_co_" in word else 1] for r in registers(x)}
            elif word.startswith("s_") and ops:
                for r in registers(ops[0]):
                    since.pop(r, None)
    assert not short, (len(short), short[:3])


def test_attention_computes_nothing_in_assembly():
    """A product's result is there some wait states after its instruction, which the
    compiler keeps for its own vector instructions and not for those of a statement."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "kv_cache_compression_anchor_amd", "csrc", "cg_attention.hip")) as f:
        text = f.read()
    statements = re.findall(r"\basm(?:\s+volatile)?\s*\(\s*((?:\"[^\"]*\"\s*)*)", text)
    assert len(statements) >= 4
    words = [line.split()[0] for s in statements for line in "".join(re.findall(r'"([^"]*)"', s)).split("\\n\\t") if line]
    assert "global_load_lds_dwordx4" in words
    assert not [w for w in words if w.startswith("v_")]
