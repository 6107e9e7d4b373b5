"""How calls of the attention over caches held in 4 bits are launched, on the CPU under
AddressSanitizer and UndefinedBehaviorSanitizer (tests/native/plan_check.cpp)."""
import os

from tests.quant_plan import ALONE, MANY16, Call, plans
from tests.test_sanitize import CSRC, ROOT, SAN, pytestmark, run  # noqa: F401


def build_and_run(tmp_path, name):
    exe = str(tmp_path / name)
    r = run(["g++", "-std=c++17", *SAN, "-Wall", "-Wextra", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
             os.path.join(ROOT, "tests", "native", name + ".cpp"), "-o", exe])
    assert r.returncode == 0, r.stderr
    r = run([exe])
    assert "runtime error" not in r.stderr and "Sanitizer" not in r.stderr, r.stderr[-4000:]
    return r


def test_every_call_has_its_kernel(tmp_path):
    r = build_and_run(tmp_path, "plan_check")
    assert r.returncode == 0 and "plans ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]


def test_long_contexts_are_cut_unless_their_workgroups_fill_the_chip():
    """More than 32 rows of a kv head, 8 kv heads of 128 channels, no shared prefix."""
    def call(seqs, n_q, most, longest, G=4):
        return Call(1024, 128, 16, 8192, 8 * G, seqs, n_q, 0, most, 0, longest)

    cut = [call(2, 1024, 512, 9216), call(3, 1536, 512, 9216), call(16, 1024, 64, 81920), call(2, 513, 512, 81920),
           call(32, 160, 5, 9216, G=8), call(1, 512, 512, 9216)]
    alone = [call(4, 2048, 512, 9216), call(32, 2048, 64, 81920), call(2, 1024, 512, 512), call(16, 1024, 64, 1024),
             call(8, 1024, 128, 2048), call(1, 512, 512, 128), call(64, 320, 5, 9216, G=8)]
    for c, p in zip(cut, plans(cut)):
        assert p.rest >= MANY16 and p.cut != ALONE and p.pieces > 1, (c, p)
    for c, p in zip(alone, plans(alone)):
        assert p.rest >= MANY16 and p.cut == ALONE, (c, p)


def test_parts_hold_every_tile_once(tmp_path):
    r = build_and_run(tmp_path, "parts_check")
    assert r.returncode == 0 and "parts ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
