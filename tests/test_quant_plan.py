"""How calls of the attention over caches held in 4 bits are launched, on the CPU under
AddressSanitizer and UndefinedBehaviorSanitizer (tests/native/plan_check.cpp)."""
import os

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
