"""The attention's arithmetic on numbers from device memory, on the CPU under
AddressSanitizer and UndefinedBehaviorSanitizer (tests/native/ranges_check.cpp)."""
import os

from tests.test_sanitize import CSRC, ROOT, SAN, pytestmark, run  # noqa: F401


def test_ranges_hold_at_the_ends_of_the_type(tmp_path):
    exe = str(tmp_path / "ranges_check")
    r = run(["g++", "-std=c++17", *SAN, "-Wall", "-Wextra", "-I", CSRC,
             os.path.join(ROOT, "tests", "native", "ranges_check.cpp"), "-o", exe])
    assert r.returncode == 0, r.stderr
    r = run([exe])
    assert r.returncode == 0 and "ranges ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "Sanitizer" not in r.stderr, r.stderr[-4000:]
