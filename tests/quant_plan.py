"""How calls of the attention over caches held in 4 bits are launched, from the library's own plan
compiled for the host (tests/native/plan_of.cpp)."""
import collections
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FEW16, FEW32, MANY16, MANY32 = range(4)  # how rows are held
SPLITS, PARTS, ALONE = range(3)          # how tokens are cut
Call = collections.namedtuple("Call", "channels head_dim page_tokens max_blocks n_heads n_seqs n_q n_groups max_q "
                                      "max_prefix max_len")
Plan = collections.namedtuple("Plan", "dp pre rest cut pieces")


def plans(calls):
    """The Plan of each Call."""
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "plan_of")
        subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "kv_cache_compression_anchor_amd", "csrc"), "-I",
                        os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "native", "plan_of.cpp"), "-o", exe],
                       check=True)
        out = subprocess.run([exe], input="".join(" ".join(map(str, c)) + "\n" for c in calls), capture_output=True,
                             text=True, check=True).stdout
    return [Plan(*map(int, line.split())) for line in out.splitlines()]
