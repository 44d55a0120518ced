"""The check that stands before a column's partials are joined, on pairs of shares that no call has stored: the function
itself, compiled for the host (no GPU)."""

import os
import subprocess

import pytest

from sliding_window_attention_kvc_gb300 import build

CTAS = 152
LEAST, MOST = -2 ** 31, 2 ** 31 - 1
FLOATS = [0x3f800000, 0x7fc00000, 0x42c80000, 0xbf800000 - 2 ** 32, 0xff800000 - 2 ** 32]     # a partial's bits
EDGES = [LEAST, -CTAS, -1, 0, 1, 75, CTAS - 1, CTAS, CTAS + 1, MOST] + FLOATS


@pytest.fixture(scope="module")
def held(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("shares")
    src, exe = tmp / "shares.cu", tmp / "shares"
    src.write_text('#include <cstdio>\n#include "kvc_tree.h"\n'
                   "int main() { int a, b, n; while (std::scanf(\"%d %d %d\", &a, &b, &n) == 3)\n"
                   "    std::printf(\"%d\\n\", kvc::tree_shares_held(a, b, n) ? 1 : 0); }\n")
    subprocess.run([build._nvcc(), "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, str(src), "-o", str(exe)], check=True)

    def run(pairs):
        text = "".join(f"{a} {b} {CTAS}\n" for a, b in pairs)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [x == "1" for x in out]

    return run


def test_only_pairs_of_one_call_are_joined(held):
    """Whatever is let through names partial slots that there are: at most CTAS of them, from 0 to CTAS - 1."""
    pairs = [(a, b) for a in EDGES for b in EDGES]
    pairs += [(a, b) for a in range(-2, CTAS + 2) for b in range(a - 2, a + 4)]
    for (a, b), ok in zip(pairs, held(pairs), strict=True):
        assert ok == (0 <= a <= b <= CTAS - 1), (a, b)


def test_it_stands_before_the_partials():
    """The combine asks before the first use of a stored share."""
    with open(os.path.join(build.CSRC, "kvc_tree.cu")) as f:
        body = f.read().split("tree_combine_kernel(", 1)[1]
    asked = body.index("if (!tree_shares_held(sh.x, sh.y, p.ctas))")
    assert body.index("p.col_shares") < asked < min(body.index(x) for x in ("const int np", "sh.x + col", "p.part_ml", "p.part_o"))
