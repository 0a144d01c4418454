"""The check of a packed batch's offsets (csrc/packed_range.h), built with the host C++ compiler:
the lengths it gives are those of Python's integers, at every corner of 32 bits."""
import itertools
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bf16_forward_attention_gb300",
                    "csrc")
DRIVER = r"""
#include <cstdio>
#include <iostream>
#include "packed_range.h"
int main() {
  int base, end, longest, total;
  while (std::cin >> base >> end >> longest >> total)
    std::printf("%d\n", attn::packed_len(base, end, longest, total));
}
"""
LO, HI = -(1 << 31), (1 << 31) - 1


def _length(base, end, longest, total):
    n = end - base
    return n if 0 <= base <= end <= total and n <= longest else -1


def _wrapping(base, end, longest, total):
    """The lengths' check with 32-bit sums that wrap: what this must not be."""
    wrap = lambda x: (x - LO) % (1 << 32) + LO
    n = wrap(end - base)
    return n if not (base < 0 or n < 0 or n > longest or wrap(base + n) > total) else -1


def test_lengths(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "d.cpp", tmp_path / "d"
    src.write_text(DRIVER)
    # -ftrapv: an overflow would end the program.
    subprocess.run([cxx, "-std=c++17", "-O1", "-ftrapv", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True)
    corners = [LO, LO + 1, -300, -1, 0, 1, 100, 299, 300, 301, HI - 300, HI - 1, HI]
    cases = [(b, e, m, t) for b, e in itertools.product(corners, corners)
             for m, t in ((1, 300), (100, 300), (300, 300), (1, HI), (HI, HI))]
    rng = random.Random(5)
    cases += [(rng.randint(LO, HI), rng.randint(LO, HI), rng.randint(1, HI), rng.randint(1, HI)) for _ in range(2000)]
    r = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True,
                       text=True, check=True)
    got = [int(x) for x in r.stdout.split()]
    assert got == [_length(*c) for c in cases]
    # The case that passes for a sequence of one token where sums wrap.
    assert _wrapping(HI, LO, 100, 300) == 1 and _length(HI, LO, 100, 300) == -1
