"""The host's checks of strided rows and of pages (csrc/rows.h), built with the host C++ compiler
and compared with the sets of elements that small tensors really hold."""
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
#include "rows.h"
using namespace attn_host;
int main() {
  char kind;
  long long x[14];
  while (std::cin >> kind) {
    const int n = kind == 'd' ? 6 : kind == 'm' ? 14 : kind == 'p' ? 6 : kind == 'q' ? 2 : 3;
    for (int i = 0; i < n; ++i) std::cin >> x[i];
    const char* base = nullptr;
    auto rows = [&](int i, long long off) {
      return RowSet{base + (1 << 20) + off * 2, x[i], x[i + 1], x[i + 2], x[i + 3], x[i + 4], x[i + 5]};
    };
    if (kind == 'd') std::printf("%d\n", rows_distinct(rows(0, 0)));
    if (kind == 'm') std::printf("%d\n", rows_meet(rows(0, x[12]), rows(6, x[13])));
    if (kind == 'p') {
      const PageSet a{base + (1 << 20) + x[0] * 2, x[2], x[3], x[4]}, b{base + (1 << 20) + x[1] * 2, x[2], x[3], x[5]};
      std::printf("%d\n", pages_meet(a, b));
    }
    if (kind == 'q') std::printf("%d\n", page_of(x[0], page_divisor(x[1])) == x[0] / x[1]);
    if (kind == 'e') {
      const RowSet r{base, x[0], x[1], x[2], (1LL << 31) - 1, (1LL << 31) - 1, 1 << 20};
      std::printf("%d\n", extent_in_range(r));
    }
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("rows")
    src, exe = d / "d.cpp", d / "d"
    src.write_text(DRIVER)
    subprocess.run([cxx, "-std=c++17", "-O1", "-ftrapv", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True)

    def run(kind, cases):
        text = "\n".join(kind + " " + " ".join(map(str, c)) for c in cases)
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True)
        return [bool(int(x)) for x in r.stdout.split()]

    return run


def _row_starts(batch, token, head, B, S, H):
    return [b * batch + s * token + h * head for b in range(B) for s in range(S) for h in range(H)]


def _some(rng):
    """Strides and sizes of a small tensor; most as torch's views have them."""
    B, S, H = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 3)
    head = rng.choice([128, 128, 256, S * 128, S * 256, 64])
    token = rng.choice([H * 128, H * 128 + 256, (H + 5) * 128, 128, 0])
    batch = rng.choice([S * token, S * token + 128, H * S * 128, (S + 1) * token])
    return batch, token, head, B, S, H


def test_rows_of_a_written_tensor_are_distinct(ask):
    rng = random.Random(1)
    cases = [_some(rng) for _ in range(3000)]
    sure = 0
    for c, said in zip(cases, ask("d", cases)):
        starts = sorted(_row_starts(*c))
        distinct = all(b - a >= 128 for a, b in zip(starts, starts[1:]))
        assert distinct or not said, c
        sure += said
    assert sure > 500
    # The forms in use are all known to be distinct.
    dense = [(4 * 3 * 128, 3 * 128, 128, 2, 4, 3), (3 * 4 * 128, 128, 4 * 128, 2, 4, 3), (4 * 1024, 1024, 128, 2, 4, 3)]
    assert all(ask("d", dense))


def test_tensors_that_share_an_element_meet(ask):
    rng = random.Random(2)
    cases = []
    for _ in range(6000):
        a = _some(rng)
        b = (*a[:5], rng.randint(1, 3)) if rng.random() < 0.7 else _some(rng)
        cases.append((*a, *b, 128 * rng.randint(0, 12), 128 * rng.randint(0, 12)))
    apart = 0
    for c, said in zip(cases, ask("m", cases)):
        a = {c[12] + x + i for x in _row_starts(*c[:6]) for i in range(0, 128, 64)}
        b = {c[13] + x + i for x in _row_starts(*c[6:12]) for i in range(0, 128, 64)}
        meet = bool(a & b)
        assert said or not meet, c
        apart += not said
    assert apart > 500
    # Queries, keys and values as columns of one projection's output, batched or not.
    for B in (1, 2):
        q, k = (2048 * 7, 2048, 128, B, 7, 8), (2048 * 7, 2048, 128, B, 7, 4)
        assert ask("m", [(*q, *k, 0, 1024), (*q, *k, 0, 1536), (*q, *k, 512, 1024)]) == [False, False, True]
    assert ask("m", [(1024 * 1, 1024, 128, 3, 1, 4, 1024, 1024, 128, 3, 1, 4, 0, 512)]) == [False]


def test_pages_that_share_an_element_meet(ask):
    rng = random.Random(3)
    cases = []
    for _ in range(3000):
        n, rows = rng.randint(1, 4), rng.randint(1, 3)
        cases.append((128 * rng.randint(0, 20), 128 * rng.randint(0, 20), n, 128 * (rows + rng.randint(0, 6)), rows, rows))
    apart = 0
    for c, said in zip(cases, ask("p", cases)):
        off_a, off_b, n, stride, rows, _ = c
        a = {off_a + i * stride + 128 * r for i in range(n) for r in range(rows)}
        b = {off_b + i * stride + 128 * r for i in range(n) for r in range(rows)}
        assert said or not a & b, c
        apart += not said
    assert apart > 500
    assert ask("p", [(0, 512, 100, 1024, 4, 4), (0, 384, 100, 1024, 4, 4)]) == [False, True]


def test_extents_do_not_wrap(ask):
    big = (1 << 40) - 1
    assert ask("e", [(big, big, big), (1 << 20, 0, 0), (0, 128, 128), (0, 0, big), (1 << 19, 1 << 19, 0)]) == [
        False, False, True, False, False]


def test_pages_of_keys(ask):
    """The multiplication that stands for a division by the page size, at the borders of pages and of
    31 bits."""
    top = (1 << 31) - 1
    rng = random.Random(4)
    sizes = [*range(1, 70), 100, 127, 128, 129, 255, 256, 257, 1000, 65535, 65536, 65537, 1 << 30, (1 << 30) + 1, top]
    sizes += [rng.randint(1, top) for _ in range(300)] + [rng.randint(1, 5000) for _ in range(300)]
    cases = []
    for d in sizes:
        n = top // d
        for q in {0, 1, 2, n // 2, n - 1, n, rng.randint(0, n)}:
            cases += [(k, d) for k in (q * d - 1, q * d, q * d + 1, q * d + d - 1) if 0 <= k <= top]
        cases += [(top, d), (top - 1, d), (rng.randint(0, top), d)]
    assert all(ask("q", cases))
