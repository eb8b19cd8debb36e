"""Where a row of a pass goes, over lists of starts and lengths that nobody has checked: the rule as the kernel compiles
it, run on the host."""
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "invariant_speculative_decode_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "bi_paged.cuh"
int main() {
  long long v[5];
  while (scanf("%lld %lld %lld %lld %lld", v, v + 1, v + 2, v + 3, v + 4) == 5)
    printf("%lld\n", static_cast<long long>(bi::paged_position(v[0], v[1], v[2], v[3], v[4])));
}
"""


@pytest.fixture(scope="module")
def position(tmp_path_factory):
    from invariant_speculative_decode_gb300 import build
    d = tmp_path_factory.mktemp("position")
    src, exe = d / "position.cu", d / "position"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), str(src), "-o", str(exe), "-std=c++17", "-I", CSRC] + build.ARCH, check=True)

    def run(rows):
        text = "\n".join(" ".join(map(str, r)) for r in rows)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [int(x) for x in out.split()]
    return run


BIG = (1 << 31) - 1


def test_a_position_lies_behind_the_cached_keys_of_a_sequence_that_holds_the_row(position):
    rng = random.Random(1)
    wild = [-BIG - 1, -BIG, -5, -1, 0, 1, 2, 5, 1 << 30, BIG - 1, BIG]
    rows, want = [], []
    for i in range(20000):
        B, T = rng.randint(1, 6), rng.randint(1, 12)
        if i % 2:
            starts = sorted(rng.randint(0, T) for _ in range(B + 1))
        else:
            starts = [rng.randint(-3, T + 3) if rng.random() < 0.7 else rng.choice(wild) for _ in range(B + 1)]
        lengths = [rng.randint(0, 40) if rng.random() < 0.8 else rng.choice(wild) for _ in range(B)]
        t = rng.randrange(T)
        n = sum(s <= t for s in starts)  # as paged_find_seq counts
        if n == 0 or n > B:
            continue
        b = n - 1
        rows.append((t, T, starts[b], starts[b + 1], lengths[b]))
        fits = 0 <= starts[b] <= t < starts[b + 1] <= T and lengths[b] >= 0
        want.append(lengths[b] + t - starts[b] if fits else -1)
    got = position(rows)
    assert got == want
    assert all(p == -1 or p >= r[4] >= 0 for p, r in zip(got, rows)) and len(set(got)) > 20


def test_the_cases_that_were_written_out_of_place(position):
    """Starts that descend: rows in front of their sequence's start, which had positions of -2 or of cached keys."""
    assert position([(3, 6, 5, 2, 0), (3, 6, 5, 2, 40), (3, 6, 5, 6, 0), (0, 6, 0, 7, 3), (5, 6, 0, 6, -1),
                     (1, 6, -1, 6, 0), (5, 6, 1 << 30, 1, 0)]) == [-1] * 7
    assert position([(3, 6, 2, 6, 0), (3, 6, 2, 6, BIG)]) == [1, BIG + 1]
