"""Host-side property test of the decode slot map with spread slots (split_map.cuh):
the slots that proportional splits leave over go to the first sequences that are long
enough.  As in the plain map, the slots must stay within C and every block must belong
to exactly one split.  The per-sequence arithmetic is the library's own (compiled here;
no GPU needed); the hand-out over sequences, which the device does 32 at a time, is
restated one sequence after another."""
import os
import random
import shutil
import subprocess

import pytest

from test_split_map import CSRC, ROOT

NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"

DRIVER = r"""
#include "split_map.cuh"
#include <cstdio>
int main() {
    int B, C, minb, gran;
    while (scanf("%d %d %d %d", &B, &C, &minb, &gran) == 4) {
        static int n[5000], ns[5000];
        long long total = 0; int longest = 0, used = 0;
        for (int i = 0; i < B; ++i) { scanf("%d", &n[i]); total += n[i]; if (n[i] > longest) longest = n[i]; }
        const int bpc = pkvq::split_blocks(total, C, B, longest, minb, gran);
        for (int i = 0; i < B; ++i) { ns[i] = n[i] > bpc ? (n[i] + bpc - 1) / bpc : 1; used += ns[i]; }
        int spare = C - used;
        printf("%d", spare);
        for (int i = 0; i < B; ++i) {
            int mine = bpc;
            if (n[i] > 0) {
                if (pkvq::spread_more(n[i], ns[i], minb) && spare-- > 0) ++ns[i];
                mine = pkvq::spread_blocks(n[i], ns[i], gran);
                ns[i] = (n[i] + mine - 1) / mine;
            }
            printf(" %d %d", ns[i], mine);
        }
        printf("\n");
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not os.path.exists(NVCC):
        pytest.skip("nvcc not found")
    d = tmp_path_factory.mktemp("spread")
    src, exe = d / "drv.cu", d / "drv"
    src.write_text(DRIVER)
    subprocess.run([NVCC, "-std=c++17", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    return str(exe)


def cases():
    rng = random.Random(11)
    yield 8, 111, 8, 1, [2048] * 8
    yield 1, 148, 8, 1, [64]
    yield 3, 3, 4, 1, [5, 100, 7]
    for _ in range(1500):
        B = rng.choice([1, 2, 3, 8, 31, 32, 33, 64, 200])
        pick = rng.choice([lambda: rng.randint(0, 40), lambda: rng.choice([0, 1, 2048, 16384]),
                           lambda: rng.randint(0, 70000), lambda n=rng.randint(1, 9000): n])
        gran = rng.choice([1, 1, 2, 4])
        yield (B, max(B, rng.choice([B, B + 1, 2 * B, 37, 111, 148, 296, 444])), rng.choice([4, 8, 16]) * gran, gran,
               [pick() for _ in range(B)])


def test_spread_slots_fit_and_cover(driver):
    all_cases = list(cases())
    inp = "".join(f"{B} {C} {m} {g} " + " ".join(map(str, n)) + "\n" for B, C, m, g, n in all_cases)
    lines = subprocess.run([driver], input=inp, capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(lines) == len(all_cases)
    for (B, C, minb, gran, n), line in zip(all_cases, lines):
        spare, *rest = map(int, line.split())
        assert spare >= 0
        ns, bpc = rest[::2], rest[1::2]
        assert sum(ns) <= C, (B, C, minb, gran, n)
        for x, s, b in zip(n, ns, bpc):
            assert s >= 1 and b >= 1 and b % gran == 0
            # splits [k b, min(x, (k + 1) b)): none empty, all blocks once
            assert (s - 1) * b < max(x, 1) and s * b >= x
    # the example of the map's own comment: 111 slots over 8 equal sequences
    _, *rest = map(int, lines[0].split())
    assert rest[::2] == [14] * 7 + [13] and rest[1::2] == [147] * 7 + [158]
