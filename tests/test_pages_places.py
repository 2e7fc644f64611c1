"""Places in the list of free pages where sequences together want more pages than 32 bits count (CPU: the plan's
arithmetic, compiled for the host)."""
import os
import subprocess

from tests.conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include "sage_pages.h"
int main() {
    using namespace sage;
    // sequences of 65536 pages each over a pool of 1000; sequence b holds b % 3 pages
    const int B = 40000, want = 1 << 16, free = 1000;
    PageSum at = 0;
    long long given = 0, lowest = 0, later = 0;
    for (int b = 0; b < B; ++b) {
        const int held = b % 3;
        const PageSum more = pages_more(want, held);
        const int got = pages_got(static_cast<int>(more), at, free);
        if (at < lowest) lowest = at;
        given += got;
        if (b > 0) later += got;
        at += more;
    }
    std::printf("%lld %lld %lld %lld\n", static_cast<long long>(at), given, later, lowest);
    std::printf("%d %d %d %d %d\n", pages_got(5, 7, 10), pages_got(5, 10, 10), pages_got(5, 2, 10), pages_got(0, 0, 10),
                pages_got(5, (1ll << 32) + 1, 10));
    std::printf("%lld %lld\n", static_cast<long long>(pages_more(3, 9)), static_cast<long long>(pages_more(9, 3)));
}
"""


def test_places_past_2_31(tmp_path):
    src, exe = tmp_path / "places.cpp", tmp_path / "places"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "bit_trainable_attention_sage_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    out = [list(map(int, line.split())) for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    total = sum((1 << 16) - b % 3 for b in range(40000))
    assert total > 1 << 31
    assert out == [[total, 1000, 0, 0], [3, 0, 5, 0, 0], [0, 6]]


def test_the_workspace_holds_places_of_64_bits():
    import ctypes

    from bit_trainable_attention_sage_gb300 import build
    build.build()
    import bit_trainable_attention_sage_gb300 as sg
    from bit_trainable_attention_sage_gb300.serving import SageKv
    need = lambda B: sg.lib().sage_pages_workspace_bytes(ctypes.byref(SageKv(B, 1, 64, 0, 0, 16, 4, 2)))  # noqa: E731
    # for each sequence a place of 8 bytes and, in 4 bytes each, seven more numbers and its row of the table
    assert need(2000) - need(1000) >= 1000 * (8 + 4 * (7 + 2))
