"""Division by a fixed divisor as a product and a shift (csrc/chunk.h), against the machine's own (CPU only)."""
import os
import subprocess
import tempfile

from layout_agnostic_paged_gb300 import build as B

SOURCE = r"""
#include <stdio.h>
#include "chunk.h"
using namespace splash;
int main() {
    const int most = 2147483647;
    uint64_t x = 88172645463325252ull;
    auto random = [&]() { x ^= x << 13; x ^= x >> 7; x ^= x << 17; return int(x >> 33); };
    for (int i = 0; i < 3000; ++i) {
        // every small divisor, the powers of two and their neighbours, and others
        const int d = i < 2100 ? i + 1 : (i < 2193 ? (1 << (i - 2100) / 3) + (i - 2100) % 3 - 1 : random() | 1);
        if (d < 1) continue;
        const FastDiv f = fast_div(d);
        const int top = most / d * d;                 // the last multiple, and what lies around multiples
        const int fixed[] = {0, 1, d - 1, d, d < most ? d + 1 : d, top - 1, top, most - 1, most};
        for (int n : fixed)
            if (n >= 0 && f(n) != n / d) return printf("%d / %d\n", n, d), 1;
        for (int k = 0; k < 300; ++k) {
            const int n = random(), m = n / d * d;
            if (f(n) != n / d || f(m) != m / d || (m > 0 && f(m - 1) != (m - 1) / d)) return printf("%d / %d\n", n, d), 1;
        }
    }
    return 0;
}
"""


def test_quotients():
    cuda = os.path.join(os.path.dirname(os.path.dirname(B.nvcc())), "include")
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "t.cpp"), os.path.join(d, "t")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-I", cuda, "-I", B.INCLUDE, "-I", B.CSRC, src, "-o", exe], check=True)
        r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
