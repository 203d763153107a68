"""The rope operators' frequency table, computed on the host, against 60-digit arithmetic (CPU only)."""
import ctypes
import math
import subprocess
from decimal import Decimal, getcontext

import pytest

from layout_agnostic_paged_gb300 import build as B
from layout_agnostic_paged_gb300 import splash as S

SOURCE = """
#include "rope_table.h"
extern "C" void table(const splash_rope_desc* d, uint64_t* turns) { splash::rope_table(*d, turns); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("rope_table")
    (d / "t.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", B.CSRC, "-I", B.INCLUDE, str(d / "t.cpp"),
                    "-o", str(d / "t.so")], check=True)
    return ctypes.CDLL(str(d / "t.so"))


def arctan_inverse(n):
    """arctan(1 / n), by its series."""
    x, s, k = Decimal(1) / n, Decimal(0), 0
    while abs(x) > Decimal(10) ** -70:
        s += x / (2 * k + 1) * (-1) ** k
        x /= n * n
        k += 1
    return s


def exact_turns(dims, base, scaling, factor=1.0, orig_ctx=4096.0, beta_fast=32.0, beta_slow=1.0, **_):
    """f_i / (2 pi) * 2^64 of every pair."""
    getcontext().prec = 60
    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    ln, fac = Decimal(base).ln(), Decimal(factor)
    if scaling == "yarn":
        pair = lambda b: dims * math.log(orig_ctx / (2 * math.pi * b)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), dims - 1)
    out = []
    for i in range(dims // 2):
        f = (ln * (Decimal(-2 * i) / dims)).exp()
        if scaling == "linear":
            f /= fac
        elif scaling == "yarn":
            g = min(max(Decimal(i - lo) / max(Decimal(hi - lo), Decimal("0.001")), Decimal(0)), Decimal(1))
            f *= 1 - g + g / fac
        out.append(f / (2 * pi) * 2 ** 64)
    return out


@pytest.mark.parametrize("dims", [2, 6, 32, 64, 128, 256])
@pytest.mark.parametrize("kw", [
    dict(base=10000.0), dict(base=500000.0), dict(base=1.0), dict(base=1.7), dict(base=1e9), dict(base=150000.0),
    dict(base=500000.0, scaling="linear", factor=8.0), dict(base=10000.0, scaling="linear", factor=3.7),
    dict(base=10000.0, scaling="yarn", factor=40.0), dict(base=1e6, scaling="yarn", factor=2.5, orig_ctx=32768.0),
    dict(base=150000.0, scaling="yarn", factor=32.0, beta_fast=1.0, beta_slow=1.0)])
def test_every_entry_is_rounded_once(lib, dims, kw):
    kw = dict(dict(scaling="none"), **kw)
    table = (ctypes.c_uint64 * (dims // 2))()
    lib.table(ctypes.byref(S.make_rope_desc(dims, **kw)), table)
    for got, want in zip(table, exact_turns(dims, **kw)):
        # half a unit, and 100 bits of a number below 2^62
        assert abs(Decimal(got) - want) <= Decimal("0.5") + Decimal(2) ** -30, (got, want)
