"""The integer rules of the 8-bit paged cache, run on the CPU from the source that the kernels are compiled
from (csrc/kv8_rules.h): which rows of which page an append's new tokens go to."""
import ctypes
import os
import random
import subprocess

import pytest

from long_context_decode_lr_b200 import build as lrbuild

HERE = os.path.dirname(os.path.abspath(__file__))
LAST = 64 * ((1 << 25) - 1)  # the longest sequence: max_pages = 2^25 - 1 full pages


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("rules") / "kv8_rules.so")
    # signed overflow ends the program instead of going unnoticed
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-shared", "-fPIC", "-I", lrbuild.CSRC, "-I", lrbuild.INCLUDE,
                    os.path.join(HERE, "kv8_rules_host.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def _pages(rules, p0, n, tries):
    got, out = [], (ctypes.c_int * 3)()
    for i in range(tries):
        if rules.kv8_page_rows(p0, n, i, out):
            got.append(tuple(out))
    return got


def _expect(p0, n):
    pages = range(p0 // 64, (p0 + n - 1) // 64 + 1) if n > 0 else ()
    return [(p, max(p0, 64 * p), min(p0 + n, 64 * p + 64)) for p in pages]


def test_page_rows(rules):
    rng = random.Random(3)
    for _ in range(2000):
        p0, n = rng.choice([0, 1, 63, 64, 65, rng.randint(0, 10000)]), rng.choice([0, 1, 2, 63, 64, 65, rng.randint(0, 500)])
        assert _pages(rules, p0, n, n // 64 + 4) == _expect(p0, n)
    assert not rules.kv8_page_rows(10, 5, -1, (ctypes.c_int * 3)())


@pytest.mark.parametrize("n", [1, 63, 64, 65, 128, 1000])
def test_page_rows_up_to_the_longest_sequence(rules, n):
    """Spare units behind the last page of a full table give nothing: no position wraps around."""
    assert _pages(rules, LAST - n, n, n // 64 + 4) == _expect(LAST - n, n)
