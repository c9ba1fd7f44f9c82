"""The integer rules of the 8-bit paged cache, run on the CPU from the source that the kernels are compiled
from (csrc/kv8_rules.h): which rows of which page an append's new tokens go to, which tiles of which segment an
attention CTA takes, where its pieces go and who writes down what is to be joined."""
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


def test_append_units(rules):
    """A unit's sequence is found, and every page of every sequence has a unit of its own."""
    rng = random.Random(4)
    for _ in range(60):
        B = rng.choice([1, 2, 31, 32, 33, 70, rng.randint(1, 400)])
        cu = [0]
        for _ in range(B):
            cu.append(cu[-1] + rng.choice([0, 0, 1, 2, 63, 64, 65, 66, rng.randint(0, 300)]))
        arr = (ctypes.c_int * len(cu))(*cu)
        taken, units = set(), rules.kv8_units(B, cu[-1])
        for b in range(B):
            n = cu[b + 1] - cu[b]
            for i in range(len(_expect(rng.choice([0, 1, 62, 63, 64, rng.randint(0, 1000)]), n))):
                u = rules.kv8_unit_of(arr, B, b) + i
                assert u < units and u not in taken and rules.kv8_sequence_of_unit(arr, B, u) == b
                taken.add(u)


def test_append_shares(rules):
    """At least one share of a page's heads and at most one for each KV head; with few tokens per sequence no more
    CTAs with something to do than a third over what is resident. The shapes named beside the rule."""
    rng = random.Random(8)
    for _ in range(2000):
        B, hkv, group = rng.randint(1, 600), rng.randint(1, 40), rng.randint(1, 8)
        hd = 8 * rng.randint(1, 32)
        threads = 64 * -(-hd // 16)
        n = B * rng.randint(0, 31) + rng.randint(0, B - 1)
        ny = rules.kv8_append_shares(B, n, hkv, hkv * group, threads, 148)
        assert 1 <= ny <= min(hkv, 8)
        if n < 32 * B:
            assert ny == 1 or (B + n // 64) * ny * 3 <= 148 * (1024 // threads) * 4
    for B, new, hkv, hq, hd, want in ((64, 4, 8, 32, 128, 4), (64, 31, 8, 32, 128, 4), (256, 4, 8, 32, 128, 1), (64, 31, 8, 32, 64, 8),
                                      (64, 31, 4, 16, 256, 2), (64, 4, 6, 48, 128, 4), (128, 10, 6, 48, 128, 2), (1, 20, 8, 32, 128, 8),
                                      (1, 32768, 8, 32, 128, 4), (128, 200, 8, 32, 128, 4), (128, 200, 8, 8, 128, 1)):
        assert rules.kv8_append_shares(B, B * new, hkv, hq, 64 * -(-hd // 16), 148) == want, (B, new, hkv, hq, hd)
    assert rules.kv8_append_shares(1 << 20, (1 << 31) - 1, 8, 32, 512, 148) == 4  # nothing wraps
    assert rules.kv8_append_shares(1 << 26, 1 << 30, 8, 32, 512, 148) == 1


def _divide(rules, lens, hkv, max_pages, window, n_cta, cluster, visit=-1):
    """(pieces of every segment, written-down segments) as the CTAs find them."""
    arr = (ctypes.c_int * len(lens))(*lens)
    room, slots = len(lens) * hkv + 1, n_cta + 1
    out, record = (ctypes.c_int * (6 * room))(), (ctypes.c_int * (2 + slots))()
    pieces, records = {}, {}
    for c in range(n_cta):
        seen = ctypes.c_longlong(0)
        n = rules.kv8_cta(arr, len(lens), hkv, max_pages, window, n_cta, cluster, c, out, room, record, slots, visit, ctypes.byref(seen))
        got = [tuple(out[6 * i:6 * i + 6]) for i in range(n)]
        for b, h, t0, t1, whole, slot in got:
            pieces.setdefault((b, h), []).append((c, t0, t1, whole, slot))
        if visit >= 0:
            assert seen.value == sum(t1 - t0 for _, _, t0, t1, _, _ in got)
        if record[1]:
            assert record[0] not in records and record[1] <= slots
            records[record[0]] = list(record[2:2 + record[1]])
    return pieces, records


def _check(rules, lens, hkv, max_pages, window, n_cta, cluster=0, visit=-1):
    pieces, records = _divide(rules, lens, hkv, max_pages, window, n_cta, cluster, visit)
    used = set()
    for b, length in enumerate(lens):
        length = min(max(length, 0), 64 * max_pages)
        page0 = max(0, length - window) // 64 if window else 0
        tiles = (-(-length // 64) - page0 + 1) // 2 if length else 0
        for h in range(hkv):
            got = pieces.pop((b, h), [])
            assert [c for c, *_ in got] == sorted({c for c, *_ in got})
            at = 0
            for _, t0, t1, _, _ in got:  # in order, without gap or overlap
                assert t0 == at and t1 > t0
                at = t1
            assert at == tiles
            assert all(whole == (len(got) == 1) for *_, whole, _ in got)
            if len(got) > 1:
                slots = [slot for *_, slot in got]
                assert not used & set(slots) and max(slots) < 2 * n_cta
                used |= set(slots)
                if not cluster:  # written down once, the slots in the order of the tiles
                    assert records.pop(b * hkv + h) == slots
                else:
                    seg = b * hkv + h
                    assert slots == [2 * (seg * cluster + i) for i in range(len(got))]
    assert not pieces and not records


def test_division(rules):
    rng = random.Random(5)
    for _ in range(300):
        B, hkv, width = rng.choice([1, 2, 3, 17, 60]), rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 5, 40])
        lens = [rng.choice([0, 0, 1, 64, 65, 128, 129, rng.randint(0, 64 * width), 64 * width + 9, -3]) for _ in range(B)]
        window = rng.choice([0, 0, 1, 63, 64, 65, rng.randint(1, 3000)])
        _check(rules, lens, hkv, width, window, rng.choice([1, 2, 7, 40, 296]), visit=rng.choice([0, 1, 16]))


def test_division_of_long_lines(rules):
    """Totals on both sides of where 32-bit divisions end, and up to full tables of the largest width."""
    edge = (2 ** 31 - 1) // 2048
    rng = random.Random(6)
    for units in (edge - 1, edge, edge + 1, edge + 12345):
        for n_cta in (1, 296, 1024):
            tiles = units - 2 - 7  # the second sequence has 5 tiles
            _check(rules, [128 * tiles, 640], 1, 2 * tiles, 0, n_cta)
            # and cut at random into shorter ones
            cut = sorted(rng.sample(range(3, units), 6))
            lens = [128 * max(0, y - x - 2) for x, y in zip([0] + cut, cut + [units])]
            _check(rules, lens, 1, max(1, max(lens) // 64), 0, n_cta)
    for n_cta in (1, 148, 296, 1024):
        _check(rules, [LAST, 0, LAST - 1, 5], 8, LAST // 64, 0, n_cta)
        _check(rules, [LAST, 0, LAST - 1, 5], 8, LAST // 64, 64 * 1000 + 1, n_cta)


def test_small_calls(rules):
    """A cluster has a segment: its CTAs take all tiles in order. At most 8 pieces to join, 4 tiles to a CTA, 2048
    page ids to check, and all CTAs of one wave."""
    rng = random.Random(7)
    clusters = set()
    for _ in range(2000):
        B, hkv, width = rng.choice([1, 2, 3, 8, 40, 256]), rng.choice([1, 2, 4, 8, 32]), rng.choice([1, 2, 3, 8, 16, 64, rng.randint(1, 80)])
        tensor = rng.randint(0, 1)
        c = rules.kv8_small_cluster(B, hkv, width, tensor)
        tiles = (width + 1) // 2
        if not c:
            most = max([x for x in (1, 2, 4, 8) if B * hkv * x <= 256], default=0)
            assert tiles > (4 if tensor else 2) * most
            continue
        clusters.add(c)
        assert c in (1, 2, 4, 8) and B * hkv * c <= 256 and -(-tiles // c) <= (4 if tensor else 2) and B * width <= 2048
        if rng.random() < 0.1:
            lens = [rng.choice([0, 1, 64 * width, 64 * width + 5, -1, rng.randint(0, 64 * width)]) for _ in range(B)]
            _check(rules, lens, hkv, width, rng.choice([0, 0, 100]), B * hkv * c, cluster=c, visit=16)
    assert clusters == {1, 2, 4, 8}
    assert [rules.kv8_small_cluster(0, 8, 1, 1), rules.kv8_small_cluster(1 << 30, 1 << 10, 1, 1)] == [0, 0]


@pytest.fixture(scope="module")
def lib():
    from long_context_decode_lr_b200 import lowram as lr
    lrbuild.build()
    return lr.library()


@pytest.mark.parametrize("batch,hkv,hq", [((1 << 26) + 1, 1, 1), (1 << 26, 8, 32), (1 << 20, 2048, 2048), (1 << 14, 1 << 17, 1 << 17)])
def test_sizes_past_an_int_are_refused(lib, batch, hkv, hq):
    """Batches whose units, warps or heads an int does not count."""
    from long_context_decode_lr_b200 import lowram as lr
    P = 0x10000
    kv = ctypes.byref(lr.lr_kv8_pages(batch, hkv, 8, 10, 4, lr.LR_BF16, 0, P, P, P, P, P, P))
    assert lib.lr_kv8_append(kv, hq, batch, None, None, P, 0, P, 0, P, 0, P, P, 256, None) == lr.LR_ERR_UNSUPPORTED
    assert lib.lr_decode_attn_kv8(kv, hq, P, 0, 0.0, None, None, P, None, P, 1 << 50, None) == lr.LR_ERR_UNSUPPORTED
    assert lib.lr_kv8_attn_workspace_bytes(kv, hq) == 0
    if batch <= 1 << 26 and batch * hkv < 1 << 31:  # without queries an append of it is fine as far as the host goes
        assert lib.lr_kv8_append(kv, 0, batch, None, None, None, 0, P, 0, P, 0, None, P, 255, None) == lr.LR_ERR_WORKSPACE
