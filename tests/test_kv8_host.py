"""The 8-bit paged cache's entry points refuse bad arguments on the host before touching device memory,
and the rules by which the attention divides its tiles and the append finds its pages hold (CPU only)."""
import ctypes
import random

import pytest

from long_context_decode_lr_b200 import build as lrbuild
from long_context_decode_lr_b200 import lowram as lr

FAKE = 0x10000  # a 256-byte-aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    lrbuild.build()
    return lr.library()


def _kv(**kw):
    d = dict(batch=2, n_kv_heads=8, head_dim=128, n_pages=10, max_pages=4, dtype=lr.LR_BF16, page_stride=0,
             k_codes=FAKE, v_codes=FAKE, k_scale=FAKE, v_scale=FAKE, page_table=FAKE, lens=FAKE)
    d.update(kw)
    return ctypes.byref(lr.lr_kv8_pages(*[d[f] for f, _ in lr.lr_kv8_pages._fields_]))


def _rope(**kw):
    d = dict(inv_freq=FAKE, rot_dim=128, interleaved=0)
    d.update(kw)
    return ctypes.byref(lr.lr_rope(*[d[f] for f, _ in lr.lr_rope._fields_]))


BAD_KV = [
    (dict(batch=-1), lr.LR_ERR_INVALID_ARG), (dict(n_kv_heads=0), lr.LR_ERR_INVALID_ARG),
    (dict(head_dim=0), lr.LR_ERR_INVALID_ARG), (dict(head_dim=12), lr.LR_ERR_UNSUPPORTED),
    (dict(head_dim=264), lr.LR_ERR_UNSUPPORTED), (dict(n_pages=0), lr.LR_ERR_INVALID_ARG),
    (dict(max_pages=0), lr.LR_ERR_INVALID_ARG), (dict(max_pages=1 << 25), lr.LR_ERR_UNSUPPORTED),
    (dict(dtype=2), lr.LR_ERR_INVALID_ARG), (dict(page_stride=65536 - 16), lr.LR_ERR_INVALID_ARG),
    (dict(page_stride=65536 + 8), lr.LR_ERR_INVALID_ARG), (dict(page_stride=-65536), lr.LR_ERR_INVALID_ARG),
    (dict(k_codes=None), lr.LR_ERR_INVALID_ARG), (dict(v_codes=FAKE + 8), lr.LR_ERR_INVALID_ARG),
    (dict(k_scale=None), lr.LR_ERR_INVALID_ARG), (dict(v_scale=FAKE + 4), lr.LR_ERR_INVALID_ARG),
    (dict(page_table=None), lr.LR_ERR_INVALID_ARG), (dict(lens=None), lr.LR_ERR_INVALID_ARG),
    (dict(n_kv_heads=9000), lr.LR_ERR_UNSUPPORTED),
]


def _append(lib, kv=None, hq=32, n=2, cu=None, rope=None, q=FAKE, qs=0, k=FAKE, ks=0, v=FAKE, vs=0, q_out=2 * FAKE, ws=FAKE,
            ws_bytes=256):
    return lib.lr_kv8_append(kv or _kv(), hq, n, cu, rope, q, qs, k, ks, v, vs, q_out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), lr.LR_ERR_INVALID_ARG), (dict(n=3), lr.LR_ERR_INVALID_ARG),
    (dict(cu=FAKE + 4), lr.LR_ERR_INVALID_ARG), (dict(q=None), lr.LR_ERR_INVALID_ARG),
    (dict(q_out=None), lr.LR_ERR_INVALID_ARG), (dict(hq=0), lr.LR_ERR_INVALID_ARG),
    (dict(k=None), lr.LR_ERR_INVALID_ARG), (dict(v=FAKE + 2), lr.LR_ERR_INVALID_ARG),
    (dict(q=FAKE + 8), lr.LR_ERR_INVALID_ARG), (dict(ks=1016), lr.LR_ERR_INVALID_ARG),
    (dict(ks=1028), lr.LR_ERR_INVALID_ARG), (dict(vs=-1024), lr.LR_ERR_INVALID_ARG),
    (dict(qs=4095), lr.LR_ERR_INVALID_ARG), (dict(q_out=FAKE, qs=8192), lr.LR_ERR_INVALID_ARG),
    (dict(rope=_rope(rot_dim=144)), lr.LR_ERR_INVALID_ARG), (dict(rope=_rope(rot_dim=24)), lr.LR_ERR_UNSUPPORTED),
    (dict(rope=_rope(rot_dim=-16)), lr.LR_ERR_INVALID_ARG), (dict(rope=_rope(interleaved=2)), lr.LR_ERR_INVALID_ARG),
    (dict(rope=_rope(inv_freq=None)), lr.LR_ERR_INVALID_ARG), (dict(ws=None), lr.LR_ERR_INVALID_ARG),
    (dict(ws=FAKE + 16), lr.LR_ERR_INVALID_ARG), (dict(ws_bytes=255), lr.LR_ERR_WORKSPACE),
])
def test_append_refuses(lib, kw, status):
    assert _append(lib, **kw) == status
    assert lib.lr_last_error()


@pytest.mark.parametrize("kw,status", BAD_KV)
def test_bad_cache_is_refused(lib, kw, status):
    assert _append(lib, kv=_kv(**kw)) == status
    assert _attn(lib, kv=_kv(**kw)) == status
    assert lib.lr_kv8_append_workspace_bytes(_kv(**kw)) == 0
    assert lib.lr_kv8_attn_workspace_bytes(_kv(**kw), 32) == 0


def _attn(lib, kv=None, hq=32, q=FAKE, window=0, o_prev=None, lse_prev=None, o=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return lib.lr_decode_attn_kv8(kv or _kv(), hq, q, window, 0.0, o_prev, lse_prev, o, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(hq=0), lr.LR_ERR_INVALID_ARG), (dict(hq=33), lr.LR_ERR_INVALID_ARG), (dict(hq=72), lr.LR_ERR_UNSUPPORTED),
    (dict(q=None), lr.LR_ERR_INVALID_ARG), (dict(o=None), lr.LR_ERR_INVALID_ARG), (dict(q=FAKE + 2), lr.LR_ERR_INVALID_ARG),
    (dict(lse=FAKE + 4), lr.LR_ERR_INVALID_ARG), (dict(window=-1), lr.LR_ERR_INVALID_ARG),
    (dict(o_prev=FAKE), lr.LR_ERR_INVALID_ARG), (dict(lse_prev=FAKE), lr.LR_ERR_INVALID_ARG),
    (dict(o_prev=FAKE, lse_prev=FAKE + 4), lr.LR_ERR_INVALID_ARG), (dict(ws=None), lr.LR_ERR_INVALID_ARG),
    (dict(ws=FAKE + 64), lr.LR_ERR_INVALID_ARG), (dict(ws_bytes=512), lr.LR_ERR_WORKSPACE),
])
def test_attention_refuses(lib, kw, status):
    assert _attn(lib, **kw) == status
    assert lib.lr_last_error()


def test_null_cache_and_lse(lib):
    assert lib.lr_kv8_append(None, 32, 2, None, None, FAKE, 0, FAKE, 0, FAKE, 0, FAKE, FAKE, 256, None) == lr.LR_ERR_INVALID_ARG
    assert lib.lr_decode_attn_kv8(None, 32, FAKE, 0, 0.0, None, None, FAKE, None, FAKE, 1 << 40, None) == lr.LR_ERR_INVALID_ARG
    shape = lr.lr_cache_shape(1, 1000, 2, 2, 128, 128, 256, lr.LR_BF16)
    pred = lr.lr_predictor(FAKE, FAKE, FAKE, FAKE, None, 1)
    for lse in (None, FAKE + 4):
        assert lib.lr_decode_attn_lse(ctypes.byref(shape), 0, 8, FAKE, FAKE, FAKE, ctypes.byref(pred), FAKE, FAKE, None, 10,
                                      None, 0, 0.0, FAKE, lse, FAKE, 1 << 40, None) == lr.LR_ERR_INVALID_ARG
    assert 256 < lib.lr_kv8_attn_workspace_bytes(_kv(), 32) < lib.lr_kv8_attn_workspace_bytes(_kv(batch=64), 32)


def _divide(tiles, n_cta):
    """The attention's division of the segments' tiles, as its kernels do it (a segment takes two units more than
    it has tiles): (CTA, first, last + 1) pieces of every segment, and the pieces' slots."""
    units = [t + 2 if t else 0 for t in tiles]
    total, active = sum(units), min(n_cta, sum(units))
    first = [sum(units[:i]) for i in range(len(tiles))]
    pieces = {i: [] for i in range(len(tiles))}
    slots = {}
    for c in range(active):
        at, end = total * c // active, total * (c + 1) // active
        while at < end:
            s = max(i for i in range(len(tiles)) if tiles[i] and first[i] <= at)
            stop = min(first[s] + tiles[s], end)
            if stop <= at:  # only units behind the tiles
                at = first[s] + units[s]
                continue
            whole = at == first[s] and stop == first[s] + tiles[s]
            pieces[s].append((c, at, stop))
            if not whole:
                c0 = ((first[s] + 1) * active - 1) // total
                c1 = ((first[s] + tiles[s]) * active - 1) // total
                slot = 2 * c + (1 if total * c // active < first[s] else 0)
                assert (c, s) not in slots and slot not in slots.values()
                slots[(c, s)] = slot
                assert c0 <= c <= c1
                pieces.setdefault(("span", s), (c0, c1))
            at = first[s] + units[s]
    return first, pieces, slots


def test_tiles_are_divided_without_gap_or_overlap():
    rng = random.Random(0)
    for _ in range(300):
        n = rng.randint(1, 40)
        tiles = [rng.choice([0, 1, 2, 3, rng.randint(0, 60)]) for _ in range(n)]
        if not sum(tiles):
            continue
        n_cta = rng.randint(1, 40)
        first, pieces, slots = _divide(tiles, n_cta)
        owners = set()
        for s, t in enumerate(tiles):
            got = pieces[s]
            assert sum(b - a for _, a, b in got) == t
            at = first[s]
            for _, a, b in got:
                assert a == at
                at = b
            if ("span", s) in pieces:  # every CTA of the span has exactly one piece, and one counter counts them
                c0, c1 = pieces[("span", s)]
                assert [c for c, _, _ in got] == list(range(c0, c1 + 1))
                assert c0 not in owners
                owners.add(c0)
        assert all(0 <= x < 2 * n_cta for x in slots.values())


def test_append_units_cover_every_page():
    """Sequence b's pages are units cu[b] / 64 + 2 b and on: never more pages than units, and the 32-way
    search finds the sequence of every unit."""
    rng = random.Random(1)

    def search(cu, B, u):
        b, n = 0, B
        while n > 1:
            step = (n + 31) // 32
            below = [lane * step < n and (lane == 0 or cu[b + lane * step] // 64 + 2 * (b + lane * step) <= u) for lane in range(32)]
            i = sum(below) - 1
            b, n = b + i * step, min(step, n - i * step)
        return b

    for _ in range(200):
        B = rng.choice([1, 2, 31, 32, 33, 70, rng.randint(1, 1500)])
        cu = [0]
        for _ in range(B):
            cu.append(cu[-1] + rng.choice([0, 0, 1, 2, 63, 64, 65, 66, rng.randint(0, 300)]))
        units = cu[-1] // 64 + 2 * B
        seen = set()
        for b in range(B):
            n, p0 = cu[b + 1] - cu[b], rng.choice([0, 1, 62, 63, 64, rng.randint(0, 1000)])
            off = cu[b] // 64 + 2 * b
            pages = 0 if n == 0 else (p0 + n - 1) // 64 - p0 // 64 + 1
            for i in range(pages):
                u = off + i
                assert u < units and u not in seen
                seen.add(u)
                if B < 80 or rng.random() < 0.02:
                    assert search(cu, B, u) == b
