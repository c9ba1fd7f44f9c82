"""The 8-bit paged cache on the GPU against the fp64 oracle: lr_kv8_append and lr_decode_attn_kv8 by
themselves, and in the decode loop a user runs (append, attend, joined with the packed context)."""
import numpy as np
import pytest
import torch

from long_context_decode_lr_b200 import lowram as lr
from oracle import kv8_oracle as orc

import helpers as H
from kv8_helpers import DT, HALF, Pool, attend, check_attention, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from long_context_decode_lr_b200 import build
    build.build()
    lr.library()


def inv_freq(rot, base=500000.0):
    return (1.0 / base ** (np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)


# ------------------------------------------------------------------------------- append

def run_append(pool, k, v, q, cu, rot, interleaved, q_out=None, stream=None):
    n = k.shape[0]
    q_out = torch.full((n, q.shape[1], pool.hd), 7.0, dtype=k.dtype, device="cuda") if q_out is None else q_out
    rope = lr.Rope(torch.from_numpy(inv_freq(rot)).cuda(), rot, interleaved) if rot else None
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    cu_dev = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    lr.lr_kv8_append(pool.kv, k, v, ws, cu_tokens=cu_dev, rope=rope, q=q, q_out=q_out, stream=stream)
    return q_out, lr.lr_get_device_error(ws, stream)


def check_append(pool, before, k, v, q, q_out, cu, rot, interleaved, bounds=True):
    """Values: unrotated numbers must be the codes of the oracle; rotated ones may be off by half a code step
    plus the fp32 rotation (two products and a sum, sine and cosine: under 2^-21 (|x0| + |x1|))."""
    want = [x.copy() for x in before]
    inv = inv_freq(rot)
    kr, touched = orc.append(*want, pool.table, pool.lens, cu, k, v, inv, rot, interleaved)
    got = pool.arrays()
    np.testing.assert_array_equal(got[3], want[3])  # value scales
    np.testing.assert_array_equal(got[1], want[1])  # value codes, untouched bytes included
    pages = np.zeros(got[2].shape, bool)
    for t in touched:
        pages[t] = True
    np.testing.assert_array_equal(got[2][~pages], want[2][~pages])
    np.testing.assert_array_equal(got[0][~pages], want[0][~pages])
    same_scale = got[2] == want[2]
    assert (got[2][pages] / want[2][pages] <= 2).all() and (got[2][pages] / want[2][pages] >= 0.5).all()
    assert same_scale[pages].mean() > 0.99  # a maximum within rounding of a power of two may go either way
    for b in range(len(pool.lens)):
        n = int(cu[b + 1] - cu[b])
        p0 = int(pool.lens[b]) - n
        held = range(p0 // 64 * 64, p0) if n else ()
        for t in held:  # the codes held before
            page = pool.table[b, t // 64]
            ok = same_scale[page]
            np.testing.assert_array_equal(got[0][page][ok, t % 64], want[0][page][ok, t % 64])
        if p0 // 64 != (p0 + n - 1) // 64 or n:
            for pg in range(p0 // 64, -(-int(pool.lens[b]) // 64) if n else p0 // 64):  # rows behind
                page, e = pool.table[b, pg], min(64, int(pool.lens[b]) - 64 * pg)
                np.testing.assert_array_equal(got[0][page][:, e:], want[0][page][:, e:])
        for i in range(n):
            x, page, slot = kr[cu[b] + i], pool.table[b, (p0 + i) // 64], (p0 + i) % 64
            s = got[2][page].astype(np.float64)[:, None]
            mag = np.abs(x)
            if rot:
                j = np.arange(rot // 2)
                i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, rot // 2 + j)
                pair = np.abs(k[cu[b] + i][:, i0]) + np.abs(k[cu[b] + i][:, i1])
                slack = np.zeros_like(x)
                slack[:, i0] = slack[:, i1] = pair * 2.0 ** -21
            else:
                slack = 0.0
            step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(mag / s, 1e-30))) - 3), 2.0 ** -9)
            y = orc.E4M3[got[0][page, :, slot]] * s
            assert (np.abs(y - x) <= step * s / 2 + 2 * slack).all()
    if q is not None:
        dev = q_out.double().cpu().numpy()
        for b in range(len(pool.lens)):
            n = int(cu[b + 1] - cu[b])
            for i in range(n):
                x = q[cu[b] + i]
                y = orc.rotate(x, int(pool.lens[b]) - n + i, inv, rot, interleaved) if rot else x
                lim = HALF[pool.dtype] * np.abs(y) + (2.0 ** -21 * 2 * np.abs(x).max() if rot else 0.0)
                assert (np.abs(dev[cu[b] + i] - y) <= lim).all()


APPENDS = {
    # new tokens per sequence, tokens held before, KV heads, query heads, head_dim, rotated dims, interleaved, dtype
    "prompt_bf16": dict(new=[130], before=[0], hkv=2, hq=8, hd=128, rot=128, inter=False),
    "chunk_mid_page": dict(new=[70, 3], before=[30, 127], hkv=2, hq=4, hd=128, rot=128, inter=False),
    "ragged_with_none": dict(new=[1, 0, 65, 2, 0, 64], before=[5, 9, 63, 64, 0, 0], hkv=1, hq=3, hd=128, rot=64, inter=False),
    "interleaved_partial": dict(new=[33, 1, 100], before=[1, 62, 28], hkv=3, hq=3, hd=128, rot=32, inter=True),
    "no_rotation": dict(new=[40, 40], before=[50, 0], hkv=2, hq=2, hd=128, rot=0, inter=False),
    "fp32_hd64": dict(new=[90, 11], before=[0, 60], hkv=2, hq=4, hd=64, rot=64, inter=False, dtype="f32"),
    "fp32_interleaved": dict(new=[66], before=[3], hkv=1, hq=2, hd=64, rot=64, inter=True, dtype="f32"),
    "hd256": dict(new=[65], before=[10], hkv=1, hq=2, hd=256, rot=256, inter=False),
    "hd40": dict(new=[65, 2], before=[10, 0], hkv=2, hq=2, hd=40, rot=16, inter=False),
    "hd8": dict(new=[7], before=[0], hkv=1, hq=1, hd=8, rot=0, inter=False, dtype="f32"),
    "hd96_half_rotated": dict(new=[70, 5], before=[10, 0], hkv=3, hq=9, hd=96, rot=48, inter=False),
    "hd72_interleaved": dict(new=[65], before=[3], hkv=1, hq=3, hd=72, rot=64, inter=True),
    "fp32_hd256": dict(new=[100], before=[7], hkv=2, hq=2, hd=256, rot=256, inter=False, dtype="f32"),
    "more_heads_than_shares": dict(new=[130, 1, 64], before=[0, 63, 64], hkv=11, hq=22, hd=64, rot=64, inter=True),
    "many_short": dict(new=[2] * 40, before=list(range(40)), hkv=1, hq=1, hd=64, rot=64, inter=False),
    "one_each": dict(new=None, before=[0, 63, 64, 17, 200], hkv=2, hq=8, hd=128, rot=128, inter=False),
    "one_each_interleaved_f32": dict(new=None, before=[1, 0, 130], hkv=2, hq=4, hd=64, rot=32, inter=True, dtype="f32"),
    "one_each_hd256": dict(new=None, before=[1, 64], hkv=1, hq=2, hd=256, rot=128, inter=False),
    "one_each_hd8": dict(new=None, before=[1, 64], hkv=1, hq=2, hd=8, rot=0, inter=False),
}


@pytest.mark.parametrize("name", list(APPENDS))
def test_append(name):
    c = APPENDS[name]
    dtype = c.get("dtype", "bf16")
    rng = np.random.default_rng(len(name))
    new = [1] * len(c["before"]) if c["new"] is None else c["new"]
    after = [p + n for p, n in zip(c["before"], new)]
    pool = Pool(rng, c["before"], c["hkv"], c["hd"], dtype, room=after)
    pool.set_lens(after)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(int)
    n = int(cu[-1])
    grow = 10.0 ** rng.uniform(-1.5, 1.5, (n, 1, 1))  # scales rise within pages
    k, kr = rounded(rng.standard_normal((n, c["hkv"], c["hd"])) * grow, dtype)
    v, vr = rounded(rng.standard_normal((n, c["hkv"], c["hd"])) * grow, dtype)
    q, qr = rounded(rng.standard_normal((n, c["hq"], c["hd"])), dtype)
    before = [x.copy() for x in (pool.kc, pool.vc, pool.ks, pool.vs)]
    q_out, err = run_append(pool, k, v, q, None if c["new"] is None else cu, c["rot"], c["inter"])
    assert err == 0
    check_append(pool, before, kr, vr, qr, q_out, cu, c["rot"], c["inter"])
    # the same call again changes nothing
    once = pool.arrays()
    run_append(pool, k, v, q, None if c["new"] is None else cu, c["rot"], c["inter"])
    for x, y in zip(once, pool.arrays()):
        np.testing.assert_array_equal(x, y)


def test_append_views_strides_and_in_place():
    """k, v, q as slices of a fused tensor; K and V pages side by side in one pool; q_out = q."""
    rng = np.random.default_rng(3)
    hkv, hq, hd, before, new = 2, 4, 128, [20, 64], [50, 3]
    after = [p + n for p, n in zip(before, new)]
    pool = Pool(rng, before, hkv, hd, room=after)
    both = torch.zeros((pool.kc.shape[0], 2, hkv, 64, hd), dtype=torch.uint8, device="cuda")
    both[:, 0].copy_(torch.from_numpy(pool.kc)), both[:, 1].copy_(torch.from_numpy(pool.vc))
    pool.dev[0], pool.dev[1] = both[:, 0], both[:, 1]
    pool.kv = lr.Kv8Pages(*pool.dev, torch.bfloat16)
    pool.set_lens(after)
    n = sum(new)
    cu = np.array([0, 50, 53])
    x, xr = rounded(rng.standard_normal((n, hq + 2 * hkv, hd)), "bf16")
    q = x[:, :hq].contiguous()
    keep = [pool.kc.copy(), pool.vc.copy(), pool.ks.copy(), pool.vs.copy()]
    q_out, err = run_append(pool, x[:, hq:hq + hkv], x[:, hq + hkv:], q, cu, 128, False, q_out=q)
    assert err == 0 and q_out is q
    check_append(pool, keep, xr[:, hq:hq + hkv], xr[:, hq + hkv:], xr[:, :hq], q_out, cu, 128, False)
    # a strided q into a dense q_out gives the same
    fresh = torch.empty_like(q)
    run_append(pool, x[:, hq:hq + hkv], x[:, hq + hkv:], x[:, :hq], cu, 128, False, q_out=fresh)
    assert torch.equal(fresh, q)
    # one token each, strided, without queries
    pool.set_lens([a + 1 for a in before])
    ws = lr.workspace(256)
    lr.lr_kv8_append(pool.kv, x[:2, hq:hq + hkv], x[:2, hq + hkv:], ws, rope=None)
    assert lr.lr_get_device_error(ws) == 0


@pytest.mark.parametrize("single", [False, True])
def test_append_non_finite(single):
    """NaN and infinities become NaN codes of their own places and leave the scale to the others."""
    rng = np.random.default_rng(4)
    pool = Pool(rng, [3], 1, 128, room=[64])
    pool.set_lens([4])
    k = np.ones((1, 1, 128), np.float32)
    k[0, 0, 5], k[0, 0, 70] = np.inf, np.nan
    v = np.full((1, 1, 128), 3.0, np.float32)
    v[0, 0, 0] = -np.inf
    (kd, kr), (vd, vr) = rounded(k, "bf16"), rounded(v, "bf16")
    keep = [x.copy() for x in (pool.kc, pool.vc, pool.ks, pool.vs)]
    run_append(pool, kd, vd, kd, None if single else [0, 1], 0, False)
    orc.append(*keep, pool.table, pool.lens, [0, 1], kr, vr, [], 0, False)
    for got, want in zip(pool.arrays(), keep):
        np.testing.assert_array_equal(got, want)
    assert np.isnan(orc.E4M3[pool.arrays()[1][pool.table[0, 0], 0, 3, 0]])


@pytest.mark.parametrize("single", [False, True])
def test_append_far_positions_and_large_pool(single):
    """Positions near 10^9 (exact angles) and codes more than 2^32 bytes into the pool."""
    rng = np.random.default_rng(5)
    hkv, hd, n_pages = 8, 128, 67000  # 64 KB a page: 4.4 GB each of K and V
    pos = 64 * 16_000_000 + 10
    kc, vc = (torch.zeros((n_pages, hkv, 64, hd), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((n_pages, hkv), device="cuda") for _ in range(2))
    table = torch.zeros((1, 16_000_001), dtype=torch.int32, device="cuda")
    table[0, 16_000_000] = n_pages - 1
    lens = torch.tensor([pos + 1], dtype=torch.int32, device="cuda")
    kv = lr.Kv8Pages(kc, vc, ks, vs, table, lens, torch.float32)
    x, xr = rounded(rng.standard_normal((1, hkv, hd)), "f32")
    inv = inv_freq(128)
    q_out, ws = torch.empty_like(x), lr.workspace(256)
    cu = None if single else torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    lr.lr_kv8_append(kv, x, x, ws, cu_tokens=cu, rope=lr.Rope(torch.from_numpy(inv).cuda(), 128), q=x, q_out=q_out)
    assert lr.lr_get_device_error(ws) == 0
    # the angle in whole turns with exact integers: inv is a ratio of integers
    turned = np.zeros_like(xr[0])
    for j in range(64):
        num, den = float(inv[j]).as_integer_ratio()
        from fractions import Fraction
        two_pi = Fraction(6283185307179586476925286766559, 10 ** 30)
        a = Fraction(num * pos, den)
        a = float(a - two_pi * (a // two_pi))
        x0, x1 = xr[0][:, j], xr[0][:, 64 + j]
        turned[:, j], turned[:, 64 + j] = x0 * np.cos(a) - x1 * np.sin(a), x1 * np.cos(a) + x0 * np.sin(a)
    # the fraction of a turn is rounded at 2^-53: times 2^30 tokens under 1e-6 radians
    assert np.abs(q_out.double().cpu().numpy()[0] - turned).max() <= (1e-6 + 2.0 ** -21) * 2 * np.abs(xr).max()
    got = kc[n_pages - 1].cpu().numpy()
    s = ks[n_pages - 1].cpu().numpy().astype(np.float64)
    y = orc.E4M3[got[:, 10]] * s[:, None]
    assert (np.abs(y - turned) <= 2.0 ** -4 * np.abs(turned) + s[:, None] * 2.0 ** -10 + 1e-5).all()
    assert int((kc != 0).any(dim=3).sum()) == hkv  # one row of each head, nowhere else


def test_append_bad_data_is_reported_and_skipped():
    rng = np.random.default_rng(6)
    hkv, hd = 2, 128
    pool = Pool(rng, [10, 70, 64, 5], hkv, hd, room=[64, 128, 128, 64])
    good = pool.table.copy()
    k, kr = rounded(rng.standard_normal((4, hkv, hd)), "bf16")
    for single in (True, False):
        for what in ("page_high", "page_negative", "len_negative", "len_long", "len_short"):
            pool.table[:] = good
            lens, bad = [11, 71, 65, 6], 1
            if what == "page_high":
                pool.table[1, 1] = pool.kc.shape[0]
            elif what == "page_negative":
                pool.table[1, 1] = -1
            elif what == "len_negative":
                lens[1] = -3
            elif what == "len_long":
                lens[1] = 64 * pool.width + 1
            elif single:
                continue  # lens 0 is an empty slot
            else:
                lens[1] = 0
            pool.lens[:] = lens
            pool.upload()
            keep = [x.copy() for x in (pool.kc, pool.vc, pool.ks, pool.vs)]
            q_out, err = run_append(pool, k, k, k, None if single else [0, 1, 2, 3, 4], 128, False)
            assert err == (lr.LR_DEVERR_PAGE if what.startswith("page") else lr.LR_DEVERR_LEN), what
            if not what.startswith("page"):
                assert (q_out[bad] == 7.0).all()
            cu = np.array([0, 1, 1, 2, 3])
            rows = [0, 2, 3]
            pool.lens[bad] = 0
            check_append(pool, keep, kr[rows], kr[rows], kr[rows], q_out[rows], cu, 128, False)
    # token ranges that descend or leave the tensor
    pool.table[:] = good
    for cu in ([0, 1, 0, 3, 4], [0, 1, 2, 3, 5], [-1, 1, 2, 3, 4]):
        pool.lens[:] = [11, 71, 65, 6]
        pool.upload()
        assert run_append(pool, k, k, k, cu, 128, False)[1] & lr.LR_DEVERR_LEN


def test_append_refuses_overlapping_tokens():
    """One row for every token (a broadcast view) is not a cache's input."""
    pool = Pool(np.random.default_rng(8), [3], 2, 128)
    k = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda").expand(3, -1, -1)
    v = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        lr.lr_kv8_append(pool.kv, k, v, lr.workspace(256), cu_tokens=cu)


def test_append_two_calls_at_once():
    """Two streams append to pages of their own in one pool at the same time."""
    rng = np.random.default_rng(9)
    new = [150, 90]
    pool = Pool(rng, [0, 0], 2, 128, room=new)
    before = pool.arrays()
    k, kr = rounded(rng.standard_normal((sum(new), 2, 128)), "bf16")
    v, vr = rounded(rng.standard_normal((sum(new), 2, 128)), "bf16")
    pool.set_lens(new)
    rope = lr.Rope(torch.from_numpy(inv_freq(128)).cuda(), 128)
    kvs = [lr.Kv8Pages(*pool.dev[:4], pool.dev[4][b:b + 1].clone(), torch.tensor([new[b]], dtype=torch.int32, device="cuda"),
                       torch.bfloat16) for b in range(2)]
    parts = [slice(0, new[0]), slice(new[0], None)]
    cus = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in new]
    streams, ws = [torch.cuda.Stream() for _ in range(2)], [lr.workspace(256) for _ in range(2)]
    torch.cuda.synchronize()
    for b in range(2):
        lr.lr_kv8_append(kvs[b], k[parts[b]], v[parts[b]], ws[b], cu_tokens=cus[b], rope=rope, stream=streams[b])
    torch.cuda.synchronize()
    assert all(lr.lr_get_device_error(w) == 0 for w in ws)
    check_append(pool, before, kr, vr, None, None, [0, new[0], sum(new)], 128, False)


def test_append_empty_slots_and_nothing():
    rng = np.random.default_rng(7)
    pool = Pool(rng, [0, 5, 0], 1, 128, room=[64, 64, 64])
    pool.set_lens([0, 6, 0])
    k, kr = rounded(rng.standard_normal((3, 1, 128)), "bf16")
    keep = [x.copy() for x in (pool.kc, pool.vc, pool.ks, pool.vs)]
    q_out, err = run_append(pool, k, k, k, None, 128, False)
    assert err == 0 and (q_out[0] == 7.0).all() and (q_out[2] == 7.0).all()
    check_append(pool, keep, kr[1:2], kr[1:2], kr[1:2], q_out[1:2], np.array([0, 0, 1, 1]), 128, False)
    before = pool.arrays()
    none = k[:0]
    _, err = run_append(pool, none, none, none, [0, 0, 0, 0], 128, False)
    assert err == 0
    for x, y in zip(before, pool.arrays()):
        np.testing.assert_array_equal(x, y)


# ------------------------------------------------------------------------------- attention

ATTN = {
    "one_token": dict(lens=[1], hkv=1, G=1),
    "page_ends": dict(lens=[63, 64, 65, 127, 128, 129, 0, 2], hkv=2, G=4),
    "gqa8": dict(lens=[700, 0, 5], hkv=2, G=8),
    "gqa5": dict(lens=[300, 129], hkv=1, G=5),
    "gqa3": dict(lens=[200, 64], hkv=2, G=3),
    "mha": dict(lens=[260, 31], hkv=4, G=1),
    "gqa2": dict(lens=[1000], hkv=3, G=2),
    "gqa6_7": dict(lens=[150], hkv=2, G=7),
    "long_split": dict(lens=[4000], hkv=1, G=4),
    "window": dict(lens=[1000, 64, 100, 0, 129, 1], hkv=2, G=4, window=65),
    "window_one": dict(lens=[130, 64], hkv=1, G=4, window=1),
    "joined": dict(lens=[300, 0, 70, 1], hkv=2, G=4, prev=True),
    "joined_gqa8_window": dict(lens=[300, 0, 70], hkv=2, G=8, prev=True, window=100),
    "scale": dict(lens=[100], hkv=1, G=4, scale=0.31),
    "many": dict(lens=[(37 * i) % 200 for i in range(150)], hkv=2, G=2),
    "f32": dict(lens=[1000, 0, 65], hkv=2, G=2, hd=64, dtype="f32"),
    "f32_hd256": dict(lens=[150], hkv=1, G=8, hd=256, dtype="f32"),
    "f32_hd40_joined": dict(lens=[150, 0], hkv=2, G=3, hd=40, dtype="f32", prev=True, window=70),
    "bf16_hd64": dict(lens=[500, 3], hkv=2, G=4, hd=64),
    "bf16_hd8": dict(lens=[100], hkv=1, G=2, hd=8),
    "f32_hd96_gqa8": dict(lens=[700, 64, 0, 33], hkv=2, G=8, hd=96, dtype="f32"),
    "f32_hd120_window": dict(lens=[500, 31], hkv=1, G=5, hd=120, dtype="f32", window=77),
    "f32_hd128_split": dict(lens=[6000], hkv=1, G=4, hd=128, dtype="f32"),
    "f32_hd200_joined": dict(lens=[130, 0, 1], hkv=2, G=7, hd=200, dtype="f32", prev=True),
    "bf16_hd96_joined": dict(lens=[260, 17], hkv=1, G=8, hd=96, prev=True, window=100),
    "bf16_hd72": dict(lens=[129, 64, 63], hkv=2, G=1, hd=72),
    "more_sequences_than_threads": dict(lens=[(7 * i) % 5 for i in range(700)], hkv=1, G=2),
    "more_sequences_than_threads_f32": dict(lens=[(7 * i) % 5 for i in range(300)], hkv=1, G=2, hd=64, dtype="f32"),
    "cluster_of_8_rests": dict(lens=[1100, 130, 1, 0, 900], hkv=2, G=4),
    "cluster_of_8_window": dict(lens=[4000, 2500], hkv=2, G=8, window=900, prev=True),
    "cluster_of_2": dict(lens=[1000 - 61 * i for i in range(16)], hkv=8, G=4),
    "cluster_of_1": dict(lens=[1 + 3 * i for i in range(150)], hkv=1, G=5, prev=True),
    "cluster_of_8_f32": dict(lens=[2000, 0, 257], hkv=1, G=8, hd=256, dtype="f32", prev=True),
    "cluster_of_4_bf16_hd72": dict(lens=[600, 64, 1, 0] * 4, hkv=4, G=3, hd=72, window=300),
    "short_segments_gqa8": dict(lens=[1 + i % 130 for i in range(90)], hkv=8, G=8),
    "bf16_hd256": dict(lens=[100, 64], hkv=2, G=4, hd=256),
}


@pytest.mark.parametrize("width", [None, 600], ids=["", "room_for_more"])
@pytest.mark.parametrize("name", list(ATTN))
def test_attention(name, width):
    """`width`: page table entries of a sequence. With no more than the tokens need most of these cases are small
    calls, which a cluster answers by itself; with room for 38400 tokens they are not."""
    c = ATTN[name]
    hd, dtype, win = c.get("hd", 128), c.get("dtype", "bf16"), c.get("window", 0)
    rng = np.random.default_rng(len(name))
    pool = Pool(rng, c["lens"], c["hkv"], hd, dtype, width=width)
    B, hq = len(c["lens"]), c["hkv"] * c["G"]
    q, qr = rounded(rng.standard_normal((B, hq, hd)) * 1.5, dtype)
    prev = prev_ref = None
    if c.get("prev"):
        po, por = rounded(rng.standard_normal((B, hq, hd)) * 0.3, dtype)
        pl = (rng.standard_normal((B, hq)) * 2 + 3).astype(np.float32)
        pl[0, 0] = -np.inf  # an empty earlier part; what its output holds is not used
        po[0, 0] = float("nan")
        por[0, 0] = np.nan
        prev, prev_ref = (po, torch.from_numpy(pl).cuda()), (por, pl.astype(np.float64))
    scale = c.get("scale", 1 / np.sqrt(hd))
    o, lse, err = attend(pool, q, win, c.get("scale", 0.0), prev)
    assert err == 0
    ref = orc.decode(qr, pool.kc, pool.vc, pool.ks, pool.vs, pool.table, pool.lens, scale, win,
                     *(prev_ref or (None, None)))
    check_attention((o, lse), ref, pool, qr, scale, max(c["lens"]))
    again = attend(pool, q, win, c.get("scale", 0.0), prev)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])  # whichever CTA joins the pieces
    if prev is not None:  # in place
        o2, lse2, _ = attend(pool, q, win, c.get("scale", 0.0), (prev[0].clone(), prev[1].clone()), in_place=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_attention_scales_far_apart():
    """Pages whose scales differ by 2^20 and more: what a page adds does not drown in another's scale. Values of
    all-zero pages, and a page that holds nearly all the weight at the smallest scale."""
    rng = np.random.default_rng(11)
    pool = Pool(rng, [64 * 6 + 9], 1, 128)
    for i, e in enumerate([-24, 3, -10, -24, 8, -2, 0]):
        pool.vs[pool.table[0, i]] = 2.0 ** e
    pool.vc[pool.table[0, 3], :, :] = 0
    pool.upload()
    q, qr = rounded(rng.standard_normal((1, 4, 128)) * 2, "bf16")
    o, lse, _ = attend(pool, q)
    ref = orc.decode(qr, pool.kc, pool.vc, pool.ks, pool.vs, pool.table, pool.lens, 128 ** -0.5)
    check_attention((o, lse), ref, pool, qr, 128 ** -0.5, 400)


@pytest.mark.parametrize("hd,dtype", [(128, "bf16"), (64, "f32"), (256, "bf16")])
def test_attention_scales_of_any_size(hd, dtype):
    """Scales that are no powers of two and far apart, 1e-7 to 1e30, in any order, keys and values."""
    rng = np.random.default_rng(16)
    pool = Pool(rng, [64 * 9, 64 * 3 + 5], 2, hd, dtype)
    for b in range(2):
        for i in range(-(-int(pool.lens[b]) // 64)):
            page = pool.table[b, i]
            pool.vs[page] = rng.choice([1e-7, 3e-3, 0.7, 19.0, 1e8, 1e30], 2)
            pool.ks[page] = rng.uniform(0.001, 0.02, 2)
    pool.upload()
    q, qr = rounded(rng.standard_normal((2, 8, hd)), dtype)
    o, lse, err = attend(pool, q)
    assert err == 0
    scale = hd ** -0.5
    ref = orc.decode(qr, pool.kc, pool.vc, pool.ks, pool.vs, pool.table, pool.lens, scale)
    check_attention((o, lse), ref, pool, qr, scale, 600)


def test_attention_result_does_not_depend_on_the_rest_of_the_batch():
    """Room in the page table, unused pages and a workspace full of other bytes change nothing."""
    rng = np.random.default_rng(17)
    pool = Pool(rng, [500, 40], 2, 128)
    q, _ = rounded(rng.standard_normal((2, 8, 128)), "bf16")
    o, lse, _ = attend(pool, q)
    wide = torch.full((2, 4000), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, :pool.width] = pool.dev[4]
    kv = lr.Kv8Pages(*pool.dev[:4], wide, pool.dev[5], torch.bfloat16)
    for fill in (0, 255):
        ws = torch.full((lr.lr_kv8_attn_workspace_bytes(kv, 8),), fill, dtype=torch.uint8, device="cuda")
        o2, lse2 = torch.full_like(o, 3.0), torch.full_like(lse, 3.0)
        lr.lr_decode_attn_kv8(kv, 8, q, o2, ws, lse=lse2)
        assert lr.lr_get_device_error(ws) == 0
        # another width divides the work into other pieces: equal to the sums' rounding
        torch.testing.assert_close(o2.float(), o.float(), rtol=2.0 ** -7, atol=2.0 ** -9)
        torch.testing.assert_close(lse2, lse, rtol=1e-6, atol=1e-5)


@pytest.mark.parametrize("hd,dtype", [(128, "bf16"), (64, "f32")])
def test_attention_over_nothing(hd, dtype):
    """No sequence has a token: 0 and -inf, or the earlier part as it is."""
    pool = Pool(np.random.default_rng(19), [0, 0, 0], 2, hd, dtype)
    q = torch.ones((3, 8, hd), dtype=DT[dtype], device="cuda")
    o, lse, err = attend(pool, q)
    assert err == 0 and (o == 0).all() and torch.isneginf(lse).all()
    prev = (torch.randn_like(q), torch.randn((3, 8), device="cuda"))
    prev[1][1] = float("-inf")
    o, lse, err = attend(pool, q, prev=prev)
    assert err == 0 and (o[1] == 0).all() and torch.equal(o[[0, 2]], prev[0][[0, 2]])
    torch.testing.assert_close(lse, prev[1], rtol=2.0 ** -22, atol=2.0 ** -22)


def test_attention_infinite_query():
    """A head with an infinite query number gives NaN, the other heads of the KV head are as without it."""
    rng = np.random.default_rng(18)
    for hd, dtype in ((128, "bf16"), (64, "f32")):
        pool = Pool(rng, [200, 30], 1, hd, dtype)
        q, _ = rounded(rng.standard_normal((2, 4, hd)), dtype)
        o, lse, _ = attend(pool, q)
        bad = q.clone()
        bad[0, 2, 5] = float("inf")
        o2, lse2, err = attend(pool, bad)
        assert err == 0 and torch.isnan(o2[0, 2]).all() and torch.isnan(lse2[0, 2])
        keep = torch.ones(2, 4, dtype=torch.bool, device="cuda")
        keep[0, 2] = False
        assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[keep], lse[keep])


def test_attention_extreme_scores():
    """Scores of hundreds: one token takes all the weight, and the earlier part may or may not."""
    rng = np.random.default_rng(12)
    pool = Pool(rng, [500], 2, 128)
    q, qr = rounded(rng.standard_normal((1, 8, 128)) * 300, "bf16")
    for lp in (-1e4, 0.0, 1e4):
        po, por = rounded(rng.standard_normal((1, 8, 128)), "bf16")
        pl = np.full((1, 8), lp, np.float32)
        o, lse, _ = attend(pool, q, prev=(po, torch.from_numpy(pl).cuda()))
        ref = orc.decode(qr, pool.kc, pool.vc, pool.ks, pool.vs, pool.table, pool.lens, 128 ** -0.5,
                         0, por, pl.astype(np.float64))
        check_attention((o, lse), ref, pool, qr, 128 ** -0.5, 500)


def test_attention_nan_stays_in_its_sequence():
    rng = np.random.default_rng(13)
    pool = Pool(rng, [100, 100, 100], 2, 128)
    pool.kc[pool.table[1, 0], 0, 7, 3] = 0x7F  # a NaN key of (sequence 1, head 0)
    pool.vc[pool.table[2, 1], 1, 3, 9] = 0xFF  # a NaN value of (sequence 2, head 1), column 9
    pool.upload()
    q, qr = rounded(rng.standard_normal((3, 8, 128)), "bf16")
    o, lse, err = attend(pool, q)
    o, lse = o.float().cpu().numpy(), lse.cpu().numpy()
    assert err == 0
    bad = np.isnan(o)
    assert bad[1, :4].all() and np.isnan(lse[1, :4]).all()
    assert bad[2, 4:, 9].all() and bad.sum() == 4 * 128 + 4 and np.isfinite(lse[2]).all()


@pytest.mark.parametrize("width", [None, 600], ids=["", "room_for_more"])
def test_attention_bad_data_is_reported_and_left_out(width):
    rng = np.random.default_rng(14)
    for page in (10 ** 6, -1):
        pool = Pool(rng, [300, 200], 2, 128, width=width)
        pool.table[0, 2] = page
        pool.upload()
        q, qr = rounded(rng.standard_normal((2, 8, 128)), "bf16")
        o, lse, err = attend(pool, q)
        assert err == lr.LR_DEVERR_PAGE
        ref = orc.decode(qr, pool.kc, pool.vc, pool.ks, pool.vs, pool.table, pool.lens, 128 ** -0.5)
        check_attention((o, lse), ref, pool, qr, 128 ** -0.5, 300)
    pool = Pool(rng, [256, 200], 2, 128, width=width)
    pool.set_lens([1000, -4] if width is None else [64 * width + 1, -4])
    if width is not None:  # clipped to the table's room, of which four pages are there
        assert attend(pool, q)[2] == lr.LR_DEVERR_LEN | lr.LR_DEVERR_PAGE
        return
    o, lse, err = attend(pool, q)
    assert err == lr.LR_DEVERR_LEN
    pool.lens[:] = [256, 0]
    ref = orc.decode(qr, pool.kc, pool.vc, pool.ks, pool.vs, pool.table, pool.lens, 128 ** -0.5)
    check_attention((o, lse), ref, pool, qr, 128 ** -0.5, 256)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [100, 300])
def test_attention_one_bad_page_of_a_large_batch(B, dtype):
    """Reported and left out wherever it is attended, and only there."""
    rng = np.random.default_rng(23)
    lens = rng.integers(0, 257, B)
    lens[[0, B // 2, B - 1]] = 256, 200, 130
    pool = Pool(rng, lens, 1, 128, dtype, width=4)
    q, qr = rounded(rng.standard_normal((B, 4, 128)), dtype)
    table = pool.table.copy()
    for b, page, window, expect in ((0, 3, 0, True), (B // 2, 0, 0, True), (B // 2, 3, 0, True), (B - 1, 2, 0, True),
                                    (B - 1, 0, 130, True), (B - 1, 0, 67, True), (B - 1, 0, 66, False), (B - 1, 3, 0, False)):
        pool.table[:] = table
        pool.table[b, page] = pool.kc.shape[0]
        pool.upload()
        o, lse, err = attend(pool, q, window=window)
        assert err == (lr.LR_DEVERR_PAGE if expect else 0), (b, page, window)
        ref = orc.decode(qr, pool.kc, pool.vc, pool.ks, pool.vs, pool.table, pool.lens, 128 ** -0.5, window=window)
        check_attention((o, lse), ref, pool, qr, 128 ** -0.5, 256)
    pool.table[:] = table
    pool.upload()
    for b in (0, 37, B - 1):
        lens = pool.lens.copy()
        pool.set_lens(np.where(np.arange(B) == b, -1, lens))
        assert attend(pool, q)[2] == lr.LR_DEVERR_LEN
        pool.set_lens(lens)
    assert attend(pool, q)[2] == 0


def test_attention_shared_pages_strided_pool_other_stream():
    """Two sequences over the same pages give the same; K and V side by side in one pool; a side stream."""
    rng = np.random.default_rng(15)
    pool = Pool(rng, [500, 300], 2, 128)
    pool.table[1] = pool.table[0]
    pool.lens[1] = 500
    both = torch.zeros((pool.kc.shape[0], 2, 2, 64, 128), dtype=torch.uint8, device="cuda")
    both[:, 0].copy_(torch.from_numpy(pool.kc)), both[:, 1].copy_(torch.from_numpy(pool.vc))
    pool.upload()
    pool.dev[0], pool.dev[1] = both[:, 0], both[:, 1]
    pool.kv = lr.Kv8Pages(*pool.dev, torch.bfloat16)
    q, qr = rounded(rng.standard_normal((1, 8, 128)), "bf16")
    q = q.expand(2, -1, -1).contiguous()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        o, lse, err = attend(pool, q, stream=st)
    assert err == 0 and torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])
    ref = orc.decode(np.repeat(qr, 2, 0), pool.kc, pool.vc, pool.ks, pool.vs, pool.table, pool.lens, 128 ** -0.5)
    check_attention((o, lse), ref, pool, np.repeat(qr, 2, 0), 128 ** -0.5, 500)


def test_attention_long_context_against_torch():
    """262K tokens (codes past 2^32 bits of offset, every CTA on a piece): torch in fp64 as the reference."""
    g = torch.Generator(device="cuda").manual_seed(1)
    hkv, hd, T = 2, 128, 262144 + 37
    n = -(-T // 64)
    kc, vc = ((torch.randn((n, hkv, 64, hd), generator=g, device="cuda") * 40).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((n, hkv), 2.0 ** -5, device="cuda") for _ in range(2))
    table = torch.randperm(n, generator=g, device="cuda").to(torch.int32)[None]
    kv = lr.Kv8Pages(kc.view(torch.uint8), vc.view(torch.uint8), ks, vs, table,
                     torch.tensor([T], dtype=torch.int32, device="cuda"), torch.bfloat16)
    q = torch.randn((1, 8, hd), generator=g, device="cuda").to(torch.bfloat16)
    o, lse = torch.empty_like(q), torch.empty((1, 8), device="cuda")
    ws = lr.workspace(lr.lr_kv8_attn_workspace_bytes(kv, 8))
    lr.lr_decode_attn_kv8(kv, 8, q, o, ws, lse=lse)
    assert lr.lr_get_device_error(ws) == 0
    for h in range(hkv):
        K, V = ((c[table[0].long(), h].double() * 2.0 ** -5).reshape(-1, hd)[:T] for c in (kc, vc))
        s = q[0, 4 * h:4 * h + 4].double() @ K.T / hd ** 0.5
        w = torch.softmax(s, 1)
        ref, mass = w @ V, w @ V.abs()
        # weights stored to 2^-12 with random signs over 10^5 tokens, and the output's own rounding
        assert ((o[0, 4 * h:4 * h + 4].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -11 * mass).all()
        assert (lse[0, 4 * h:4 * h + 4].double() - torch.logsumexp(s, 1)).abs().max() < 1e-4


# ------------------------------------------------------------------------------- together

def test_decode_loop_in_a_graph():
    """Seventy decode steps (append, then attend) replayed from one captured graph, lengths and tokens
    changing on the device, against the oracle run token by token."""
    rng = np.random.default_rng(20)
    hkv, G, hd, B, steps = 2, 4, 128, 3, 70
    start = [0, 60, 131]
    pool = Pool(rng, start, hkv, hd, room=[n + steps for n in start])
    hq = hkv * G
    tokens = rng.standard_normal((steps, B, hq + 2 * hkv, hd)) * (1 + np.arange(steps) / 10)[:, None, None, None]
    x_all, xr = rounded(tokens, "bf16")
    x = x_all[0].clone()
    rope = lr.Rope(torch.from_numpy(inv_freq(hd)).cuda(), hd)
    q_out = torch.empty((B, hq, hd), dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(q_out), torch.empty((B, hq), device="cuda")
    ws_a, ws = lr.workspace(256), lr.workspace(lr.lr_kv8_attn_workspace_bytes(pool.kv, hq))
    lens = pool.dev[5]

    def step():
        lens.add_(1)
        lr.lr_kv8_append(pool.kv, x[:, hq:hq + hkv], x[:, hq + hkv:], ws_a, rope=rope, q=x[:, :hq], q_out=q_out)
        lr.lr_decode_attn_kv8(pool.kv, hq, q_out, o, ws, lse=lse)

    keep = [t.clone() for t in pool.dev[:4]]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()  # warm-up
    torch.cuda.current_stream().wait_stream(st)
    for t, u in zip(pool.dev[:4], keep):
        t.copy_(u)
    lens.copy_(torch.tensor(start, dtype=torch.int32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = [a.copy() for a in (pool.kc, pool.vc, pool.ks, pool.vs)]
    inv = inv_freq(hd)
    for i in range(steps):
        x.copy_(x_all[i])
        graph.replay()
        now = np.array(start) + i + 1
        orc.append(*want, pool.table, now, range(B + 1), xr[i][:, hq:hq + hkv], xr[i][:, hq + hkv:], inv, hd, False)
        if i % 23 == 0 or i == steps - 1:
            got = pool.arrays()
            np.testing.assert_array_equal(got[1], want[1])
            np.testing.assert_array_equal(got[3], want[3])
            qr = q_out.double().cpu().numpy()
            pool.kc, pool.vc, pool.ks, pool.vs = got
            ref = orc.decode(qr, *got, pool.table, now, hd ** -0.5)
            check_attention((o, lse), ref, pool, qr, hd ** -0.5, int(now.max()))
    assert lr.lr_get_device_error(ws) == 0 and lr.lr_get_device_error(ws_a) == 0


@pytest.mark.parametrize("path", ["pair", "general"])
def test_packed_context_and_recent_tokens_in_one_softmax(path, monkeypatch):
    """lr_decode_attn_lse over the packed context, joined with the 8-bit pages of the tokens since."""
    from oracle import lowram_oracle as lorc
    monkeypatch.setenv("LOWRAM_DECODE_PATH", path)
    p = H.packed_problem(H.small(T=500, batch=2))
    w = p.w
    rng = np.random.default_rng(21)
    q_st, q_ref = H.queries(p, 0)
    shape = H.shape_of(w)
    o, lse = torch.empty_like(q_st), torch.empty(q_st.shape[:2], device="cuda")
    ws = lr.workspace(lr.lr_decode_workspace_bytes(shape, w.n_q_heads, 0))
    lr.lr_decode_attn_lse(shape, 0, w.n_q_heads, q_st, p.st["A"], p.st["Bt"], H.gpu_predictor(p), p.st["idx"],
                          p.st["val"], p.st["ptr"], p.k, None, 0, 0.0, o, lse, ws)
    plain, _ = H.gpu_decode(p, 0, q_st)
    np.testing.assert_array_equal(o.double().cpu().numpy(), plain)  # the same call but for lse
    pool = Pool(rng, [130, 17], w.n_kv_heads, w.head_dim, mixed=False)
    o2, lse2, err = attend(pool, q_st, prev=(o, lse))
    assert err == 0
    # reference: the pages' tokens as the exact tail of the oracle's own joint softmax
    for b, n in enumerate(pool.lens):
        t = np.arange(n)
        pg = pool.table[b, t // 64]
        K = (orc.E4M3[pool.kc[pg, :, t % 64]] * pool.ks[pg][..., None]).transpose(1, 0, 2)
        V = (orc.E4M3[pool.vc[pg, :, t % 64]] * pool.vs[pg][..., None]).transpose(1, 0, 2)
        r = p.ref
        ref = lorc.decode_sequence(q_ref[b], r["A"][b], r["Bt"][b], r["W_lin"][b], r["W1"][b], r["b1"][b], r["W2"][b],
                                   None, 0, r["idx"][b], r["val"][b], None, lorc.default_scale(w.head_dim, 0.0),
                                   w.n_kv_heads, w.head_dim, K, V)
        H.assert_attention_close(o2[b].double().cpu().numpy(), ref)
    # an empty context: -inf, and joining leaves it out
    empty = H.shape_of(w, T=0)
    lr.lr_decode_attn_lse(empty, 0, w.n_q_heads, q_st, p.st["A"], p.st["Bt"], H.gpu_predictor(p), None, None, None, 0,
                          None, 0, 0.0, o, lse, lr.workspace(lr.lr_decode_workspace_bytes(empty, w.n_q_heads, 0)))
    assert torch.isneginf(lse).all() and (o == 0).all()
    a, b_ = attend(pool, q_st, prev=(o, lse)), attend(pool, q_st)
    assert torch.equal(a[0], b_[0]) and torch.equal(a[1], b_[1])


def test_lse_of_the_packed_context():
    """Against the keys the cache stands for: log of the sum of exponentials of the rebuilt keys' scores. The
    tensor-core scores are off by 2^-15 of |q||k| scale at most (bf16 hi + lo query parts over a bf16 A)."""
    p = H.packed_problem(H.small(T=300))
    w = p.w
    q_st, q_ref = H.queries(p, 1)
    shape = H.shape_of(w)
    o, lse = torch.empty_like(q_st), torch.empty(q_st.shape[:2], device="cuda")
    ws = lr.workspace(lr.lr_decode_workspace_bytes(shape, w.n_q_heads, 0))
    lr.lr_decode_attn_lse(shape, 1, w.n_q_heads, q_st, p.st["A"], p.st["Bt"], H.gpu_predictor(p), p.st["idx"],
                          p.st["val"], p.st["ptr"], p.k, None, 0, 0.0, o, lse, ws)
    A, Bt, hd = p.ref["A"][0], p.ref["Bt"][0], w.head_dim
    for h in range(w.n_kv_heads):
        row = (1 * w.n_kv_heads + h) * hd
        Qh = q_ref[0][h * w.q_per_kv:(h + 1) * w.q_per_kv] @ Bt[row:row + hd]      # [G, r]
        s = Qh @ A.T * hd ** -0.5
        want = s.max(1) + np.log(np.exp(s - s.max(1, keepdims=True)).sum(1))
        got = lse[0, h * w.q_per_kv:(h + 1) * w.q_per_kv].double().cpu().numpy()
        lim = 2.0 ** -15 * (np.abs(Qh) @ np.abs(A).T).max(1) * hd ** -0.5 + 1e-4
        assert (np.abs(got - want) <= lim).all()
