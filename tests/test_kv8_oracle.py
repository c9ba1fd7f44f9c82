"""CPU pins of the 8-bit paged cache's oracle: its codes are torch's e4m3 codes, its scales are the smallest
powers of two, appending token by token equals the cache's definition, attention over one page is
the softmax written out."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as orc


def test_codes_are_e4m3():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(np.isnan(every), np.isnan(orc.E4M3))
    ok = ~np.isnan(every)
    np.testing.assert_array_equal(every[ok], orc.E4M3[ok])
    rng = np.random.default_rng(0)
    grid = orc.E4M3[:0x7F]
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.uniform(-4, 2, 20000), (grid[1:] + grid[:-1]) / 2,
                        -(grid[1:] + grid[:-1]) / 2, grid, [0.0, -0.0, 448.0, -448.0]]).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(orc.e4m3_codes(x), want)
    np.testing.assert_array_equal(orc.e4m3_codes([np.nan, np.inf, -np.inf, 1e9]), [0x7F, 0x7F, 0x7F, 0x7E])


@pytest.mark.parametrize("amax,want", [(0.0, 2.0 ** -24), (1e-12, 2.0 ** -24), (448.0, 1.0), (448.0001, 2.0),
                                       (224.0, 0.5), (7.0, 2.0 ** -6), (7.0000005, 2.0 ** -5), (3.4e38, 2.0 ** 120)])
def test_fresh_scale(amax, want):
    assert orc.fresh_scale(amax) == want


def test_append_token_by_token_and_attention():
    rng = np.random.default_rng(1)
    hkv, hd, T = 2, 16, 70
    k, v = rng.standard_normal((T, hkv, hd)), rng.standard_normal((T, hkv, hd)) * np.linspace(0.1, 30, T)[:, None, None]
    table = np.array([[1, 0]], np.int32)
    st = [np.full((2, hkv, 64, hd), 0x7F, np.uint8) for _ in range(2)] + [np.full((2, hkv), np.nan, np.float32) for _ in range(2)]
    inv = 1.0 / 100.0 ** (np.arange(8) / 8)
    kr = np.zeros_like(k)
    for t in range(T):
        kr[t] = orc.append(*st, table, [t + 1], [0, 1], k[t:t + 1], v[t:t + 1], inv, 16, False)[0][0]
    # a number is off by half a step of its page's final scale, once per change of scale at most
    for codes, scale, x in ((st[0], st[2], kr), (st[1], st[3], v)):
        for t in range(T):
            page = table[0, t // 64]
            got = orc.E4M3[codes[page, :, t % 64]] * scale[page][:, None]
            assert (np.abs(got - x[t]) <= 2.0 ** -4 * np.abs(x[t]) + scale[page][:, None] * 2.0 ** -9).all()
    q = rng.standard_normal((1, 4, hd))
    o, lse, mass = orc.decode(q, *st, table, [T], 0.25)
    K = np.stack([orc.E4M3[st[0][table[0, t // 64], :, t % 64]] * st[2][table[0, t // 64]][:, None] for t in range(T)])
    V = np.stack([orc.E4M3[st[1][table[0, t // 64], :, t % 64]] * st[3][table[0, t // 64]][:, None] for t in range(T)])
    for g in range(4):
        s = 0.25 * K[:, g // 2] @ q[0, g]
        p = np.exp(s) / np.exp(s).sum()
        np.testing.assert_allclose(o[0, g], p @ V[:, g // 2], rtol=1e-12, atol=1e-14)
        np.testing.assert_allclose(lse[0, g], np.log(np.exp(s).sum()), rtol=1e-12)
    # joined parts equal the whole
    a = orc.decode(q, *st, table, [40], 0.25)
    whole = orc.decode(q, *st, table, [T], 0.25, window=T - 40, o_prev=a[0], lse_prev=a[1])
    np.testing.assert_allclose(whole[0], o, rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(whole[1], lse, rtol=1e-12)


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(2)
    inv = 1.0 / 10000.0 ** (np.arange(4) / 4)
    for inter in (False, True):
        x, y = rng.standard_normal((1, 12)), rng.standard_normal((1, 12))
        a = orc.rotate(x, 5, inv, 8, inter)
        np.testing.assert_allclose(np.linalg.norm(a), np.linalg.norm(x), rtol=1e-13)
        np.testing.assert_array_equal(a[:, 8:], x[:, 8:])
        d1 = (orc.rotate(x, 9, inv, 8, inter) * orc.rotate(y, 4, inv, 8, inter)).sum()
        d2 = (orc.rotate(x, 1009, inv, 8, inter) * orc.rotate(y, 1004, inv, 8, inter)).sum()
        np.testing.assert_allclose(d1, d2, rtol=1e-10)
