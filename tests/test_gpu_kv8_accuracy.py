"""The 8-bit cache's attention holds what it promises of its queries and weights: limits that a missing term of
either would break (tests/kv8_accuracy.py; the CPU tests show that it would)."""
import numpy as np
import pytest
import torch

from oracle import kv8_oracle as orc

import kv8_accuracy as acc
from kv8_helpers import Pool, attend, rounded

pytestmark = pytest.mark.gpu

ONE = 0x38  # the code of 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from long_context_decode_lr_b200 import build, lowram as lr
    build.build()
    lr.library()


def _pool(lens, hd, dtype, width=None):
    """Scales 1, keys and values 0."""
    pool = Pool(np.random.default_rng(0), lens, 1, hd, dtype, width=width)
    pool.kc[:], pool.vc[:], pool.ks[:], pool.vs[:] = 0, 0, 1.0, 1.0
    return pool


def _first(pool, t=0):
    return pool.table[:, 0], 0, t  # row t of every sequence


@pytest.mark.parametrize("width", [None, 600], ids=["", "room_for_more"])
@pytest.mark.parametrize("hd,dtype", [(64, "f32"), (128, "f32"), (256, "f32"), (128, "bf16"), (256, "bf16")])
def test_one_key(hd, dtype, width):
    """Every dim of the head once: the log-sum-exp of one token is its score."""
    rng = np.random.default_rng(hd)
    pool = _pool([1] * hd, hd, dtype, width)
    pages, h, t = _first(pool)
    pool.kc[pages, h, t, np.arange(hd)] = ONE
    pool.upload()
    q, qr = rounded(np.clip(np.abs(rng.standard_normal((hd, 8, hd))), 0.01, None), dtype)
    _, lse, err = attend(pool, q, scale=0.125)
    score = 0.125 * qr[np.arange(hd), :, np.arange(hd)]
    assert err == 0
    assert (np.abs(lse.double().cpu().numpy() - score) <= acc.score_limit(score)).all()


def _two_tokens(hd, dtype, lowest, width, n=256):
    """Sequences of two tokens, scores 0 and s: (pool, q, s [n, 8])."""
    rng = np.random.default_rng(hd)
    pool = _pool([2] * n, hd, dtype, width)
    pages, h, t = _first(pool, 1)
    pool.kc[pages, h, t, 5] = ONE
    q = np.zeros((n, 8, hd))
    q[:, :, 5] = rng.uniform(8 * lowest, -0.01, (n, 8))
    q, qr = rounded(q, dtype)
    return pool, q, 0.125 * qr[:, :, 5]


@pytest.mark.parametrize("width", [None, 600], ids=["", "room_for_more"])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_two_tokens_fp32(hd, width):
    pool, q, s = _two_tokens(hd, "f32", -30, width)
    pages, h, t = _first(pool, 1)
    pool.vc[pages, h, t, :] = ONE
    pool.upload()
    o, _, err = attend(pool, q, scale=0.125)
    p = np.exp(s)
    assert err == 0
    assert (np.abs(o.double().cpu().numpy() - (p / (1 + p))[..., None]) <= acc.weight_limit(s)[..., None]).all()


@pytest.mark.parametrize("width", [None, 600], ids=["", "room_for_more"])
def test_two_tokens_on_the_tensor_cores(width):
    pool, q, s = _two_tokens(128, "bf16", -10, width)
    pages, h, _ = _first(pool)
    pool.vc[pages, h, 0, :] = pool.vc[pages, h, 1, :] = ONE
    pool.upload()
    _, lse, _ = attend(pool, q, scale=0.125)
    prev = (torch.full_like(q, -1.0), lse)
    o, _, err = attend(pool, q, scale=0.125, prev=prev)
    got = o.double().cpu().numpy()
    assert err == 0
    assert (np.abs(got) <= acc.joined_limit(s[..., None], got)).all()


@pytest.mark.parametrize("width", [None, 600], ids=["", "room_for_more"])
@pytest.mark.parametrize("lens,hd,G", [([1000, 0, 65], 64, 2), ([6000], 128, 4), ([150], 256, 8), ([700, 64, 0, 33], 96, 8)])
def test_fp32_norm(lens, hd, G, width):
    rng = np.random.default_rng(hd + G)
    pool = Pool(rng, lens, 2, hd, "f32", width=width, mixed=False)
    q, qr = rounded(rng.standard_normal((len(lens), 2 * G, hd)), "f32")
    o, lse, err = attend(pool, q)
    ref, rl, mass = orc.decode(qr, pool.kc, pool.vc, pool.ks, pool.vs, pool.table, pool.lens, hd ** -0.5)
    assert err == 0
    assert np.linalg.norm(o.double().cpu().numpy() - ref) <= acc.L2_LIMIT * np.linalg.norm(mass)


@pytest.mark.parametrize("spread", [3.0, 300.0])
@pytest.mark.parametrize("hd,dtype", [(128, "bf16"), (64, "f32"), (128, "f32"), (256, "bf16")])
def test_every_number_within_its_own_tokens_limit(hd, dtype, spread):
    """Scores of a few and of hundreds, alone and joined with an earlier part near, under and over them."""
    rng = np.random.default_rng(hd + int(spread))
    pool = Pool(rng, [500], 2, hd, dtype)
    q, qr = rounded(rng.standard_normal((1, 8, hd)) * spread, dtype)
    scale, t = hd ** -0.5, np.arange(500)
    pages = pool.table[0, t // 64]
    for lp in (None, -1e4, 3.0 * spread, 1e4):
        prev, prev_ref = None, None
        if lp is not None:
            po, por = rounded(rng.standard_normal((1, 8, hd)), dtype)
            prev, prev_ref = (po, torch.full((1, 8), lp, device="cuda")), (por, lp)
        o, lse, err = attend(pool, q, prev=prev)
        assert err == 0
        for g in range(8):
            K, V = (orc.E4M3[c[pages, g // 4, t % 64]] * s[pages, g // 4][:, None].astype(np.float64) for c, s in ((pool.kc, pool.ks), (pool.vc, pool.vs)))
            ro, rl, lim, llim = acc.per_token_limit(qr[0, g], K, V, scale, dtype == "bf16", None if prev is None else (prev_ref[0][0, g], lp))
            assert (np.abs(o[0, g].double().cpu().numpy() - ro) <= lim).all()
            assert abs(float(lse[0, g]) - rl) <= llim
