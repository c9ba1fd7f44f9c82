"""The limits of kv8_accuracy.py bite: the kernels' splits pass them, and with a term left out they do not (CPU)."""
import numpy as np

from oracle import kv8_oracle as orc

import kv8_accuracy as acc


def test_split_is_right_to_2_to_the_minus_23():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(2.0 ** 13, 2.0 ** 15, 200000), 2.0 ** rng.uniform(-8, 15, 200000)])
    x = x.astype(np.float32).astype(np.float64)
    err = np.abs(acc.fp16_terms(x, 2) - x) / x
    assert 2.0 ** -24 < err.max() <= 2.0 ** -23
    small = 2.0 ** rng.uniform(-60, -14, 200000)
    assert np.abs(acc.fp16_terms(small, 2) - small).max() <= 2.0 ** -36


def test_e4m3_terms():
    """What the header says of the tensor-core kernel's numbers: weights right to 2^-11, or to 2^-27 of the largest
    under 2^-17 of it; bf16 queries exact down to 2^-14 of their head's largest, right to 2^-22 of it below."""
    rng = np.random.default_rng(3)
    p = 2.0 ** -rng.uniform(0, 40, 400000)
    err = np.abs(acc.e4m3_weights(p, 3) - p)
    assert (err <= np.where(p >= 2.0 ** -17, 2.0 ** -11 * p, 2.0 ** -27)).all()
    assert (err[p >= 2.0 ** -17] > 2.0 ** -12 * p[p >= 2.0 ** -17]).any()
    for top in np.arange(128.0, 256.0):  # the largest number of a head, as the kernel scales it: 8 bits
        x = (np.arange(128, 256) * 2.0 ** -np.arange(30)[:, None]).ravel()
        x = x[x <= top]
        q1 = orc.E4M3[orc.e4m3_codes(x)]
        err = np.abs(q1 + orc.E4M3[orc.e4m3_codes((x - q1) * 32.0)] / 32.0 - x)
        assert (err[x >= 2.0 ** -14 * top] == 0).all() and err.max() <= 2.0 ** -22 * top


def test_limits_need_every_term():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((256, 64)).astype(np.float32).astype(np.float64)
    for terms, ok in ((2, True), (1, False)):  # one key: dim d of head h
        err = np.abs(acc.split_queries(q, terms) - q) / 8
        assert (err <= acc.score_limit(q / 8)).all() == ok
    s = -rng.uniform(0.01, 30, 4000)
    p = np.exp(s)
    for terms, ok in ((2, True), (1, False)):
        err = np.abs(acc.split_weights(p, terms) - p) / (1 + p)
        assert (err <= acc.weight_limit(s)).all() == ok
    s = -rng.uniform(0.01, 10, 4000)
    p = np.exp(s)
    for terms, ok in ((3, True), (2, False)):
        left = 0.5 * ((1 + acc.e4m3_weights(p, terms)) / (1 + p) - 1)
        assert (np.abs(left) <= acc.joined_limit(s, left)).all() == ok


def test_norm_limit_needs_every_term():
    rng = np.random.default_rng(2)
    for n, hd in ((1000, 64), (6000, 128), (150, 256)):
        q, K, V = rng.standard_normal((8, hd)) * 1.5, rng.standard_normal((n, hd)) * 0.375, rng.standard_normal((n, hd)) * 0.375
        q = q.astype(np.float32).astype(np.float64)
        ref, _, mass = acc.attention(q, K, V, hd ** -0.5)
        for tq, tp, ok in ((2, 2, True), (1, 2, False), (2, 1, False)):
            got, _, _ = acc.attention(q, K, V, hd ** -0.5, lambda x: acc.split_queries(x, tq), lambda x: acc.split_weights(x, tp))
            assert (np.linalg.norm(got - ref) <= acc.L2_LIMIT * np.linalg.norm(mass)) == ok, (n, hd, tq, tp)
