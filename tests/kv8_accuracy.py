"""What the 8-bit cache's attention promises of its queries and weights, as limits that a missing term breaks, and
the two ways of splitting them in numpy.

Units are u = 2^-24, a rounding of fp32. Two problems show a number of the kernel by itself:

- "one key": a sequence of one token whose key has a single 1, in dim d. Its log-sum-exp is the score
  scale q[d]. Roundings: the query's split (2 u), log2 e and ln 2 (1 u each), the join of the terms, the product
  with the factor, the product with ln 2 (1 u each): 7 u |score|; the limit is 8 u.
- "two tokens": scores 0 and s < 0, values 0 and 1, so that o = p / (1 + p) with p = e^s. Relative error: the
  score's 8 u |s|, the exponential's 2^-22 = 4 u, the weight's split (2 u), the join of the terms, the sum, its
  reciprocal and the product with it (1 u each): 10 u + 8 u |s|; the limit is 12 u + 8 u |s|, and absolute 2^-51
  where the second term of the weight is an fp16 subnormal.
"""
import numpy as np

U = 2.0 ** -24


def score_limit(score):
    return 8 * U * np.abs(score)


def weight_limit(s):
    p = np.exp(s)
    return (12 + 8 * np.abs(s)) * U * p / (1 + p) + 2.0 ** -51


# Weights of the tensor-core kernel are rounded to fp16, right to 2^-11, where fp32 keeps the sum that divides them. Joined with an
# earlier part of the same weight and the opposite value -1, two tokens of value 1 leave half of
# (1 + p^) / (1 + p) - 1, right to 20 roundings of numbers under 1, and rounded to bf16.
def joined_limit(s, got):
    p = np.exp(s)
    return 0.5 * 2.0 ** -11 * p / (1 + p) + 20 * U + 2.0 ** -8 * np.abs(got)


# Over many tokens errors have random signs. Scores under 4: a score's systematic error is 2 u of it (log2 e and the
# factor), the exponential's 4 u, the splits' 4 u: under 16 u = 2^-20 of sum w |v|, per number and so in the norm.
L2_LIMIT = 16 * U


def fp16_terms(x, terms):
    """x as the sum of `terms` fp16 numbers, the second one 2^11 times as fine."""
    t0 = x.astype(np.float16).astype(np.float64)
    if terms == 1:
        return t0
    return t0 + ((x - t0) * 2048.0).astype(np.float16).astype(np.float64) / 2048.0


def split_queries(q, terms):
    """Each head scaled to [2^14, 2^15) by a power of two."""
    e = 2.0 ** (np.floor(np.log2(np.abs(q).max(-1, keepdims=True))) - 14)
    return fp16_terms(q / e, terms) * e


def split_weights(p, terms):
    return fp16_terms(p * 32768.0, terms) / 32768.0


def e4m3_weights(p, terms):
    """p times 256 to fp16, then terms of four bits, each 32 times as fine as the one before."""
    from oracle import kv8_oracle as orc
    rest = (p * 256.0).astype(np.float16).astype(np.float64)
    total = np.zeros_like(p)
    for i in range(terms):
        t = orc.E4M3[orc.e4m3_codes(rest)]
        total += t / 32.0 ** i
        rest = (rest - t) * 32.0
    return total / 256.0


def attention(q, K, V, scale, split_q=lambda x: x, split_p=lambda x: x):
    """(o [heads, hd], lse, sum w |v|) in fp64 but for the splits; q [heads, hd], K and V [tokens, hd]."""
    s = scale * split_q(q) @ K.T
    p = np.exp(s - s.max(1, keepdims=True))
    total = p.sum(1, keepdims=True)
    return split_p(p) @ V / total, s.max(1) + np.log(total[:, 0]), p @ np.abs(V) / total


def per_token_limit(q, K, V, scale, bf16, prev=None):
    """(o, lse, limit of o, limit of lse) of one head in fp64. A score is a sum of fp32 products, off by at most
    (hd + 12) u scale sum |q||k| of its own token; its weight by that, the exponential and the split relative to
    its own size, and all of them by the sum's relative error. prev: (o_prev, lse_prev), exact."""
    s, slack, vals = scale * K @ q, (K.shape[1] + 12) * U * scale * np.abs(K) @ np.abs(q), V
    if prev is not None:
        s, slack, vals = np.append(s, prev[1]), np.append(slack, 2 * U * abs(prev[1])), np.concatenate([V, prev[0][None]])
    p = np.exp(s - s.max())
    w = p / p.sum()
    # an fp32 score in units of log 2, and the largest one that it is taken from
    own = np.expm1(slack + 4 * U * (np.abs(s) + np.abs(s).max())) + (2.0 ** -11 if bf16 else 2.0 ** -21) + len(s) * U
    weight = w * (own + (w * own).sum())
    o = w @ vals
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    lse = s.max() + np.log(p.sum())
    return o, lse, weight @ np.abs(vals) + half * np.abs(o) + 2.0 ** -27 * np.abs(vals).max(0), (w * own).sum() + 8 * U * abs(lse)
