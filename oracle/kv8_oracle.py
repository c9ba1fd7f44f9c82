"""Plain fp64 numpy definition of the 8-bit paged cache: e4m3 codes with a power-of-two scale per
page and KV head, appending with rotary embedding, decode attention. Slow loops, one token at a
time; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np

PAGE = 64
MIN_SCALE = 2.0 ** -24


def _e4m3_table():
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v[c] = -x if c & 128 else x
    v[0x7F] = v[0xFF] = np.nan
    return v


E4M3 = _e4m3_table()
_GRID = E4M3[:0x7F]  # 0 .. 448 ascending: the index is the code


def e4m3_codes(x):
    """Codes of finite values, nearest even, saturating at 448; NaN and infinities give 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    ok = np.isfinite(x)
    a = np.where(ok, np.minimum(a, 448.0), 0.0)
    hi = np.minimum(np.searchsorted(_GRID, a), 0x7E)  # first grid value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == _GRID[hi], hi, code)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(ok, code, 0x7F).astype(np.uint8)


def fresh_scale(amax):
    """Smallest power of two s >= 2^-24 with amax <= 448 s."""
    s = MIN_SCALE
    while amax > 448.0 * s:
        s *= 2.0
    return s


def rotate(x, pos, inv_freq, rot, interleaved):
    """x [heads, hd] of one token at `pos`."""
    y = np.array(x, dtype=np.float64)
    for j in range(rot // 2):
        a = float(pos) * float(inv_freq[j])
        c, s = np.cos(a), np.sin(a)
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, rot // 2 + j)
        x0, x1 = np.array(y[:, i0]), np.array(y[:, i1])
        y[:, i0], y[:, i1] = x0 * c - x1 * s, x1 * c + x0 * s
    return y


def append(k_codes, v_codes, k_scale, v_scale, table, lens, cu, k, v, inv_freq, rot, interleaved):
    """In place on the code and scale arrays. Returns the rotated keys [n, Hkv, hd] in fp64 and the
    (page, head) pairs whose key and value scales were settled."""
    B, hkv = len(lens), k.shape[1]
    kr = np.array(k, dtype=np.float64)
    touched = []
    for b in range(B):
        n = int(cu[b + 1] - cu[b])
        p0 = int(lens[b]) - n
        for i in range(n):
            if rot:
                kr[cu[b] + i] = rotate(k[cu[b] + i], p0 + i, inv_freq, rot, interleaved)
        pos = p0
        while pos < lens[b]:
            end = min(int(lens[b]), (pos // PAGE + 1) * PAGE)
            page, slot, rows = int(table[b, pos // PAGE]), pos % PAGE, slice(cu[b] + pos - p0, cu[b] + end - p0)
            for h in range(hkv):
                for codes, scale, x in ((k_codes, k_scale, kr[rows, h]), (v_codes, v_scale, v[rows, h])):
                    f = np.abs(x[np.isfinite(x)])
                    s = fresh_scale(f.max() if f.size else 0.0)
                    if slot:
                        old = float(scale[page, h])
                        s = max(s, old)
                        if s > old:
                            codes[page, h, :slot] = rescaled(codes[page, h, :slot], old / s)
                    scale[page, h] = s
                    codes[page, h, slot:slot + end - pos] = e4m3_codes(x / s)
                touched.append((page, h))
            pos = end
    return kr, touched


def rescaled(codes, ratio):
    """Codes times ratio; NaN codes stay NaN."""
    return e4m3_codes(E4M3[codes] * ratio)


def decode(q, k_codes, v_codes, k_scale, v_scale, table, lens, scale, window=0, o_prev=None, lse_prev=None):
    """(o [B, Hq, hd], lse [B, Hq], mass): mass [B, Hq, hd] is sum_t w_t |v_t| (plus the earlier
    part's), the magnitude that rounding errors of the weights are relative to."""
    B, hq, hd = q.shape
    hkv = k_codes.shape[1]
    G = hq // hkv
    o, lse, mass = np.zeros((B, hq, hd)), np.full((B, hq), -np.inf), np.zeros((B, hq, hd))
    for b in range(B):
        n = int(lens[b])
        lo = max(0, n - window) if window else 0
        for h in range(hkv):
            ids = [int(table[b, t // PAGE]) for t in range(lo, n)]
            ok = [i for i, p in enumerate(ids) if 0 <= p < k_codes.shape[0]]
            t = np.array([lo + i for i in ok], dtype=np.int64)
            p = np.array([ids[i] for i in ok], dtype=np.int64)
            K = E4M3[k_codes[p, h, t % PAGE]] * k_scale[p, h].astype(np.float64)[:, None] if len(t) else np.zeros((0, hd))
            V = E4M3[v_codes[p, h, t % PAGE]] * v_scale[p, h].astype(np.float64)[:, None] if len(t) else np.zeros((0, hd))
            for g in range(h * G, (h + 1) * G):
                s = scale * (K @ q[b, g])
                vals = V
                if lse_prev is not None and lse_prev[b, g] != -np.inf:
                    s = np.concatenate([[lse_prev[b, g]], s])
                    vals = np.concatenate([o_prev[b, g][None], V])
                if not len(s):
                    continue
                m = s.max()
                w = np.exp(s - m)
                lse[b, g] = m + np.log(w.sum())
                w = w / w.sum()
                o[b, g] = w @ vals
                mass[b, g] = w @ np.abs(vals)
    return o, lse, mass
