"""Problem builders of the 8-bit paged cache tests: a pool with permuted pages, on the host and
the GPU, and the tolerances of both operators."""
import numpy as np
import torch

from long_context_decode_lr_b200 import lowram as lr
from oracle import kv8_oracle as orc

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step of the type, relative


def rounded(x, dtype):
    """(device tensor, fp64 values) of x in the storage type."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DT[dtype])
    return t.cuda(), t.double().numpy()


class Pool:
    """Pages of a batch in random order, with numpy copies; unused space holds NaN codes and NaN scales."""

    def __init__(self, rng, lens, hkv, hd, dtype="bf16", room=None, width=None, spare=2, mixed=True, shift=0.0):
        self.hkv, self.hd, self.dtype = hkv, hd, dtype
        room = [max(n, 0) for n in (lens if room is None else room)]
        need = [-(-n // 64) for n in room]
        self.width = max(1, max(need, default=1)) if width is None else width
        n_pages = sum(need) + spare
        order = rng.permutation(n_pages).astype(np.int32)
        self.table = np.full((len(lens), self.width), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lens = np.array(lens, np.int32)
        self.kc = np.full((n_pages, hkv, 64, hd), 0x7F, np.uint8)
        self.vc = self.kc.copy()
        self.ks = np.full((n_pages, hkv), np.nan, np.float32)
        self.vs = self.ks.copy()
        for b, n in enumerate(lens):
            for i in range(-(-max(n, 0) // 64)):
                page, rows = self.table[b, i], min(64, n - 64 * i)
                for h in range(hkv):
                    for codes, scale in ((self.kc, self.ks), (self.vc, self.vs)):
                        s = 2.0 ** (rng.integers(-8, -4) if mixed else -7)
                        scale[page, h] = s
                        x = rng.standard_normal((rows, hd)) + shift
                        codes[page, h, :rows] = orc.e4m3_codes(x * 1.5 / 2.0 ** -7 / 4)
        self.upload()

    def upload(self):
        d = lambda x: torch.from_numpy(x.copy()).cuda()  # noqa: E731
        self.dev = [d(x) for x in (self.kc, self.vc, self.ks, self.vs, self.table, self.lens)]
        self.kv = lr.Kv8Pages(*self.dev, DT[self.dtype])

    def set_lens(self, lens):
        self.lens[:] = lens
        self.dev[5].copy_(torch.from_numpy(self.lens))

    def arrays(self):
        return [t.cpu().numpy() for t in self.dev[:4]]


def attend(pool, q, window=0, scale=0.0, prev=None, stream=None, ws=None, in_place=False):
    """(o, lse, error word) of lr_decode_attn_kv8; outputs start as garbage."""
    hq = q.shape[1]
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    if in_place:
        o, lse = prev
    ws = lr.workspace(lr.lr_kv8_attn_workspace_bytes(pool.kv, hq)) if ws is None else ws
    lr.lr_decode_attn_kv8(pool.kv, hq, q, o, ws, lse=lse, window=window, scale=scale,
                          o_prev=None if prev is None else prev[0], lse_prev=None if prev is None else prev[1],
                          stream=stream)
    return o, lse, lr.lr_get_device_error(ws, stream)


def check_attention(got, ref, pool, q, scale, n_max):
    """Against the fp64 result. The output is rounded to its type (half a step). The weights p carry a
    relative error: scores of fp32 sums are off by at most (hd + 8) 2^-24 sum|q||k| scale, an exponential
    and the sum of n of them by (n + 8) 2^-24, and the tensor-core kernel stores p to 12 significant
    bits (2^-12, counted for bf16). Codes and scales are exact."""
    o, lse = (t.double().cpu().numpy() for t in got[:2])
    ro, rl, mass = ref
    K = np.nanmax(np.abs(orc.E4M3[pool.kc])) * (np.nanmax(pool.ks) if np.isfinite(pool.ks).any() else 0.0)
    s_abs = scale * np.abs(q).sum(-1) * K                                    # >= sum |q||k| scale
    dx = (pool.hd + 8) * 2.0 ** -24 * s_abs
    eps = np.expm1(2 * dx) + (n_max + 8) * 2.0 ** -24 + (2.0 ** -11 if pool.dtype == "bf16" else 0.0)
    tol = HALF[pool.dtype] * np.abs(ro) + eps[..., None] * mass + 1e-30
    assert np.isfinite(o).all()
    worst = (np.abs(o - ro) / tol).max() if o.size else 0.0
    assert worst <= 1.0, f"o off by {worst:.2f} tolerances"
    empty = np.isneginf(rl)
    np.testing.assert_array_equal(np.isneginf(lse), empty)
    ltol = dx + (n_max + 16) * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(empty, 0, rl))
    assert (np.abs(np.where(empty, 0, lse) - np.where(empty, 0, rl)) <= ltol).all()
