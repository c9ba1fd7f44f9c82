"""The 8-bit paged cache at the edges of what its documentation allows, on the GPU."""
from fractions import Fraction

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


@pytest.mark.parametrize("n", [1, 64, 100])
def test_append_fills_the_longest_table(n):
    """The last tokens of a sequence of 64 (2^25 - 1) tokens: the page table has no entry behind them, and what lies
    there (here: ids that no pool has) is not looked at."""
    rng = np.random.default_rng(n)
    width = (1 << 25) - 1
    room = torch.full((width + 65,), -1, dtype=torch.int32, device="cuda")
    pages = -(-n // 64)
    room[width - pages:width] = torch.arange(pages, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((pages, 1, 64, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, 1), 2.0 ** -24, device="cuda") for _ in range(2))
    lens = torch.tensor([64 * width], dtype=torch.int32, device="cuda")
    kv = lr.Kv8Pages(kc, vc, ks, vs, room[:width].view(1, width), lens, torch.bfloat16)
    x, xr = rounded(rng.standard_normal((n, 1, 64)), "bf16")
    cu, ws = torch.tensor([0, n], dtype=torch.int32, device="cuda"), lr.workspace(256)
    lr.lr_kv8_append(kv, x, x, ws, cu_tokens=cu)
    assert lr.lr_get_device_error(ws) == 0
    want = [np.zeros((pages, 1, 64, 64), np.uint8) for _ in range(2)] + [np.full((pages, 1), 2.0 ** -24, np.float32) for _ in range(2)]
    orc.append(*want, np.arange(pages)[None], [64 * pages], [0, n], xr, xr, [], 0, False)
    for got, w in zip((kc, vc, ks, vs), want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)


@pytest.mark.parametrize("width", [None, 600], ids=["", "room_for_more"])
@pytest.mark.parametrize("hd,dtype", [(128, "bf16"), (64, "f32"), (256, "bf16")])
def test_attention_over_the_largest_values(hd, dtype, width):
    """Values up to 3e38, as lr_kv8_append stores them: their sum over the tokens is far out of fp32's range, their
    weighted mean is not. Pages of small values between them, an earlier part as large."""
    rng = np.random.default_rng(hd)
    pool = Pool(rng, [500, 64, 3], 2, hd, dtype, width=width, mixed=False)
    for b, n in enumerate(pool.lens):
        for i in range(-(-int(n) // 64)):
            if i % 3 == 1:
                continue
            page, rows = pool.table[b, i], min(64, int(n) - 64 * i)
            pool.vs[page] = 2.0 ** 120
            pool.vc[page, :, :rows] = orc.e4m3_codes(rng.uniform(200, 225, (2, rows, hd)))  # 2.7e38 to 3e38
    pool.upload()
    q, qr = rounded(0.1 * rng.standard_normal((3, 8, hd)), dtype)  # near equal weights
    po, por = rounded(rng.uniform(2e38, 3e38, (3, 8, hd)), dtype)
    pl = rng.uniform(3, 7, (3, 8)).astype(np.float32)
    for prev, ref_prev in ((None, ()), ((po, torch.from_numpy(pl).cuda()), (por, pl.astype(np.float64)))):
        o, lse, err = attend(pool, q, prev=prev)
        assert err == 0
        ref = orc.decode(qr, pool.kc, pool.vc, pool.ks, pool.vs, pool.table, pool.lens, hd ** -0.5, 0, *ref_prev)
        assert np.abs(ref[0]).max() > 1.5e38
        check_attention((o, lse), ref, pool, qr, hd ** -0.5, 500)


@pytest.mark.parametrize("rot,inter", [(0, False), (128, False), (128, True), (64, False)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("single", [False, True])
def test_append_to_a_page_whose_scale_is_no_power_of_two(single, dtype, rot, inter):
    """A page written by somebody else, with scales 3 and 0.7: codes are those of the fp32 quotient, numbers halfway
    between two codes and their neighbours among them. Rotated keys are not compared, their values are."""
    rng = np.random.default_rng(rot + inter)
    mids = (orc.E4M3[:0x7E] + orc.E4M3[1:0x7F]) / 2
    mids = np.resize(mids[mids < 200], 128).astype(np.float32)
    for s in (np.float32(3.0), np.float32(0.7)):
        pool = Pool(rng, [5], 2, 128, dtype, room=[64])
        for scale in (pool.ks, pool.vs):
            scale[pool.table[0, 0]] = s
        pool.upload()
        pool.set_lens([6])
        x = np.stack([mids * s, np.nextafter(-mids * s, np.float32(1e9))])[None]  # [1, 2 heads, 128]
        xd, xr = rounded(x, dtype)
        quotient = (xr.astype(np.float32) / s).astype(np.float64)
        cu = None if single else torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        rope = None
        if rot:
            inv = torch.from_numpy((1 / 10000.0 ** (np.arange(0, rot, 2) / rot)).astype(np.float32)).cuda()
            rope = lr.Rope(inv, rot, inter)
        ws = lr.workspace(256)
        lr.lr_kv8_append(pool.kv, xd, xd, ws, cu_tokens=cu, rope=rope)
        assert lr.lr_get_device_error(ws) == 0
        kc, vc, ks, vs = pool.arrays()
        page = pool.table[0, 0]
        assert (vs[page] == s).all() and (ks[page] >= s).all()
        np.testing.assert_array_equal(vc[page, :, 5], orc.e4m3_codes(quotient)[0])
        np.testing.assert_array_equal(vc[page, :, :5], pool.vc[page, :, :5])
        if not rot:
            np.testing.assert_array_equal(kc[page, :, 5], orc.e4m3_codes(quotient)[0])


@pytest.mark.parametrize("path", ["pair", "general"])
def test_nan_query_over_the_packed_context_is_not_an_empty_context(path, monkeypatch):
    """The log-sum-exp of a head whose scores are NaN is NaN, so that the joined result is too: -inf would leave the
    packed context out without a word."""
    monkeypatch.setenv("LOWRAM_DECODE_PATH", path)
    p = H.packed_problem(H.small(T=300))
    w = p.w
    q, _ = H.queries(p, 0)
    q = q.clone()
    q[0, 1, 3] = float("nan")
    shape = H.shape_of(w)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = lr.workspace(lr.lr_decode_workspace_bytes(shape, w.n_q_heads, 0))
    lr.lr_decode_attn_lse(shape, 0, w.n_q_heads, q, p.st["A"], p.st["Bt"], H.gpu_predictor(p), p.st["idx"], p.st["val"],
                          p.st["ptr"], p.k, None, 0, 0.0, o, lse, ws)
    want = torch.zeros(w.n_q_heads, dtype=torch.bool, device="cuda")
    want[1] = True
    assert torch.equal(torch.isnan(lse[0]), want) and torch.isfinite(lse[0][~want]).all()
    pool = Pool(np.random.default_rng(0), [70], w.n_kv_heads, w.head_dim)
    clean, _ = H.queries(p, 0)
    joined, lse2, _ = attend(pool, clean, prev=(o, lse))
    assert torch.isnan(joined[0, 1]).all() and torch.equal(torch.isnan(lse2[0]), want)
    assert torch.isfinite(joined[0][~want]).all()


TWO_PI = 2 * Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899, 10 ** 80)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pos", [0, 1, 12345, 2 ** 30 + 7, 64 * ((1 << 25) - 1) - 1])
@pytest.mark.parametrize("single", [False, True])
def test_rotation_angles_at_every_position(single, pos, dtype):
    """Queries (1, 0) turn into cosine and sine: within 2^-22 (fp32) or 2^-20 (bf16) of the exact angle's, plus the
    output's rounding, for frequencies under and over one radian per token, positive and negative."""
    inv = np.array([0.0, 1.0, 3.0, 6.2, -0.7, 100.5, 1e-6, 3e9] + list(np.random.default_rng(1).uniform(-6.3, 6.3, 56)), np.float32)
    width = pos // 64 + 1
    table = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((1, 1, 64, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((1, 1), device="cuda") for _ in range(2))
    kv = lr.Kv8Pages(kc, vc, ks, vs, table, torch.tensor([pos + 1], dtype=torch.int32, device="cuda"), DT[dtype])
    x = torch.zeros((1, 1, 128), dtype=DT[dtype], device="cuda")
    x[:, :, :64] = 1.0
    out, ws = torch.empty_like(x), lr.workspace(256)
    cu = None if single else torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    lr.lr_kv8_append(kv, x, x, ws, cu_tokens=cu, rope=lr.Rope(torch.from_numpy(inv).cuda(), 128), q=x, q_out=out)
    assert lr.lr_get_device_error(ws) == 0
    got = out[0, 0].double().cpu().numpy()
    angles = [Fraction(float(f)) * pos for f in inv]
    angles = np.array([float(a - TWO_PI * (a // TWO_PI)) for a in angles])
    want = np.concatenate([np.cos(angles), np.sin(angles)])
    assert (np.abs(got - want) <= (2.0 ** -20 if dtype == "bf16" else 2.0 ** -22) + HALF[dtype] * np.abs(want)).all()


def test_window_past_an_int_is_the_whole_sequence():
    rng = np.random.default_rng(2)
    pool = Pool(rng, [200], 1, 128)
    q, _ = rounded(rng.standard_normal((1, 4, 128)), "bf16")
    o, lse, _ = attend(pool, q)
    for window in (2 ** 31, 2 ** 32 + 64, 10 ** 12):
        o2, lse2, err = attend(pool, q, window=window)
        assert err == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)
    with pytest.raises(RuntimeError):
        attend(pool, q, window=-1)


@pytest.mark.parametrize("width", [None, 600], ids=["", "room_for_more"])
@pytest.mark.parametrize("hd,dtype", [(128, "bf16"), (64, "f32")])
@pytest.mark.parametrize("before", ["nothing", "memcpy", "memset", "two_streams", "itself"])
def test_attention_captured_behind(before, hd, dtype, width):
    """A captured call that starts the graph, or follows a copy of its lengths, a memset, work joined from another
    stream or another call whose result it takes; replayed with other inputs, equal to the same calls without a graph."""
    rng = np.random.default_rng(hd)
    pool = Pool(rng, [300, 200], 2, hd, dtype, width=width)
    src, lens = pool.dev[5].clone(), pool.dev[5]
    q, _ = rounded(rng.standard_normal((2, 8, hd)), dtype)
    prev_o, prev_lse, scratch = torch.randn_like(q), torch.randn((2, 8), device="cuda"), torch.empty(64, device="cuda")
    first = (torch.empty_like(q), torch.empty((2, 8), device="cuda"))
    out = (torch.empty_like(q), torch.empty((2, 8), device="cuda"))
    need = lr.lr_kv8_attn_workspace_bytes(pool.kv, 8)
    ws, ws2, side = lr.workspace(need), lr.workspace(need), torch.cuda.Stream()

    def call():
        if before == "memcpy":
            lens.copy_(src)
        elif before == "memset":
            scratch.zero_()
        elif before == "two_streams":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                lens.copy_(src)
            scratch.zero_()
            torch.cuda.current_stream().wait_stream(side)
        elif before == "itself":
            lr.lr_decode_attn_kv8(pool.kv, 8, q, first[0], ws2, lse=first[1], window=100)
        p = first if before == "itself" else (prev_o, prev_lse)
        lr.lr_decode_attn_kv8(pool.kv, 8, q, out[0], ws, lse=out[1], o_prev=p[0], lse_prev=p[1])

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in ([300, 200], [0, 17], [129, 300]):
        host = torch.tensor([min(n[0], 300), min(n[1], 200)], dtype=torch.int32)
        src.copy_(host)
        if before not in ("memcpy", "two_streams"):
            lens.copy_(src)
        q.copy_(torch.randn_like(q))
        out[0].fill_(7.0), out[1].fill_(7.0)
        graph.replay()
        got = [t.clone() for t in out]
        out[0].fill_(5.0), out[1].fill_(5.0)
        call()
        assert lr.lr_get_device_error(ws) == 0
        assert torch.equal(got[0], out[0]) and torch.equal(got[1], out[1]) and torch.isfinite(out[0].float()).all()


@pytest.mark.parametrize("window", [1, 63, 64, 65, 130, 200])
@pytest.mark.parametrize("behind", [0, 1, 64, 77])
@pytest.mark.parametrize("hd,dtype", [(128, "bf16"), (64, "f32")])
def test_attention_at_the_end_of_the_longest_table(hd, dtype, behind, window):
    """The last tokens of a sequence of 64 (2^25 - 1) tokens, or a few less: the same as of a short one."""
    rng = np.random.default_rng(window + behind)
    width = (1 << 25) - 1
    short = Pool(rng, [64 * 5 - behind], 1, hd, dtype, room=[64 * 5])
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, width - 5:] = short.dev[4][0, :5]
    lens = torch.tensor([64 * width - behind], dtype=torch.int32, device="cuda")
    kv = lr.Kv8Pages(*short.dev[:4], table, lens, DT[dtype])
    q, qr = rounded(rng.standard_normal((1, 4, hd)), dtype)
    o, lse, ws = torch.empty_like(q), torch.empty((1, 4), device="cuda"), lr.workspace(lr.lr_kv8_attn_workspace_bytes(kv, 4))
    lr.lr_decode_attn_kv8(kv, 4, q, o, ws, lse=lse, window=window)
    assert lr.lr_get_device_error(ws) == 0
    ref = orc.decode(qr, short.kc, short.vc, short.ks, short.vs, short.table, short.lens, hd ** -0.5, window)
    check_attention((o, lse), ref, short, qr, hd ** -0.5, 200)
