"""Timed cases of the 8-bit paged KV cache: appending new tokens and the decode step over it.

Every case is one call of a serving loop over the cache of `include/lowram.h`: pages of 64
tokens, keys and values as e4m3 codes with one scale for each page and KV head.

- op "append": new keys and values of a batch go into their pages, rotated by their position
  (rotary embedding), next to the rotated queries.
- op "attn": one decode step, one query token per sequence, over the cached tokens, with the
  log-sum-exp of every head; "joined" cases add an earlier partial result to the same softmax.

The plain forms are elementary torch operations in 32 bits (64 for the rotation angles).
"""
import math

import torch

own = False

PAGE = 64        # tokens of a page
E4M3_MAX = 448.0
MIN_EXP = -24    # smallest scale: 2^-24
ROPE_BASE = 500000.0


# ---------------------------------------------------------------------------------- cases

def listed():
    llama = dict(hkv=8, group=4, hd=128, dtype="bf16")
    return [
        # one chat of a thousand tokens: the smallest call, where latency counts
        dict(name="attn_1k", op="attn", batch=1, max_len=1000, ragged=False, window=0, joined=False, **llama),
        # 32K-token context of the Mistral-shaped group, held in 8 bits
        dict(name="attn_32k", op="attn", batch=1, max_len=32768, ragged=False, window=0, joined=False, **llama),
        # 262K-token context of the Llama-shaped group
        dict(name="attn_262k", op="attn", batch=1, max_len=262144, ragged=False, window=0, joined=False, **llama),
        # four 131K-token sequences: the largest decode step of the benchmark sweep
        dict(name="attn_131k_b4", op="attn", batch=4, max_len=131072, ragged=False, window=0, joined=False, **llama),
        # a serving batch: 64 sequences of ragged lengths (one padded slot), eight query heads a KV head
        dict(name="attn_ragged_b64", op="attn", batch=64, max_len=12001, ragged=True, window=0, joined=False,
             hkv=4, group=8, hd=128, dtype="bf16"),
        # tokens generated since the packing, joined with the result over the packed context, last 4096 only
        dict(name="attn_joined_b16", op="attn", batch=16, max_len=9001, ragged=True, window=4096, joined=True, **llama),
        # the small fp32 configuration (two KV heads, head_dim 64)
        dict(name="attn_tiny_f32", op="attn", batch=2, max_len=1024, ragged=False, window=0, joined=False,
             hkv=2, group=2, hd=64, dtype="f32"),
        # one new token for one sequence of 32K: a decode step's append
        dict(name="append_1", op="append", batch=1, new=1, before=32768 - 30, ragged=False, rot=128,
             interleaved=False, **llama),
        # one new token for each of 64 sequences
        dict(name="append_64", op="append", batch=64, new=1, before=5000, ragged=False, rot=128, interleaved=False,
             **llama),
        # a 32K-token prompt going into an empty cache
        dict(name="append_32k", op="append", batch=1, new=32768, before=0, ragged=False, rot=128, interleaved=False,
             **llama),
        # prompt chunks and single tokens of 24 sequences in one call, half of the head rotated in adjacent pairs
        dict(name="append_mixed", op="append", batch=24, new=2000, before=777, ragged=True, rot=64, interleaved=True,
             **llama),
        # a prompt of the small fp32 configuration
        dict(name="append_tiny_f32", op="append", batch=2, new=1000, before=24, ragged=False, rot=64,
             interleaved=False, hkv=2, group=2, hd=64, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    f32 = rng.random() < 0.2
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    hd = rng.choice([64, 96, 128]) if f32 else 128
    case = dict(hkv=hkv, group=group, hd=hd, dtype="f32" if f32 else "bf16", ragged=rng.random() < 0.5)
    if rng.random() < 0.6:
        batch = _log(rng, 1, 128)
        room = (60_000 if f32 else 524_288) // batch  # the largest listed step holds 524,288 tokens
        max_len = _log(rng, 1, min(262_144, room))
        case.update(op="attn", batch=batch, max_len=max_len, joined=rng.random() < 0.3,
                    window=rng.choice([0, 0, 0, max(1, max_len // 3)]))
    else:
        batch = _log(rng, 1, 128)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, 32_768 // batch)
        case.update(op="append", batch=batch, new=new, before=rng.choice([0, _log(rng, 1, 20_000)]),
                    rot=rng.choice([hd, hd // 2, 0]), interleaved=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------------------------- inputs

def _spread(n, batch, ragged):
    """Lengths of the batch's sequences: n each, or spread over 1 .. n in a fixed shuffled order."""
    if not ragged or batch == 1:
        return [n] * batch
    return [max(1, n * (1 + (b * 37 + 11) % batch) // batch) for b in range(batch)]


def _shapes(case):
    """(tokens in the cache after the call, new tokens) of every sequence."""
    if case["op"] == "attn":
        lens = _spread(case["max_len"], case["batch"], case["ragged"])
        if case["ragged"] and case["batch"] >= 8:
            lens[case["batch"] // 2] = 0  # a padded slot of the batch
        return lens, [0] * case["batch"]
    new = _spread(case["new"], case["batch"], case["ragged"])
    if case["ragged"] and case["new"] > 1:
        new = [1 if b % 3 == 2 else n for b, n in enumerate(new)]  # every third sequence decodes
    before = [max(0, case["before"] - 13 * b) if case["ragged"] else case["before"] for b in range(case["batch"])]
    return [p + n for p, n in zip(before, new)], new


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _pages(lens):
    return [-(-n // PAGE) for n in lens]


def _pow2_scale(amax):
    """Smallest power of two s, at least 2^-24, with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)))


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    hkv, hd, B = case["hkv"], case["hd"], case["batch"]
    lens, new = _shapes(case)
    need = _pages(lens)
    width = max(1, max(need))
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    order_host = order.cpu()
    for b, n in enumerate(need):
        table[b, :n] = order_host[at:at + n]
        at += n
    s = dict(table=table.to(dev), lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    # keys carry a few strong channels, values do not; magnitudes drift from page to page
    strong = 0.6 + 2.2 * (torch.rand(hd, generator=g, device=dev) < 0.06)
    codes, scales = {}, {}
    for name in ("k", "v"):
        codes[name] = torch.empty((n_pages, hkv, PAGE, hd), dtype=torch.uint8, device=dev)
        scales[name] = torch.empty((n_pages, hkv), device=dev)
        for p0 in range(0, n_pages, 1024):
            p1 = min(n_pages, p0 + 1024)
            x = torch.randn((p1 - p0, hkv, PAGE, hd), generator=g, device=dev)
            x = x * strong if name == "k" else x
            x *= 0.5 + torch.rand((p1 - p0, hkv, 1, 1), generator=g, device=dev)
            sc = _pow2_scale(x.abs().amax((2, 3)))
            scales[name][p0:p1] = sc
            codes[name][p0:p1] = (x / sc[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    s.update(k_codes=codes["k"], v_codes=codes["v"], k_scale=scales["k"], v_scale=scales["v"])
    hq = hkv * case["group"]
    dt = _dtype(case)
    if case["op"] == "attn":
        # what lies behind a sequence's last token is whatever the pool held: NaN codes here
        for b, n in enumerate(lens):
            if n % PAGE:
                for name in ("k", "v"):
                    codes[name][int(table[b, n // PAGE]), :, n % PAGE:] = 0x7F
        s["q"] = (1.3 * torch.randn((B, hq, hd), generator=g, device=dev)).to(dt)
        if case["joined"]:
            s["o_prev"] = (0.3 * torch.randn((B, hq, hd), generator=g, device=dev)).to(dt)
            s["lse_prev"] = 4.0 + 4.0 * torch.rand((B, hq), generator=g, device=dev)
        return s
    n = sum(new)
    # one projection gives queries, keys and values side by side: rows of the fused tensor
    qkv = torch.randn((n, hq + 2 * hkv, hd), generator=g, device=dev)
    qkv[:, hq:hq + hkv] *= strong
    s["qkv"] = qkv.to(dt)
    if case["new"] > 1:
        cu = torch.zeros(B + 1, dtype=torch.int64)
        cu[1:] = torch.cumsum(torch.tensor(new), 0)
        s["cu"] = cu.to(torch.int32).to(dev)
    else:
        s["cu"] = None  # one token each
    rot = case["rot"]
    if rot:
        s["inv_freq"] = (1.0 / ROPE_BASE ** (torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(dev)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    hkv, hd = case["hkv"], case["hd"]
    hq = hkv * case["group"]
    s.update(case=dict(case), hq=hq)
    if case["op"] == "attn":
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device="cuda")
    else:
        n = s["qkv"].shape[0]
        s["q_out"] = torch.empty((n, hq, hd), dtype=_dtype(case), device="cuda")
    if own:
        from long_context_decode_lr_b200 import lowram as lr
        s["lr"] = lr
        s["kv"] = lr.Kv8Pages(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                              _dtype(case))
        if case["op"] == "attn":
            s["ws"] = lr.workspace(lr.lr_kv8_attn_workspace_bytes(s["kv"], hq))
        else:
            s["ws"] = lr.workspace(lr.lr_kv8_append_workspace_bytes(s["kv"]))
            s["rope"] = lr.Rope(s["inv_freq"], case["rot"], case["interleaved"]) if case["rot"] else None
    return s


# ---------------------------------------------------------------------------------- one pass

def run(s):
    return _run_attn(s) if s["case"]["op"] == "attn" else _run_append(s)


def _run_attn(s):
    case = s["case"]
    if own:
        s["lr"].lr_decode_attn_kv8(s["kv"], s["hq"], s["q"], s["o"], s["ws"], lse=s["lse"], window=case["window"],
                                   o_prev=s.get("o_prev"), lse_prev=s.get("lse_prev"))
        return [s["o"], s["lse"]]
    B, hkv, G, hd = case["batch"], case["hkv"], case["group"], case["hd"]
    table = s["table"].clamp_min(0).long()
    width = table.shape[1]
    T = width * PAGE
    t = torch.arange(T, device=table.device)
    n = s["lens"].long()[:, None]
    seen = t < n
    if case["window"]:
        seen = seen & (t >= n - case["window"])
    seen = seen[:, None, :]                                                       # [B, 1, T]

    def rows(codes, scale):
        x = codes.view(torch.float8_e4m3fn)[table].float() * scale[table][..., None, None]
        return x.transpose(1, 2).reshape(B, hkv, T, hd).masked_fill(~seen[..., None], 0.0)

    q = s["q"].float().view(B, hkv, G, hd) / math.sqrt(hd)
    x = torch.matmul(q, rows(s["k_codes"], s["k_scale"]).transpose(2, 3))          # [B, hkv, G, T]
    x = x.masked_fill(~seen[:, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    if case["joined"]:
        prev = s["lse_prev"].view(B, hkv, G, 1)
        top = torch.maximum(top, prev)
    ref = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - ref)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows(s["v_codes"], s["v_scale"]))
    if case["joined"]:
        w = torch.exp(prev - ref)
        o = o + w * s["o_prev"].float().view(B, hkv, G, hd)
        total = total + w
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (ref + torch.log(total)).view(B, hkv * G)
    return [o.view(B, hkv * G, hd).to(s["q"].dtype), lse]


def _run_append(s):
    case = s["case"]
    hkv, hd, rot = case["hkv"], case["hd"], case["rot"]
    hq = s["hq"]
    q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hkv], s["qkv"][:, hq + hkv:]
    outs = [s["k_codes"].view(torch.float8_e4m3fn), s["v_codes"].view(torch.float8_e4m3fn), s["k_scale"],
            s["v_scale"], s["q_out"]]
    if own:
        s["lr"].lr_kv8_append(s["kv"], k, v, s["ws"], cu_tokens=s["cu"], rope=s["rope"], q=q, q_out=s["q_out"])
        return outs
    n = q.shape[0]
    dev = q.device
    j = torch.arange(n, device=dev)
    cu = torch.arange(case["batch"] + 1, device=dev) if s["cu"] is None else s["cu"].long()
    b = torch.searchsorted(cu, j, right=True) - 1
    lens = s["lens"].long()
    pos = lens[b] - cu[b + 1] + j
    page, slot = s["table"].long()[b, pos // PAGE], pos % PAGE
    qf, kf, vf = q.float(), k.float(), v.float()
    if rot:
        a = pos.double()[:, None, None] * s["inv_freq"].double()
        c, d = torch.cos(a).float(), torch.sin(a).float()
        qf, kf = _rotate(qf, c, d, rot, case["interleaved"]), _rotate(kf, c, d, rot, case["interleaved"])
    s["q_out"].copy_(qf)
    # the pages that receive tokens, and the tokens that they already hold: only a sequence's first page has any
    n_pages = s["k_codes"].shape[0]
    touched = torch.zeros(n_pages, dtype=torch.bool, device=dev)
    touched[page] = True
    has_new = cu[1:] > cu[:-1]
    pos0 = torch.where(has_new, lens - (cu[1:] - cu[:-1]), torch.zeros_like(lens))
    page0 = s["table"].long().gather(1, (pos0 // PAGE)[:, None])[:, 0].clamp_min(0)
    held = torch.where(has_new, pos0 % PAGE, torch.zeros_like(pos0))
    held_in = torch.zeros(n_pages, dtype=torch.int64, device=dev).index_put((page0,), held, accumulate=True)
    for x, codes, scale in ((kf, s["k_codes"], s["k_scale"]), (vf, s["v_codes"], s["v_scale"])):
        amax = torch.zeros((n_pages, hkv), device=dev)
        amax.scatter_reduce_(0, page[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
        fresh = _pow2_scale(amax)
        now = torch.where(held_in[:, None] > 0, torch.maximum(scale, fresh), fresh)
        f8 = codes.view(torch.float8_e4m3fn)
        old = f8[page0].float()                                                     # [B, hkv, 64, hd]
        moved = (old * (scale[page0] / now[page0])[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        keep = (torch.arange(PAGE, device=dev) < held[:, None]) & has_new[:, None]
        rows_b, rows_s = keep.nonzero(as_tuple=True)
        codes[page0[rows_b], :, rows_s] = moved[rows_b, :, rows_s]
        codes[page, :, slot] = (x / now[page][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale.copy_(torch.where(touched[:, None], now, scale))
    return outs


def _rotate(x, c, s, rot, interleaved):
    y = x.clone()
    if interleaved:
        x0, x1 = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = x0 * c - x1 * s, x1 * c + x0 * s
    else:
        h = rot // 2
        x0, x1 = x[..., :h], x[..., h:rot]
        y[..., :h], y[..., h:rot] = x0 * c - x1 * s, x1 * c + x0 * s
    return y


# ---------------------------------------------------------------------------------- work

def work(case):
    lens, new = _shapes(case)
    hkv, hd = case["hkv"], case["hd"]
    hq = hkv * case["group"]
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attn":
        read = [min(n, case["window"]) if case["window"] else n for n in lens]
        t = sum(read)
        rows = case["batch"] * hq
        b = 2 * t * hkv * hd + 2 * rows * hd * es + rows * 4 + 8 * sum(_pages(read)) * hkv
        if case["joined"]:
            b += rows * (hd * es + 4)
        return dict(bytes=b, flops=4 * t * hq * hd)
    n = sum(new)
    b = n * (hq + 2 * hkv) * hd * es + n * hq * hd * es + 2 * n * hkv * hd + 8 * sum(_pages(new)) * hkv
    return dict(bytes=b, flops=3 * n * (hq + hkv) * case["rot"] + 2 * n * 2 * hkv * hd)


# ---------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    lens, new = _shapes(case)
    hkv, G, hd = case["hkv"], case["group"], case["hd"]
    hq = hkv * G
    table = s["table"].cpu()
    if case["op"] == "attn":
        o = torch.zeros((case["batch"], hq, hd), dtype=torch.float64, device="cuda")
        lse = torch.full((case["batch"], hq), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            lo = max(0, n - case["window"]) if case["window"] else 0
            ids = table[b, :-(-n // PAGE)].long().cuda()
            for h in range(hkv):
                heads = slice(h * G, (h + 1) * G)
                x = torch.zeros((G, 0), dtype=torch.float64, device="cuda")
                v = torch.zeros((0, hd), dtype=torch.float64, device="cuda")
                if n > lo:
                    k = s["k_codes"][ids, h].view(torch.float8_e4m3fn).double() * s["k_scale"][ids, h].double()[:, None, None]
                    v = s["v_codes"][ids, h].view(torch.float8_e4m3fn).double() * s["v_scale"][ids, h].double()[:, None, None]
                    k, v = k.reshape(-1, hd)[lo:n], v.reshape(-1, hd)[lo:n]
                    x = s["q"][b, heads].double() @ k.T / math.sqrt(hd)
                if case["joined"]:
                    x = torch.cat([s["lse_prev"][b, heads].double()[:, None], x], 1)
                if not x.shape[1]:
                    continue
                lse[b, heads] = torch.logsumexp(x, 1)
                w = torch.exp(x - lse[b, heads][:, None])
                if case["joined"]:
                    o[b, heads] = w[:, :1] * s["o_prev"][b, heads].double() + w[:, 1:] @ v
                else:
                    o[b, heads] = w @ v
        return [o, lse]
    if sum(new) * hkv * hd > 200_000_000:
        return None
    start, q_out = 0, torch.empty((sum(new), hq, hd), dtype=torch.float64, device="cuda")
    codes = [s[c].view(torch.float8_e4m3fn).double() for c in ("k_codes", "v_codes")]
    scales = [s[c].double() for c in ("k_scale", "v_scale")]
    for b, n in enumerate(new):
        x = s["qkv"][start:start + n].double()
        p0 = lens[b] - n
        if case["rot"]:
            half = case["rot"] // 2
            i0 = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
            i1 = i0 + (1 if case["interleaved"] else half)
            z = torch.polar(torch.ones((n, half), dtype=torch.float64, device="cuda"),
                            torch.arange(p0, lens[b], device="cuda", dtype=torch.float64)[:, None] * s["inv_freq"].double())
            turned = torch.complex(x[:, :hq + hkv, i0], x[:, :hq + hkv, i1]) * z[:, None]
            x[:, :hq + hkv, i0], x[:, :hq + hkv, i1] = turned.real, turned.imag
        q_out[start:start + n] = x[:, :hq]
        for c, sc, rows in zip(codes, scales, (x[:, hq:hq + hkv], x[:, hq + hkv:])):
            for i in range(p0 // PAGE, -(-lens[b] // PAGE)):
                lo, hi = max(p0, i * PAGE), min(lens[b], (i + 1) * PAGE)
                page = int(table[b, i])
                r = rows[lo - p0:hi - p0].transpose(0, 1)
                top = r.abs().amax((1, 2))
                f = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)).clamp_min(MIN_EXP))
                f = torch.where((top <= E4M3_MAX * f / 2) & (f > 2.0 ** MIN_EXP), f / 2, f)  # log2 of a power of two
                if lo > i * PAGE:
                    f = torch.maximum(f, sc[page])
                    c[page, :, :lo - i * PAGE] *= (sc[page] / f)[:, None, None]
                c[page, :, lo - i * PAGE:hi - i * PAGE] = r / f[:, None, None]
                sc[page] = f
        start += n
    return [*codes, *scales, q_out]
