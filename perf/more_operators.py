"""What the 8-bit paged cache and the shared prefix are measured on: the append
that quantises keys and values as it writes them (`ra_paged_append_fp8`), the
same pages read back (`ra_paged_read_fp8`) and attended to
(`ra_paged_decode_fp8`), and attention for requests that share a prefix
(`ra_paged_decode_prefix`).

`run` computes a case in plain torch operations, or, with `own` true,
through the package's calls.  Ragged lengths are a fixed set of values per
case, handed to the requests in an order that the seed gives, so a case's
work does not depend on its seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BASE = 10000.0
CODE, SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu


def listed():
    return [
        # One step of a serving loop: a new token for most of 256 requests.
        dict(name="append8-step", op="append8", n_req=256, max_len=8000, new_max=1, heads=32,
             kv_heads=8, d=128, rot=128, inter=False, scaled=True, norm=True, page=16),
        # Prompts arrive: 64 requests, some 22K new tokens in all.
        dict(name="append8-prompts", op="append8", n_req=64, max_len=1500, new_max=1000, heads=12,
             kv_heads=4, d=64, rot=64, inter=True, scaled=False, norm=False, page=64),
        # The history of one request, for the next chunk of its prompt.
        dict(name="read8-chunk", op="read8", n_req=1, max_len=6001, heads=32, kv_heads=8, d=128,
             page=16),
        # A batch's histories, handed on to a call that takes dense keys and values.
        dict(name="read8-batch", op="read8", n_req=64, max_len=16384, heads=32, kv_heads=8, d=128,
             page=64),
        # Few short requests: latency.
        dict(name="decode8-short", op="decode8", n_req=16, max_len=2000, n_q=1, heads=32,
             kv_heads=8, d=128, page=16, window=0),
        # A windowed layer of small heads, three new tokens each (two of them drafts).
        dict(name="decode8-window", op="decode8", n_req=60, max_len=9000, n_q=3, heads=12,
             kv_heads=4, d=64, page=32, window=4096),
        # An ordinary batch: 128 requests of up to 8K tokens.
        dict(name="decode8-batch", op="decode8", n_req=128, max_len=8192, n_q=1, heads=32,
             kv_heads=8, d=128, page=64, window=0),
        # Two long histories, the longer of 1M tokens, four new tokens each.
        dict(name="decode8-1m", op="decode8", n_req=2, max_len=1048576, n_q=4, heads=32,
             kv_heads=8, d=128, page=128, window=0),
        # A few users of one short system prompt.
        dict(name="prefix-few", op="prefix", n_groups=1, per_group=8, prefix=1001, max_len=300,
             n_q=1, heads=32, kv_heads=8, d=128, page=16, bf16=True),
        # An ordinary batch on one long system prompt.
        dict(name="prefix-batch", op="prefix", n_groups=1, per_group=128, prefix=8192,
             max_len=2048, n_q=1, heads=32, kv_heads=8, d=128, page=64, bf16=True),
        # Several documents, each with its questions, three new tokens at a time.
        dict(name="prefix-documents", op="prefix", n_groups=5, per_group=24, prefix=20000,
             max_len=500, n_q=3, heads=12, kv_heads=4, d=64, page=32, bf16=False),
        # Many samples drawn from one long prompt.
        dict(name="prefix-samples", op="prefix", n_groups=1, per_group=512, prefix=32768,
             max_len=600, n_q=1, heads=32, kv_heads=8, d=128, page=128, bf16=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append8", "read8", "decode8", "decode8", "prefix", "prefix"])
    page = rng.choice([16, 32, 64, 128, 256])
    d = rng.choice([64, 128])
    heads, kv_heads = rng.choice([(1, 1), (4, 2), (8, 8), (8, 1), (12, 4), (16, 16), (32, 8),
                                  (32, 32), (64, 8)])
    if op == "append8":
        n_req = _log(rng, 1, 256)
        return dict(op=op, n_req=n_req, max_len=_log(rng, 1, 8000),
                    new_max=_log(rng, 1, max(1, 8192 // n_req)), heads=heads, kv_heads=kv_heads,
                    d=d, rot=rng.choice([16, 32, 48, 64]), inter=rng.random() < 0.5,
                    scaled=rng.random() < 0.5, norm=rng.random() < 0.7, page=page)
    if op == "read8":
        n_req = _log(rng, 1, 256)
        most = (1 << 20) * 1024 // (n_req * kv_heads * d)
        return dict(op=op, n_req=n_req, max_len=_log(rng, 1, max(2, min(most, 1 << 17))),
                    heads=heads, kv_heads=kv_heads, d=d, page=page)
    if op == "decode8":
        n_req = _log(rng, 1, 256)
        # Keys times head width up to the batch case's, one in six longer.
        most = (1 << 20) * 1024 // (n_req * kv_heads * d)
        most = min(most, 1 << 20) if rng.random() < 0.17 else min(most, 1 << 14)
        return dict(op=op, n_req=n_req, max_len=_log(rng, 1, max(2, most)),
                    n_q=rng.choice([1, 1, 1, 2, 3, 4, 8]), heads=heads, kv_heads=kv_heads, d=d,
                    page=page, window=0 if rng.random() < 0.7 else _log(rng, 1, 4096))
    n_q = rng.choice([1, 1, 1, 2, 4, 8])
    n_groups, per_group = _log(rng, 1, 8), _log(rng, 2, 256)
    # Rows times prefix times head width up to half of the largest case's.
    most = 512 * 32 * 32768 * 128 // (2 * n_groups * per_group * n_q * heads * d)
    own_most = (1 << 20) * 512 // (n_groups * per_group * kv_heads * d)
    return dict(op=op, n_groups=n_groups, per_group=per_group,
                prefix=_log(rng, 1, max(2, min(most, 65536 // n_groups))),
                max_len=_log(rng, 1, max(2, min(own_most, 2048))), n_q=n_q, heads=heads,
                kv_heads=kv_heads, d=d, page=page, bf16=rng.random() < 0.5)


# ------------------------------------------------------------------ the cases' sizes

def _n_req(case):
    return case["n_req"] if "n_req" in case else case["n_groups"] * case["per_group"]


def _lens(case):
    """The lengths of the cached histories: from 1 up to max_len, the mean a
    third of it; the new tokens are among them where they attend."""
    n = _n_req(case)
    u = (np.arange(n) + 1.0) / n
    return np.maximum(case.get("n_q", 1), np.round(case["max_len"] * u * u)).astype(np.int64)


def _prefixes(case):
    """The prefix lengths of the groups: the longest first, then shorter ones."""
    u = 1.0 - 0.5 * np.arange(case["n_groups"]) / case["n_groups"]
    return np.maximum(1, np.round(case["prefix"] * u)).astype(np.int64)


def _news(case):
    """New tokens per request, up to new_max; every 16th request is idle."""
    n = case["n_req"]
    u = (np.arange(n) + 1.0) / n
    x = np.ceil(case["new_max"] * u * u).astype(np.int64)
    x[15::16] = 0
    return x


def _ceil(a, b):
    return -(-a // b)


def _tokens(case):
    """Rows of a step's token tensors: the new tokens, padded to a multiple of 8."""
    return max(8, _ceil(int(_news(case).sum()), 8) * 8)


def _freqs(case):
    """Rotary frequencies in radians per position, fp64, and the factor on
    cos and sin: the plain geometric set, or one stretched 8 times where the
    wavelength is long, blended between 1 and 32 turns in 4096 positions."""
    R = case["rot"]
    f = BASE ** (-np.arange(0, R, 2, dtype=np.float64) / R)
    if not case["scaled"]:
        return f, 1.0
    turns = 4096 * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    return f * keep + f / 8.0 * (1.0 - keep), 0.1 * math.log(8.0) + 1.0


def _phases(f):
    """The frequencies as turns per position in units of 2^-64 (int64, wrapped)."""
    x = f / (2 * math.pi)
    x = x - np.floor(x)
    hi = np.floor(x * 2.0 ** 32)
    lo = np.floor((x * 2.0 ** 32 - hi) * 2.0 ** 32)
    return torch.from_numpy(((hi.astype(np.uint64) << np.uint64(32))
                             | lo.astype(np.uint64)).view(np.int64).copy())


def work(case):
    H, Hkv, d = case["heads"], case["kv_heads"], case["d"]
    op = case["op"]
    if op == "append8":
        rows = int(_news(case).sum())
        return {"bytes": rows * (4 * H * d + 4 * Hkv * d + 2 * Hkv * (d + 1) + 12),
                "flops": 12 * rows * (H + Hkv) * d}
    ln = _lens(case)
    if op == "read8":
        return {"bytes": int(ln.sum()) * Hkv * (6 * d + 2), "flops": 2 * int(ln.sum()) * Hkv * d}
    nq, n = case["n_q"], _n_req(case)
    if op == "decode8":
        w = case["window"]
        seen = np.minimum(ln, w + nq - 1) if w else ln
        pairs = sum(int((np.minimum(ln - nq + j + 1, w) if w else ln - nq + j + 1).sum())
                    for j in range(nq))
        return {"bytes": int(seen.sum()) * Hkv * (2 * d + 2) + n * nq * H * (d * 6 + 4),
                "flops": 4 * d * H * pairs}
    pre = _prefixes(case)
    pairs = sum(int((ln - nq + j + 1).sum()) for j in range(nq))
    pairs += int(pre.sum()) * case["per_group"] * nq
    return {"bytes": int(pre.sum() + ln.sum()) * Hkv * d * 4
            + n * nq * H * (d * (4 if case["bf16"] else 6) + 4), "flops": 4 * d * H * pairs}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    return g, np.random.default_rng(int(seed) * 104729 + 7)


def _tables(lens, ps, r, slack=3):
    """Pages dealt out in random order to each list of lengths: the block
    tables (-1 behind each row's last page) and the number of pages."""
    n_pages = sum(int(_ceil(ln, ps).sum()) for ln in lens) + slack
    ids, at, tables = r.permutation(n_pages).astype(np.int32), 0, []
    for ln in lens:
        have = _ceil(ln, ps)
        table = np.full((len(ln), int(have.max())), -1, dtype=np.int32)
        mine = np.arange(table.shape[1])[None, :] < have[:, None]
        table[mine] = ids[at:at + int(have.sum())]
        at += int(have.sum())
        tables.append(torch.from_numpy(table).to(DEV))
    return tables, n_pages


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def _randn(shape, g, dtype, scale=1.0):
    out = torch.empty(shape, device=DEV, dtype=dtype)
    out.normal_(0.0, scale, generator=g)
    return out


def _codes(n_pages, ps, Hkv, d, g):
    """Quantised pages: codes as rows whose largest entry is near the top of
    the type have them, and scales that differ from token to token."""
    c = _randn((n_pages, ps, Hkv, d), g, torch.bfloat16, 110.0).clamp_(-448.0, 448.0).to(CODE)
    e = torch.randint(127 - 8, 127 - 5, (n_pages, Hkv, ps), device=DEV, dtype=torch.uint8,
                      generator=g)
    return c, e.view(SCALE)


def prepare(case, seed):
    g, r = _gen(seed)
    s = {"case": case}
    op, ps, H, Hkv, d = (case[k] for k in ("op", "page", "heads", "kv_heads", "d"))
    n = _n_req(case)
    order = r.permutation(n)
    ln = _lens(case)[order]
    if op == "append8":
        nw = _news(case)[order]
        T = _tokens(case)
        # q, k and v are views of one packed projection; a few of its columns are large.
        qkv = _randn((T, H + 2 * Hkv, d), g, torch.bfloat16, 1.5)
        qkv[:, :, ::29] *= 8.0
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        f, s["mscale"] = _freqs(case)
        s["freqs"] = torch.from_numpy(f).to(DEV)
        s["phases"] = _phases(f).to(DEV)
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"] = _randn((d,), g, torch.float32, 0.2) + 1.0
            s["kw"] = _randn((d,), g, torch.float32, 0.2) + 1.0
        # The slots and positions that an extend gave, and the pages.
        (table,), n_pages = _tables([ln + nw], ps, r, 40)
        table = table.cpu().numpy()
        cu = np.concatenate([[0], np.cumsum(nw)])
        t = np.arange(T)
        req = np.minimum(np.searchsorted(cu[1:], t, side="right"), n - 1)
        real = t < cu[-1]
        pos = np.where(real, ln[req] + t - cu[req], 0)
        slot = np.where(real, table[req, pos // ps].astype(np.int64) * ps + pos % ps, -1)
        s["slots"], s["pos"] = torch.from_numpy(slot).to(DEV), _i32(pos)
        for name in ("kc", "vc"):
            s[name] = torch.zeros((n_pages, ps, Hkv, d), device=DEV, dtype=torch.uint8).view(CODE)
        for name in ("ks", "vs"):
            s[name] = torch.full((n_pages, Hkv, ps), 127, device=DEV, dtype=torch.uint8).view(SCALE)
        s["qo"] = torch.zeros((T, H, d), device=DEV, dtype=torch.bfloat16)
        return s
    s["lens"] = _i32(ln)
    if op in ("read8", "decode8"):
        (s["table"],), n_pages = _tables([ln], ps, r)
        s["kc"], s["ks"] = _codes(n_pages, ps, Hkv, d, g)
        s["vc"], s["vs"] = _codes(n_pages, ps, Hkv, d, g)
        if op == "read8":
            s["tokens"] = int(ln.sum())
            s["cu"] = _i32(np.concatenate([[0], np.cumsum(ln)]))
        else:
            s["q"] = _randn((n * case["n_q"], H, d), g, torch.bfloat16, 1.5)
        return s
    pre = _prefixes(case)[r.permutation(case["n_groups"])]
    (s["table"], s["ptable"]), n_pages = _tables([ln, pre], ps, r)
    s["plens"] = _i32(pre)
    s["cu_req"] = _i32(np.arange(case["n_groups"] + 1) * case["per_group"])
    s["kc"] = _randn((n_pages, ps, Hkv, d), g, torch.bfloat16)
    s["vc"] = _randn((n_pages, ps, Hkv, d), g, torch.bfloat16)
    s["q"] = _randn((n * case["n_q"], H, d), g, torch.bfloat16, 1.5)
    return s


# ------------------------------------------------------------------ plain forms

def _cos_sin(s, pos):
    a = pos.to(torch.float64)[:, None] * s["freqs"][None, :]
    return ((torch.cos(a) * s["mscale"]).float()[:, None, :],
            (torch.sin(a) * s["mscale"]).float()[:, None, :])


def _norm_rope(x, w, cos, sin, case):
    y, R = x.float(), case["rot"]
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
    if case["inter"]:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((rot, y[..., R:]), -1)


def _quantise(y):
    """Codes, and the scale's exponent plus 127, of each row of y (fp32)."""
    m, e = torch.frexp(y.abs().amax(-1, keepdim=True))  # amax = m 2^e, m in [1/2, 1)
    e = (e - 9 + (m > 0.875)).clamp(-117, 120)
    return torch.ldexp(y, -e).to(CODE), (e + 127).to(torch.uint8)[..., 0]


def _plain_append(s):
    case = s["case"]
    cos, sin = _cos_sin(s, s["pos"])
    at = torch.nonzero(s["slots"] >= 0).flatten()
    sl = s["slots"][at]
    page, row = sl // case["page"], sl % case["page"]
    for x, c, e in ((_norm_rope(s["k"], s["kw"], cos, sin, case), "kc", "ks"),
                    (s["v"].float(), "vc", "vs")):
        code, exp = _quantise(x[at])
        s[c].view(torch.uint8)[page, row] = code.view(torch.uint8)
        s[e].view(torch.uint8)[page, :, row] = exp
    s["qo"][at] = _norm_rope(s["q"], s["qw"], cos, sin, case)[at].to(torch.bfloat16)
    return s["qo"], s["kc"], s["vc"], s["ks"], s["vs"]


def _values(codes, scales):
    """What codes [..., ps, kv_heads, d] with scales [..., kv_heads, ps] stand for, in fp32."""
    return codes.float() * scales.float().transpose(-1, -2)[..., None]


def _plain_read(s):
    ps, cu = s["case"]["page"], s["cu"].long()
    t = torch.arange(s["tokens"], device=DEV)
    req = torch.searchsorted(cu[1:], t, right=True)
    pos = s["lens"].long()[req] - (cu[req + 1] - t)
    page, row = s["table"][req, pos // ps].long(), pos % ps
    out = []
    for c, e in (("kc", "ks"), ("vc", "vs")):
        scale = s[e].view(torch.uint8)[page, :, row].view(SCALE).float()
        code = s[c].view(torch.uint8)[page, row].view(CODE).float()
        out.append((code * scale[..., None]).to(torch.bfloat16))
    return tuple(out)


def _plain_pages(s, table, side):
    """The pages of a table as [rows of it, kv_heads, keys, d] in fp32."""
    ids = table.long().clamp(min=0)
    c = s[side + "c"]
    if c.dtype == CODE:
        x = _values(c.view(torch.uint8)[ids].view(CODE),
                    s[side + "s"].view(torch.uint8)[ids].view(SCALE))
    else:
        x = c[ids].float()
    return x.flatten(1, 2).transpose(1, 2)


def _plain_decode(s):
    case = s["case"]
    nq, H, Hkv, d, w = (case[k] for k in ("n_q", "heads", "kv_heads", "d", "window"))
    n, L = s["table"].shape[0], s["table"].shape[1] * case["page"]
    q = s["q"].view(n, nq, Hkv, H // Hkv, d).permute(0, 2, 1, 3, 4).float()
    x = torch.matmul(q.reshape(n, Hkv, -1, d), _plain_pages(s, s["table"], "k").transpose(2, 3))
    at = torch.arange(L, device=DEV)[None, None, :]
    qp = s["lens"].long()[:, None, None] - nq + torch.arange(nq, device=DEV)[None, :, None]
    ok = at <= qp
    if w:
        ok = ok & (at > qp - w)
    x = (x * (1.0 / math.sqrt(d))).view(n, Hkv, nq, H // Hkv, L)
    x = x.masked_fill(~ok[:, None, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    # Keys outside a row's are zeros of p; what their pages hold is finite here.
    o = torch.matmul(p.reshape(n, Hkv, -1, L), _plain_pages(s, s["table"], "v"))
    o = o.view(n, Hkv, nq, H // Hkv, d) / l
    lse = (m + torch.log(l)).squeeze(-1)
    return (o.permute(0, 2, 1, 3, 4).reshape(n * nq, H, d),
            lse.permute(0, 2, 1, 3).reshape(n * nq, H))


def _plain_prefix(s):
    case = s["case"]
    nq, H, Hkv, d = (case[k] for k in ("n_q", "heads", "kv_heads", "d"))
    G, per, n = case["n_groups"], case["per_group"], _n_req(case)
    g, ps = H // Hkv, case["page"]
    Lp, L = s["ptable"].shape[1] * ps, s["table"].shape[1] * ps
    q = s["q"].view(n, nq, Hkv, g, d).permute(0, 2, 1, 3, 4).float() * (1.0 / math.sqrt(d))
    # The prefix: [groups, kv heads, rows of the group, keys].
    qg = q.reshape(G, per, Hkv, nq * g, d).transpose(1, 2).reshape(G, Hkv, per * nq * g, d)
    x = torch.matmul(qg, _plain_pages(s, s["ptable"], "k").transpose(2, 3))
    at = torch.arange(Lp, device=DEV)[None, None, None, :]
    x.masked_fill_(at >= s["plens"].long()[:, None, None, None], float("-inf"))
    # The requests' own keys.
    y = torch.matmul(q.reshape(n, Hkv, nq * g, d), _plain_pages(s, s["table"], "k").transpose(2, 3))
    qp = s["lens"].long()[:, None, None] - nq + torch.arange(nq, device=DEV)[None, :, None]
    ok = torch.arange(L, device=DEV)[None, None, :] <= qp
    y = y.view(n, Hkv, nq, g, L).masked_fill_(~ok[:, None, :, None, :], float("-inf"))
    y = y.view(n, Hkv, nq * g, L)

    def by_group(z):
        return z.reshape(G, per, Hkv, nq * g, -1).transpose(1, 2).reshape(G, Hkv, per * nq * g, -1)

    m = torch.maximum(x.amax(-1, keepdim=True), by_group(y.amax(-1, keepdim=True)))
    own_m = m.view(G, Hkv, per, nq * g, 1).transpose(1, 2).reshape(n, Hkv, nq * g, 1)
    p, r = torch.exp_(x.sub_(m)), torch.exp_(y.sub_(own_m))
    l = p.sum(-1, keepdim=True) + by_group(r.sum(-1, keepdim=True))
    o = torch.matmul(p, _plain_pages(s, s["ptable"], "v"))
    o = (o + by_group(torch.matmul(r, _plain_pages(s, s["table"], "v")))) / l

    def rows(z):  # to [tokens, heads, ...]
        z = z.view(G, Hkv, per, nq, g, -1).permute(0, 2, 3, 1, 4, 5)
        return z.reshape(n * nq, H, -1)

    out = rows(o)
    return out.to(torch.bfloat16) if case["bf16"] else out, rows(m + torch.log(l))[..., 0]


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        return _own(s, case, op)
    if op == "append8":
        return _plain_append(s)
    if op == "read8":
        return _plain_read(s)
    return _plain_decode(s) if op == "decode8" else _plain_prefix(s)


# ------------------------------------------------------------------ the package's calls

def _own(s, case, op):
    import blockwise_online_softmax_gb300 as ra

    if op == "append8":
        ra.ra_paged_append_fp8(s["q"], s["k"], s["v"], s["phases"], s["kc"], s["vc"], s["ks"],
                               s["vs"], s["slots"], s["pos"], q_weight=s["qw"], k_weight=s["kw"],
                               eps=1e-6, interleaved=case["inter"], mscale=s["mscale"],
                               q_out=s["qo"])
        return s["qo"], s["kc"], s["vc"], s["ks"], s["vs"]
    if op == "read8":
        return ra.ra_paged_read_fp8(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"],
                                    s["cu"], tokens=s["tokens"])
    if op == "decode8":
        return ra.ra_paged_decode_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"],
                                      s["lens"], window=case["window"])
    out = torch.empty_like(s["q"]) if case["bf16"] else None
    return ra.ra_paged_decode_prefix(s["q"], s["kc"], s["vc"], s["ptable"], s["plens"],
                                     s["cu_req"], s["table"], s["lens"], out=out)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_turn(x, w, s, case):
    x, R = x.double(), case["rot"]
    if w is not None:
        x = x / ((x * x).sum(-1, keepdim=True) / case["d"] + 1e-6).sqrt() * w.double()
    turn = s["pos"].double().view(-1, 1, 1) * s["freqs"]
    e = torch.polar(torch.full_like(turn, s["mscale"]), turn)
    part = x[..., :R]
    if case["inter"]:
        z = torch.view_as_complex(part.unflatten(-1, (R // 2, 2)).contiguous()) * e
        z = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(part[..., :R // 2].contiguous(), part[..., R // 2:].contiguous()) * e
        z = torch.cat((z.real, z.imag), -1)
    out = x.clone()
    out[..., :R] = z
    return out


def _exact_codes(x):
    """Rows in 64 bits to (the codes' values, the scales' values): the largest
    entry fits 448 scales, codes are multiples of the type's step, halves to even."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)  # (log2 is rounded)
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(-117, 120)
    y = x / torch.exp2(e)
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(y.abs(), min=1e-300))),
                                  min=-6.0) - 3.0)
    return torch.round(y / step) * step, torch.exp2(e)[..., 0]


def _exact_append(s, case):
    ps, slots = case["page"], s["slots"].cpu()
    q = _exact_turn(s["q"], s["qw"], s, case).cpu()
    out = [s["qo"].double().cpu()]
    real = torch.nonzero(slots >= 0).flatten()
    out[0][real] = q[real]
    scales = []
    for x, c, e in ((_exact_turn(s["k"], s["kw"], s, case), "kc", "ks"), (s["v"].double(), "vc", "vs")):
        val, scale = (y.cpu() for y in _exact_codes(x))
        pages, sc = s[c].cpu().double(), s[e].cpu().double()
        pages.flatten(0, 1)[slots[real]] = val[real]
        sc.transpose(1, 2)[slots[real] // ps, slots[real] % ps] = scale[real]
        out.append(pages)
        scales.append(sc)
    return tuple(out + scales)


def _exact_rows(s, table, i, length, ps, side):
    """The first `length` keys (or values) of row i of a table, in 64 bits."""
    ids = table[i, :math.ceil(length / ps)].long()
    if s["kc"].dtype == torch.bfloat16:
        return s[side + "c"][ids].double().flatten(0, 1)[:length]
    x = s[side + "c"].view(torch.uint8)[ids].view(CODE).double()
    e = s[side + "s"].view(torch.uint8)[ids].double() - 127.0
    return (x * torch.exp2(e).permute(0, 2, 1).unsqueeze(-1)).flatten(0, 1)[:length]


def _exact_read(s, case):
    out = []
    for side in ("k", "v"):
        x = [_exact_rows(s, s["table"], i, n, case["page"], side) for i, n in enumerate(s["lens"].tolist())]
        out.append(torch.cat(x))
    return tuple(out)


def _exact_attend(s, case):
    H, Hkv, d, nq = (case[k] for k in ("heads", "kv_heads", "d", "n_q"))
    g, ps, w = H // Hkv, case["page"], case.get("window", 0)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    plens = s["plens"].tolist() if "plens" in s else []
    shared = None
    for i, n in enumerate(s["lens"].tolist()):
        k, v = (_exact_rows(s, s["table"], i, n, ps, side) for side in "kv")
        P = 0
        if plens:
            grp = i // case["per_group"]
            if i % case["per_group"] == 0:
                shared = [_exact_rows(s, s["ptable"], grp, plens[grp], ps, side) for side in "kv"]
            P = plens[grp]
            k, v = torch.cat((shared[0], k)), torch.cat((shared[1], v))
        for j in range(nq):
            hi = P + n - nq + j + 1
            lo = max(0, hi - w) if w else 0
            q = s["q"][i * nq + j].double().view(Hkv, g, d)
            x = torch.einsum("hgd,thd->hgt", q, k[lo:hi]) / math.sqrt(d)
            lse[i * nq + j] = torch.logsumexp(x, -1).flatten()
            out[i * nq + j] = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), v[lo:hi]).reshape(H, d)
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append8":
        return _exact_append(s, case)
    if case["op"] == "read8":
        return _exact_read(s, case)
    if work(case)["flops"] > 4e11 or s["q"].shape[0] > 20000:  # fp64 runs at a thousandth of the bf16 rate
        return None
    return _exact_attend(s, case)
