"""What the serving and training operators around the attention kernels are
measured on: page bookkeeping (`ra_paged_extend`, `ra_paged_release`), the
per-head norm with rotary positions and its gradient (`ra_qk_norm_rope`,
`ra_qk_norm_rope_backward`), the same with the key/value pages written
(`ra_paged_append`), and attention over the pages (`ra_paged_decode`).

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


def listed():
    return [
        # One step of a serving loop: a new token for most of 256 requests.
        dict(name="extend-step", op="extend", n_req=256, max_len=8000, new_max=1, page=16),
        # Prompts arrive: 64 requests of up to 16K new tokens each.
        dict(name="extend-prompts", op="extend", n_req=64, max_len=1500, new_max=16384, page=64),
        # A quarter of a small batch has finished.
        dict(name="release-step", op="release", n_req=64, max_len=4000, every=4, page=16),
        # Half of a large batch is dropped at once.
        dict(name="release-half", op="release", n_req=2048, max_len=8000, every=2, page=16),
        # The 128K-token GQA ring's q and k before the ring, zigzag order.
        dict(name="rope-ring-128k", op="rope", T=131072, heads=32, kv_heads=8, d=128, rot=128,
             inter=False, scaled=False, norm=True, layout="zigzag", P=16, f32=False),
        # The gradients of the same, after the backward ring.
        dict(name="rope-ring-128k-grad", op="rope_grad", T=131072, heads=32, kv_heads=8, d=128,
             rot=128, inter=False, scaled=False, norm=True, layout="zigzag", P=16, f32=False),
        # fp32 training of a short odd sequence, interleaved pairs, half the head rotated.
        dict(name="rope-odd-f32-grad", op="rope_grad", T=4099, heads=8, kv_heads=8, d=64, rot=32,
             inter=True, scaled=True, norm=True, layout="contiguous", P=1, f32=True),
        # One token of each of 256 requests goes into the pages.
        dict(name="append-step", op="append", n_req=256, max_len=8000, new_max=1, heads=32,
             kv_heads=8, d=128, rot=128, inter=False, scaled=True, norm=True, page=16),
        # Prompts of up to 2K tokens go into the pages, no norm, d = 64.
        dict(name="append-prompts", op="append", n_req=24, max_len=100, new_max=2048, heads=12,
             kv_heads=4, d=64, rot=64, inter=True, scaled=False, norm=False, page=64),
        # The smallest decode: 16 short requests, small pages.
        dict(name="decode-short", op="decode", n_req=16, max_len=2000, n_q=1, heads=32, kv_heads=8,
             d=128, page=16, window=0),
        # An ordinary batch: 128 requests of up to 8K tokens.
        dict(name="decode-batch", op="decode", n_req=128, max_len=8192, n_q=1, heads=32,
             kv_heads=8, d=128, page=64, window=0),
        # Two long histories, the longer of 1M tokens, four new tokens each.
        dict(name="decode-1m", op="decode", n_req=2, max_len=1048576, n_q=4, heads=32, kv_heads=8,
             d=128, page=128, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "release", "rope", "rope_grad", "append", "decode", "decode"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if op == "extend":
        if rng.random() < 0.5:
            return dict(op=op, n_req=_log(rng, 1, 4096), max_len=_log(rng, 1, 20000),
                        new_max=rng.randint(1, 8), page=page)
        return dict(op=op, n_req=_log(rng, 1, 64), max_len=_log(rng, 1, 20000),
                    new_max=_log(rng, 9, 16384), page=page)
    if op == "release":
        return dict(op=op, n_req=_log(rng, 1, 2048), max_len=_log(rng, 1, 8000),
                    every=rng.randint(1, 5), page=page if page > 8 else 16)
    d = rng.choice([64, 128])
    heads, kv_heads = rng.choice([(1, 1), (4, 2), (8, 8), (8, 1), (12, 4), (16, 16), (32, 8),
                                  (32, 32), (64, 8)])
    if op in ("rope", "rope_grad"):
        P, layout = rng.choice([(1, "contiguous"), (8, "contiguous"), (4, "zigzag"),
                                (16, "zigzag"), (8, "striped")])
        f32 = rng.random() < 0.3
        top = 131072 * 40 * 128 // ((heads + kv_heads) * d * (2 if f32 else 1))
        T = max(1, _log(rng, 1, min(top, 131072)) // (2 * P)) * 2 * P
        if P == 1:
            T = max(1, T - rng.randint(0, 1))
        return dict(op=op, T=T, heads=heads, kv_heads=kv_heads, d=d,
                    rot=rng.choice([16, 32, 48, 64] + ([96, 128] if d == 128 else [])),
                    inter=rng.random() < 0.5, scaled=rng.random() < 0.5, norm=rng.random() < 0.7,
                    layout=layout, P=P, f32=f32)
    if op == "append":
        n_req = _log(rng, 1, 256)
        return dict(op=op, n_req=n_req, max_len=_log(rng, 1, 8000),
                    new_max=_log(rng, 1, max(1, 8192 // n_req)), heads=heads, kv_heads=kv_heads,
                    d=d, rot=rng.choice([16, 32, 48, 64]), inter=rng.random() < 0.5,
                    scaled=rng.random() < 0.5, norm=rng.random() < 0.7, page=page)
    n_req = _log(rng, 1, 256)
    # Keys times head width up to the batch case's, one in six longer.
    most = (1 << 20) * 1024 // (n_req * kv_heads * d)
    most = min(most, 1 << 20) if rng.random() < 0.17 else min(most, 1 << 14)
    g = heads // kv_heads
    return dict(op=op, n_req=n_req, max_len=_log(rng, 1, max(2, most)),
                n_q=rng.choice([1, 1, 1, 2, 3, min(5, 128 // g), 128 // g if g >= 4 else 16]),
                heads=heads, kv_heads=kv_heads, d=d, page=page,
                window=0 if rng.random() < 0.7 else _log(rng, 1, 4096))


# ------------------------------------------------------------------ the cases' sizes

def _lens(case):
    """The lengths of the cached histories: from 1 (0 for the last of several
    when bookkeeping) up to max_len, the mean a third of it."""
    n = case["n_req"]
    u = (np.arange(n) + 1.0) / n
    return np.maximum(1, np.round(case["max_len"] * u * u)).astype(np.int64)


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


def _layout_pos(case):
    """Position held by each row of a ring tensor."""
    T, P = case["T"], case["P"]
    c, h = T // P, T // P // 2
    b, r = np.divmod(np.arange(T, dtype=np.int64), c)
    if case["layout"] == "zigzag":
        return np.where(r < h, b * h + r, (2 * P - 1 - b) * h + r - h)
    if case["layout"] == "striped":
        return r * P + b
    return b * c + r


def work(case):
    op = case["op"]
    if op in ("extend", "release"):
        n, ps = case["n_req"], case["page"]
        ln = _lens(case)
        if op == "release":
            pages = int(_ceil(ln, ps)[::case["every"]].sum())
            return {"bytes": 8 * pages + 12 * n + 8, "flops": 0}
        nw = _news(case)
        pages = int((_ceil(ln + nw, ps) - _ceil(ln, ps)).sum())
        return {"bytes": 8 * pages + 12 * _tokens(case) + 16 * n + 12, "flops": 0}
    H, Hkv, d = case["heads"], case["kv_heads"], case["d"]
    if op in ("rope", "rope_grad"):
        rows, e = case["T"] * (H + Hkv), 4 if case["f32"] else 2
        if op == "rope":
            return {"bytes": rows * d * 2 * e, "flops": 12 * rows * d}
        return {"bytes": rows * d * (4 + 2 * e), "flops": 24 * rows * d}
    if op == "append":
        rows = int(_news(case).sum())
        return {"bytes": rows * (2 * H + 4 * Hkv) * d * 2 + 12 * rows,
                "flops": 12 * rows * (H + Hkv) * d}
    ln, nq, w = _lens_q(case), case["n_q"], case["window"]
    seen = np.minimum(ln, w + nq - 1) if w else ln
    keys = int(seen.sum())
    pairs = sum(int((np.minimum(ln - nq + j + 1, w) if w else ln - nq + j + 1).sum())
                for j in range(nq))
    return {"bytes": keys * Hkv * d * 4 + case["n_req"] * nq * H * (d * 6 + 4),
            "flops": 4 * d * H * pairs}


def _lens_q(case):
    """Decode: lengths that include the new tokens."""
    return np.maximum(_lens(case), case["n_q"])


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    return g, np.random.default_rng(int(seed) * 104729 + 7)


def _pool(ln, total, ps, width, slack, r):
    """Pages dealt out in random order: the block table for lengths `ln`
    (-1 behind each row's last page), the free list and its count."""
    n = len(ln)
    have = _ceil(ln, ps)
    n_pages = int(_ceil(total, ps).sum()) + slack
    ids = r.permutation(n_pages).astype(np.int32)
    used = int(have.sum())
    table = np.full((n, width), -1, dtype=np.int32)
    table[np.arange(width)[None, :] < have[:, None]] = ids[:used]
    free = np.full(n_pages, -1, dtype=np.int32)
    free[:n_pages - used] = ids[used:]
    return n_pages, torch.from_numpy(table).to(DEV), torch.from_numpy(free).to(DEV), n_pages - used


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def _randn(shape, g, dtype, scale=1.0):
    out = torch.empty(shape, device=DEV, dtype=dtype)
    out.normal_(0.0, scale, generator=g)
    return out


def _rope_inputs(case, s, rows, dtype, g):
    H, Hkv, d = case["heads"], case["kv_heads"], case["d"]
    # q, k and v are views of one packed projection.
    qkv = _randn((rows, H + 2 * Hkv, d), g, dtype, 1.5)
    s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    f, s["mscale"] = _freqs(case)
    s["freqs"] = torch.from_numpy(f).to(DEV)
    s["phases"] = _phases(f).to(DEV)
    s["qw"] = s["kw"] = None
    if case["norm"]:
        s["qw"] = _randn((d,), g, torch.float32, 0.2) + 1.0
        s["kw"] = _randn((d,), g, torch.float32, 0.2) + 1.0


def prepare(case, seed):
    g, r = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("rope", "rope_grad"):
        dtype = torch.float32 if case["f32"] else torch.bfloat16
        T, H, Hkv, d = case["T"], case["heads"], case["kv_heads"], case["d"]
        _rope_inputs(case, s, T, dtype, g)
        s["pos"] = torch.from_numpy(_layout_pos(case)).to(DEV)
        if op == "rope_grad":
            s["dqo"] = _randn((T, H, d), g, torch.float32)
            s["dko"] = _randn((T, Hkv, d), g, torch.float32)
        return s
    ps = case["page"]
    order = r.permutation(case["n_req"])
    if op == "decode":
        H, Hkv, d, nq = case["heads"], case["kv_heads"], case["d"], case["n_q"]
        ln = _lens_q(case)[order]
        width = int(_ceil(int(ln.max()), ps))
        n_pages, s["table"], _, _ = _pool(ln, ln, ps, width, 3, r)
        s["lens"] = _i32(ln)
        s["width"] = width
        s["kc"] = _randn((n_pages, ps, Hkv, d), g, torch.bfloat16)
        s["vc"] = _randn((n_pages, ps, Hkv, d), g, torch.bfloat16)
        s["q"] = _randn((case["n_req"] * nq, H, d), g, torch.bfloat16, 1.5)
        return s
    ln = _lens(case)[order]
    if op == "release":
        fin = np.zeros(case["n_req"], dtype=np.int32)
        fin[::case["every"]] = 1
        fin = fin[order]
        width = int(_ceil(case["max_len"], ps)) + 1
        _, s["table"], s["free"], count = _pool(ln, ln, ps, width, 40, r)
        s["lens"], s["fin"], s["count"] = _i32(ln), _i32(fin), _i32([count])
        s["lens_out"], s["count_out"] = torch.empty_like(s["lens"]), torch.empty_like(s["count"])
        return s
    nw = _news(case)[order]
    width = int(_ceil(case["max_len"] + case["new_max"], ps)) + 1
    n_pages, s["table"], s["free"], count = _pool(ln, ln + nw, ps, width, 40, r)
    s["T"] = _tokens(case)
    if op == "extend":
        s["lens"], s["news"], s["count"] = _i32(ln), _i32(nw), _i32([count])
        s["lens_out"], s["count_out"] = torch.empty_like(s["lens"]), torch.empty_like(s["count"])
        return s
    # append: the slots and positions that an extend gave, the pages, and the step's rows.
    _rope_inputs(case, s, s["T"], torch.bfloat16, g)
    cu = np.concatenate([[0], np.cumsum(nw)])
    t = np.arange(s["T"])
    req = np.minimum(np.searchsorted(cu[1:], t, side="right"), case["n_req"] - 1)
    pos = ln[req] + t - cu[req]
    real = t < cu[-1]
    pages = r.permutation(n_pages)[:int(_ceil(ln + nw, ps).sum())]
    first = np.concatenate([[0], np.cumsum(_ceil(ln + nw, ps))])
    page = pages[np.minimum(first[req] + pos // ps, len(pages) - 1)]
    s["slots"] = torch.from_numpy(np.where(real, page * ps + pos % ps, -1).astype(np.int64)).to(DEV)
    s["pos"] = _i32(np.where(real, pos, 0))
    shape = (n_pages, ps, case["kv_heads"], case["d"])
    s["kc"] = torch.zeros(shape, device=DEV, dtype=torch.bfloat16)
    s["vc"] = torch.zeros(shape, device=DEV, dtype=torch.bfloat16)
    s["qo"] = torch.zeros((s["T"], case["heads"], case["d"]), device=DEV, dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms

def _cos_sin(s, pos):
    a = pos.to(torch.float64)[:, None] * s["freqs"][None, :]
    return ((torch.cos(a) * s["mscale"]).float()[:, None, :],
            (torch.sin(a) * s["mscale"]).float()[:, None, :])


def _rotate(y, cos, sin, R, inter):
    if inter:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((rot, y[..., R:]), -1)


def _norm_rope(x, w, cos, sin, case):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
    return _rotate(y, cos, sin, case["rot"], case["inter"]).to(x.dtype)


def _norm_rope_grad(x, w, dy, cos, sin, case):
    gy = _rotate(dy, cos, -sin, case["rot"], case["inter"])
    if w is None:
        return gy.to(x.dtype), None
    y = x.float()
    inv = torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
    hat = y * inv
    dw = (gy * hat).sum(1, dtype=torch.float64).sum(0).float()
    u = gy * w
    return (inv * (u - hat * (u * hat).mean(-1, keepdim=True))).to(x.dtype), dw


def _plain_extend(s):
    ps, T, table, free = s["case"]["page"], s["T"], s["table"], s["free"]
    ln, nw = s["lens"].long(), s["news"].long()
    old, new = (ln + ps - 1) // ps, (ln + nw + ps - 1) // ps
    need = new - old
    first = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    at = s["count"].long() - 1 - (first[:, None] + col - old[:, None])
    fresh = (col >= old[:, None]) & (col < new[:, None])
    table.copy_(torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table))
    s["lens_out"].copy_(ln + nw)
    s["count_out"].copy_(s["count"] - need.sum())
    end = torch.cumsum(nw, 0)
    cu = torch.cat((torch.zeros_like(end[:1]), end))
    t = torch.arange(T, device=DEV)
    req = torch.searchsorted(end, t, right=True).clamp(max=ln.numel() - 1)
    real = t < end[-1]
    pos = torch.where(real, ln[req] + t - cu[req], 0)
    slot = torch.where(real, table[req, pos // ps].long() * ps + pos % ps, -1)
    return table, s["lens_out"], s["count_out"], slot, pos.int(), cu.int()


def _plain_release(s):
    ps, table, free = s["case"]["page"], s["table"], s["free"]
    ln, fin = s["lens"].long(), s["fin"] != 0
    have = torch.where(fin, (ln + ps - 1) // ps, 0)
    first = torch.cumsum(have, 0) - have
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    at = s["count"].long() + first[:, None] + col
    mine = col < have[:, None]
    # Entries that are no page of a finished request go to a place behind the list.
    whole = torch.cat((free, free[:1]))
    whole.scatter_(0, torch.where(mine, at, free.numel()).flatten(), table.flatten())
    free.copy_(whole[:-1])
    s["count_out"].copy_(s["count"] + have.sum())
    s["lens_out"].copy_(torch.where(fin, 0, ln))
    return free, s["lens_out"], s["count_out"]


def _plain_append(s):
    case = s["case"]
    cos, sin = _cos_sin(s, s["pos"])
    real = s["slots"] >= 0
    at = torch.nonzero(real).flatten()
    sl = s["slots"][at]
    H, d = case["kv_heads"], case["d"]
    s["kc"].view(-1, H, d)[sl] = _norm_rope(s["k"], s["kw"], cos, sin, case)[at]
    s["vc"].view(-1, H, d)[sl] = s["v"][at]
    s["qo"][at] = _norm_rope(s["q"], s["qw"], cos, sin, case)[at]
    return s["qo"], s["kc"], s["vc"]


def _plain_decode(s):
    case = s["case"]
    n, nq, H, Hkv, d = (case[k] for k in ("n_req", "n_q", "heads", "kv_heads", "d"))
    L = s["width"] * case["page"]
    ids = s["table"].long().clamp(min=0)
    k = s["kc"][ids].view(n, L, Hkv, d).permute(0, 2, 1, 3).float()
    q = s["q"].view(n, nq, Hkv, H // Hkv, d).permute(0, 2, 1, 3, 4).float()
    x = torch.matmul(q.reshape(n, Hkv, -1, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    at = torch.arange(L, device=DEV)[None, None, :]
    qp = s["lens"].long()[:, None, None] - nq + torch.arange(nq, device=DEV)[None, :, None]
    ok = at <= qp
    if case["window"]:
        ok = ok & (at > qp - case["window"])
    x = x.view(n, Hkv, nq, H // Hkv, L).masked_fill(~ok[:, None, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    v = s["vc"][ids].view(n, L, Hkv, d).permute(0, 2, 1, 3).float()
    o = torch.matmul(p.reshape(n, Hkv, -1, L), v).view(n, Hkv, nq, H // Hkv, d) / l
    lse = (m + torch.log(l)).squeeze(-1)
    return (o.permute(0, 2, 1, 3, 4).reshape(n * nq, H, d),
            lse.permute(0, 2, 1, 3).reshape(n * nq, H))


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        return _own(s, case, op)
    if op == "extend":
        return _plain_extend(s)
    if op == "release":
        return _plain_release(s)
    if op == "append":
        return _plain_append(s)
    if op == "decode":
        return _plain_decode(s)
    cos, sin = _cos_sin(s, s["pos"])
    if op == "rope":
        return (_norm_rope(s["q"], s["qw"], cos, sin, case),
                _norm_rope(s["k"], s["kw"], cos, sin, case))
    dq, dqw = _norm_rope_grad(s["q"], s["qw"], s["dqo"], cos, sin, case)
    dk, dkw = _norm_rope_grad(s["k"], s["kw"], s["dko"], cos, sin, case)
    return dq, dk, dqw, dkw


# ------------------------------------------------------------------ the package's calls

def _own(s, case, op):
    import blockwise_online_softmax_gb300 as ra

    if op == "extend":
        slots, pos, cu, lens, count, _ = ra.ra_paged_extend(
            s["lens"], s["news"], s["table"], s["free"], s["count"], page_size=case["page"],
            tokens=s["T"], lengths_out=s["lens_out"], free_count_out=s["count_out"])
        return s["table"], lens, count, slots, pos, cu
    if op == "release":
        lens, count = ra.ra_paged_release(
            s["lens"], s["fin"], s["table"], s["free"], s["count"], page_size=case["page"],
            lengths_out=s["lens_out"], free_count_out=s["count_out"])
        return s["free"], lens, count
    if op == "decode":
        return ra.ra_paged_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"],
                                  window=case["window"])
    how = dict(q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, interleaved=case["inter"],
               mscale=s["mscale"])
    if op == "append":
        ra.ra_paged_append(s["q"], s["k"], s["v"], s["phases"], s["kc"], s["vc"], s["slots"],
                           s["pos"], q_out=s["qo"], **how)
        return s["qo"], s["kc"], s["vc"]
    how.update(layout=case["layout"], P=case["P"])
    if op == "rope":
        return ra.ra_qk_norm_rope(s["q"], s["k"], s["phases"], **how)
    return ra.ra_qk_norm_rope_backward(s["q"], s["k"], s["phases"], s["dqo"], s["dko"], **how)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_angles(s, pos):
    turn = pos.double().view(-1, 1, 1) * s["freqs"]
    return torch.polar(torch.full_like(turn, s["mscale"]), turn)


def _exact_pairs(x, R, inter):
    part = x[..., :R]
    part = part.unflatten(-1, (R // 2, 2)) if inter else part.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    return torch.view_as_complex(part.contiguous())


def _exact_turn(x, e, R, inter):
    z = torch.view_as_real(_exact_pairs(x, R, inter) * e)
    out = x.clone()
    out[..., :R] = (z if inter else z.transpose(-1, -2)).flatten(-2)
    return out


def _exact_rope(x, w, e, case):
    x = x.double()
    if w is not None:
        x = x / ((x * x).sum(-1, keepdim=True) / case["d"] + 1e-6).sqrt() * w.double()
    return _exact_turn(x, e, case["rot"], case["inter"])


def _exact_rope_grad(x, w, dy, e, case):
    back = _exact_turn(dy.double(), e.conj(), case["rot"], case["inter"])
    if w is None:
        return back, None
    x = x.double()
    rms = ((x * x).sum(-1, keepdim=True) / case["d"] + 1e-6).sqrt()
    dw = (back * x / rms).sum((0, 1))
    u = back * w.double()
    return u / rms - x * (u * x).sum(-1, keepdim=True) / (case["d"] * rms ** 3), dw


def _exact_pages(s, case, op):
    ps = case["page"]
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    ln, top = s["lens"].cpu().numpy().astype(int).copy(), int(s["count"])
    if op == "release":
        for i in np.flatnonzero(s["fin"].cpu().numpy()):
            k = math.ceil(ln[i] / ps)
            free[top:top + k] = table[i, :k]
            top, ln[i] = top + k, 0
        return tuple(torch.from_numpy(x) for x in (free, ln.astype(np.int32),
                                                   np.array([top], np.int32)))
    slots, pos, cu = np.full(s["T"], -1, np.int64), np.zeros(s["T"], np.int32), [0]
    for i, k in enumerate(s["news"].cpu().numpy()):
        for c in range(math.ceil(ln[i] / ps), math.ceil((ln[i] + k) / ps)):
            top -= 1
            table[i, c] = free[top]
        p = np.arange(ln[i], ln[i] + k)
        pos[cu[-1]:cu[-1] + k] = p
        slots[cu[-1]:cu[-1] + k] = table[i, p // ps].astype(np.int64) * ps + p % ps
        ln[i] += k
        cu.append(cu[-1] + int(k))
    return tuple(torch.from_numpy(x) for x in (table, ln.astype(np.int32), np.array([top], np.int32),
                                               slots, pos, np.array(cu, np.int32)))


def _exact_decode(s, case):
    n, nq, H, Hkv, d = (case[k] for k in ("n_req", "n_q", "heads", "kv_heads", "d"))
    out = torch.empty((n * nq, H, d), dtype=torch.float64, device=DEV)
    lse = torch.empty((n * nq, H), dtype=torch.float64, device=DEV)
    for i, length in enumerate(s["lens"].tolist()):
        ids = s["table"][i, :math.ceil(length / case["page"])].long()
        k = s["kc"][ids].flatten(0, 1)[:length]
        v = s["vc"][ids].flatten(0, 1)[:length]
        for j in range(nq):
            hi = length - nq + j + 1
            lo = max(0, hi - case["window"]) if case["window"] else 0
            for h in range(Hkv):
                rows = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
                x = s["q"][i * nq + j, rows].double() @ k[lo:hi, h].double().T / math.sqrt(d)
                lse[i * nq + j, rows] = torch.logsumexp(x, -1)
                out[i * nq + j, rows] = torch.softmax(x, -1) @ v[lo:hi, h].double()
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("extend", "release"):
        return _exact_pages(s, case, op)
    if op == "decode":
        if case["n_req"] * case["n_q"] * case["kv_heads"] > 20000:
            return None
        return _exact_decode(s, case)
    e = _exact_angles(s, s["pos"])
    if op == "rope":
        return _exact_rope(s["q"], s["qw"], e, case), _exact_rope(s["k"], s["kw"], e, case)
    if op == "rope_grad":
        dq, dqw = _exact_rope_grad(s["q"], s["qw"], s["dqo"], e, case)
        dk, dkw = _exact_rope_grad(s["k"], s["kw"], s["dko"], e, case)
        return dq, dk, dqw, dkw
    q, kc, vc = s["qo"].double(), s["kc"].double(), s["vc"].double()
    nk, nq = _exact_rope(s["k"], s["kw"], e, case), _exact_rope(s["q"], s["qw"], e, case)
    here = s["slots"] >= 0
    page, row = (s["slots"] // case["page"])[here], (s["slots"] % case["page"])[here]
    kc[page, row], vc[page, row], q[here] = nk[here], s["v"].double()[here], nq[here]
    return q, kc, vc
