"""Plain 64-bit forms of the page bookkeeping and of the q/k norm with rotary
positions, for the tests (numpy, loops and all)."""
import numpy as np


def extend(lengths, new_tokens, table, free, count, page_size, tokens):
    """The step's outputs, and the table after it: (slots, positions, cu,
    lengths, count, status, table)."""
    n, width = table.shape
    ln = np.maximum(np.asarray(lengths, dtype=np.int64), 0)
    nw = np.maximum(np.asarray(new_tokens, dtype=np.int64), 0)
    table = table.copy()
    need = [-(-(a + b) // page_size) - -(-a // page_size) for a, b in zip(ln, nw)]
    bad = sum(-(-(a + b) // page_size) > width for a, b in zip(ln, nw))
    most = 2 ** 31 - 1  # the status words are int32 and saturate
    status = [min(most, max(0, sum(need) - count)), bad, min(most, max(0, int(nw.sum()) - tokens))]
    slots, pos, cu = np.full(tokens, -1, np.int64), np.zeros(tokens, np.int64), [0]
    if any(status):
        return slots, pos, [0] * (n + 1), ln, count, status, table
    for i in range(n):
        for c in range(-(-ln[i] // page_size), -(-(ln[i] + nw[i]) // page_size)):
            count -= 1
            table[i, c] = free[count]
        for j in range(nw[i]):
            p = ln[i] + j
            pos[cu[-1] + j] = p
            slots[cu[-1] + j] = int(table[i, p // page_size]) * page_size + p % page_size
        cu.append(cu[-1] + int(nw[i]))
    return slots, pos, cu, ln + nw, count, status, table


def release(lengths, finished, table, free, count, page_size):
    free, ln = free.copy(), np.maximum(np.asarray(lengths, dtype=np.int64), 0)
    for i in np.flatnonzero(finished):
        for c in range(-(-ln[i] // page_size)):
            free[count] = table[i, c]
            count += 1
        ln[i] = 0
    return free, ln, count


def pairs(rot, interleaved):
    """Columns (a, b) of each rotated pair."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rope(x, weight, pos, freqs, *, eps, mscale=1.0, interleaved=False):
    """Norm and rotation of x [T, heads, d] at pos [T]; also the size of the
    terms each output is a sum of (|a| + |b| of its pair, times mscale)."""
    y = np.asarray(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    out, size = y.copy(), np.abs(y)
    a, b = pairs(2 * len(freqs), interleaved)
    t = np.asarray(pos, dtype=np.float64)[:, None, None] * freqs
    c, s = mscale * np.cos(t), mscale * np.sin(t)
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    size[..., a] = size[..., b] = abs(mscale) * (np.abs(y[..., a]) + np.abs(y[..., b]))
    return out, size


def rope_grad(x, weight, pos, freqs, dy, *, eps, mscale=1.0, interleaved=False):
    """(dx, dweight) for the loss sum(dy * rope(x)), and the sums of the
    absolute terms of each (the scales of their rounding errors)."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    g, ga = dy.copy(), np.abs(dy)
    a, b = pairs(2 * len(freqs), interleaved)
    t = np.asarray(pos, dtype=np.float64)[:, None, None] * freqs
    c, s = mscale * np.cos(t), mscale * np.sin(t)
    g[..., a] = dy[..., a] * c + dy[..., b] * s
    g[..., b] = dy[..., b] * c - dy[..., a] * s
    ga[..., a] = ga[..., b] = abs(mscale) * (np.abs(dy[..., a]) + np.abs(dy[..., b]))
    if weight is None:
        return g, None, ga, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u, ua = g * weight, ga * np.abs(weight)
    dx = r * (u - x * r * r * (u * x).mean(-1, keepdims=True))
    dxa = r * (ua + np.abs(x) * r * r * (ua * np.abs(x)).mean(-1, keepdims=True))
    return dx, (g * x * r).sum((0, 1)), dxa, (ga * np.abs(x) * r).sum((0, 1))
