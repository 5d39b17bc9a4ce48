"""Plain 64-bit reference of the paged 4-bit KV cache, for tests: the quantiser
in rational arithmetic, page unpacking, the step mask listed row by row, the
attention, and the page plan as a walk over the sequences."""
from fractions import Fraction as F

import numpy as np


def bf16_up(x: F) -> F:
    """The smallest bf16 number >= x (x >= 0)."""
    if x == 0:
        return F(0)
    e = -133
    while F(2) ** e * 256 <= x:
        e += 1
    # x < 256 * 2^e: multiples of 2^e have at most 8 significant bits there
    n = -((-x) // F(2) ** e)
    return n * F(2) ** e


def nearest_even(x: F) -> int:
    f = x.numerator // x.denominator
    r = x - f
    return f + (1 if r > F(1, 2) or (r == F(1, 2) and f % 2) else 0)


def quantise_exact(x):
    """(codes, scale as float, zero point) of one vector in exact arithmetic."""
    if not np.isfinite(x).all():
        return np.zeros(len(x), int), float("nan"), 0
    fx = [F(float(v)) for v in x]
    hi, lo = max(F(0), *fx), min(F(0), *fx)
    s = bf16_up((hi - lo) / 15)
    if s == 0:
        return np.zeros(len(x), int), 0.0, 0
    z = nearest_even(-lo / s)
    return np.array([min(15, max(0, nearest_even(v / s) + z)) for v in fx]), float(s), z


def quantise(x):
    """(codes, scale, zero point) of vectors [..., D] in doubles (finite inputs
    whose span is exact in doubles)."""
    x = np.asarray(x, np.float64)
    hi, lo = np.maximum(x.max(-1), 0), np.minimum(x.min(-1), 0)
    span = hi - lo
    with np.errstate(divide="ignore"):
        e = np.maximum(np.frexp(span / 15)[1] - 8, -133)
    step = 2.0 ** e
    s = np.floor(span / 15 / step) * step
    s = np.where(15 * s >= span, s, s + step)
    d = np.where(s > 0, s, 1)
    z = np.rint(-lo / d)
    c = np.clip(np.rint(x / d[..., None]) + z[..., None], 0, 15)
    return c.astype(int), s, z.astype(int)


def unpack(pages, D):
    """uint8 pages [n, heads, blocks, 16 D + 128] (numpy) -> K and V codes
    [n, heads, page, D], scales and zero points [n, heads, page]."""
    n, heads, blocks, _ = pages.shape
    out = []
    for part in range(2):
        words = np.ascontiguousarray(pages[..., part * 8 * D:(part + 1) * 8 * D]).view("<u4")
        words = words.reshape(n, heads, blocks, D // 64, 16, 8)
        c = np.empty((n, heads, blocks, 16, D), int)
        for ch in range(D):
            in_panel = ch % 64
            bit = 4 * (in_panel % 8 // 2) + 16 * (in_panel % 2)
            c[..., ch] = (words[..., ch // 64, :, in_panel // 8] >> bit) & 15
        p = np.ascontiguousarray(pages[..., 16 * D + part * 64:16 * D + (part + 1) * 64]).view("<u4")
        s = ((p >> 16) << 16).astype(np.uint32).view(np.float32).astype(np.float64)
        z = (p & 0xffff).astype(int) - 0x4300
        out.append((c.reshape(n, heads, blocks * 16, D), s.reshape(n, heads, -1), z.reshape(n, heads, -1)))
    return out


def pack(k, v, n_pages, page, slots, fill=255):
    """Pages holding the vectors k, v [n, heads, D] (float) in their slots; all
    other bytes are `fill`."""
    n, heads, D = k.shape
    pages = np.full((n_pages, heads, page // 16, 16 * D + 128), fill, np.uint8)
    for part, x in enumerate((k, v)):
        c, s, z = quantise(x)
        par = ((s.astype(np.float32).view(np.uint32)) | 0x4300 | z.astype(np.uint32)).astype("<u4")
        for i, slot in enumerate(slots):
            pg, off = divmod(int(slot), page)
            blk, tok = divmod(off, 16)
            words = np.zeros((heads, D // 8), np.uint64)
            for ch in range(D):
                words[:, ch // 8] |= c[i, :, ch].astype(np.uint64) << np.uint64(4 * (ch % 8 // 2) + 16 * (ch % 2))
            rows = words.astype("<u4").view(np.uint8).reshape(heads, D // 64, 32)
            for pan in range(D // 64):
                at = part * 8 * D + pan * 512 + tok * 32
                pages[pg, :, blk, at:at + 32] = rows[:, pan]
            at = 16 * D + part * 64 + tok * 4
            pages[pg, :, blk, at:at + 4] = np.ascontiguousarray(par[i]).view(np.uint8).reshape(heads, 4)
    return pages


def visible(W, N, G, i):
    """Step rows that step row i sees."""
    n1 = N - 1
    if i == 0:
        return [0]
    if i <= W * n1:
        l, j = divmod(i - 1, W)
        return [0] + list(range(1, 2 + j)) + [1 + m * W + j for m in range(1, l + 1)]
    g, k = divmod(i - 1 - W * n1, n1)
    first = 1 + W * n1 + g * n1
    return [0] + list(range(first, first + k + 1))


def attention(q, ks, vs, kc, vc, W, N, G):
    """One sequence in doubles: q [T, H, D], step k/v [T, Hkv, D], cached values
    [len, Hkv, D].  Returns (out [T, H, D], spread [T, H]): spread is the norm
    over channels of the root of sum p^2 v^2, what independent relative errors
    of the probabilities add up to."""
    T, H, D = q.shape
    group = H // ks.shape[1]
    out, spread = np.zeros((T, H, D)), np.zeros((T, H))
    for i in range(T):
        see = visible(W, N, G, i)
        for h in range(H):
            keys = np.concatenate([kc[:, h // group], ks[see, h // group]])
            vals = np.concatenate([vc[:, h // group], vs[see, h // group]])
            a = keys @ q[i, h] / np.sqrt(D)
            p = np.exp(a - a.max())
            p /= p.sum()
            out[i, h] = p @ vals
            spread[i, h] = np.sqrt(((p[:, None] * vals) ** 2).sum())
    return out, spread


def plan(lens, n_new, free, n_free, table, n_slots, stride, page):
    """(slots, table, new_lens, left), or None where it does not fit."""
    table = table.copy()
    stack = list(free[:n_free])
    slots = np.full(n_slots, -1, np.int64)
    new_lens, at = np.array(lens).copy(), 0
    for b, (n, k) in enumerate(zip(lens, n_new)):
        if n < 0:
            continue
        if k < 0 or n + k > table.shape[1] * page or (stride and k > stride):
            return None
        for j in range(-(-n // page), -(-(n + k) // page)):
            if not stack:
                return None
            table[b, j] = stack.pop()
        first = b * stride if stride else at
        if not stride and at + k > n_slots:
            return None
        for i in range(k):
            p = n + i
            slots[first + i] = table[b, p // page] * page + p % page
        at += k
        new_lens[b] = n + k
    return slots, table, new_lens, len(stack)
