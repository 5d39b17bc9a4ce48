"""64-bit statements of the paged bf16 KV cache's operators, for its tests.

``turn``: the position rotation.  ``attend``: a step's rows over their prefix,
their own tokens and the step rows they see, with the spread that roundings of
the probabilities can cause.  Plain torch and numpy; nothing of the library.
"""
import math

import numpy as np
import torch


def sees(W, N, G):
    """bool [T, T]: which step rows (columns) a step row sees, from the branches' meaning."""
    T = 1 + (W + G) * (N - 1)
    see = np.zeros((T, T), bool)
    see[:, 0] = True
    for level in range(N - 1):
        for col in range(W):
            r = 1 + level * W + col
            see[r, 1: 2 + col] = True                       # level 0 up to its column
            see[r, [1 + m * W + col for m in range(level + 1)]] = True
    for g in range(G):
        for i in range(N - 1):
            r = 1 + W * (N - 1) + g * (N - 1)
            see[r + i, r: r + i + 1] = True
    return see


def turn(x, pos, rot, theta=1e4, neighbours=False, freq=None):
    """x float64 [n, heads, D] turned to positions pos: pairs as complex numbers."""
    y, i = np.array(x, np.float64), np.arange(rot // 2)
    f = np.power(float(theta), -2.0 * i / rot) if freq is None else np.asarray(freq, np.float64)
    lo, hi = (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)
    # the angle modulo a circle in extended precision: a product of 31 and 53 bits
    angle = np.asarray(np.mod(np.asarray(pos, np.longdouble)[:, None] * f.astype(np.longdouble), _TWO_PI), np.float64)
    z = (y[..., lo] + 1j * y[..., hi]) * np.exp(1j * angle)[:, None]
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


# 2 pi to the precision of long double (atan's)
_TWO_PI = 8 * np.arctan(np.longdouble(1))


def cached(pages, row, n, page):
    """float64 [n, heads, D]: the first n tokens in the pages of a table's row (bad pages: None entries)."""
    n_pages = pages.shape[0]
    idx = torch.as_tensor(np.asarray(row[: -(-n // page)], np.int64), device=pages.device)
    ok = (idx >= 0) & (idx < n_pages)
    x = pages[idx.clamp(0, n_pages - 1)].transpose(1, 2).flatten(0, 1)[:n].double()
    return x, ok.repeat_interleave(page)[:n]


def attend(k_pages, v_pages, q, k_step, v_step, lens, table, W, N, G, prefixes=()):
    """prefixes: (first sequence, sequences after the last, length, pages).
    Returns out and spread, float64 [batch, T, heads, D] (rows of lens < 0: NaN):
    spread = sqrt(sum p^2 (v - o)^2), what independent relative errors of the
    probabilities move the output by."""
    page, Hkv, D = k_pages.shape[2], k_pages.shape[1], k_pages.shape[3]
    see = torch.as_tensor(sees(W, N, G), device=q.device)
    T, B = see.shape[0], len(lens)
    q = q.double().reshape(B, T, -1, D)
    H = q.shape[2]
    steps = [x.double().reshape(B, T, Hkv, D) for x in (k_step, v_step)]
    out = torch.full((B, T, H, D), float("nan"), dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(out)
    for b, n in enumerate(lens):
        if n < 0:
            continue
        parts, live = [[], []], []
        for lo, hi, m, row in prefixes:
            if lo <= b < hi and m > 0:
                for i, pages in enumerate((k_pages, v_pages)):
                    x, ok = cached(pages, row, m, page)
                    parts[i].append(x)
                live.append(ok)
        for i, pages in enumerate((k_pages, v_pages)):
            x, ok = cached(pages, table[b], n, page)
            parts[i] += [x, steps[i][b]]
        live.append(ok)
        K, V = (torch.cat(p) for p in parts)                # [keys, Hkv, D]
        keep = torch.cat(live)
        keep = torch.cat([keep[None].expand(T, -1), see], 1)   # [T, keys]
        for g in range(Hkv):
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                s = q[b, :, h] @ K[:, g].T / math.sqrt(D)
                p = torch.softmax(torch.where(keep, s, float("-inf")), -1)
                # a hidden key's value takes no part, whatever it is
                v = torch.where(torch.isfinite(V[:, g]), V[:, g], 0.0)
                o = p @ v
                p2 = p * p                                  # (the spread of the finite part)
                spread[b, :, h] = torch.sqrt(torch.clamp(p2 @ (v * v) - 2 * o * (p2 @ v) + p2.sum(-1, keepdim=True) * o * o, min=0))
                for j in torch.nonzero(~torch.isfinite(V[:, g]).all(-1)).flatten().tolist():
                    o = torch.where(keep[:, j, None] & ~torch.isfinite(V[j, g]), o + V[j, g], o)
                out[b, :, h] = o
    return out, torch.nan_to_num(spread)                    # (rows that are NaN have none)
