"""The paged bf16 KV cache on the GPU, through KV16Cache and the C ABI, against
the 64-bit reference of kv16_ref.

Tolerances.  Slots and what is not turned: equal.  Turned rows: x cos - x' sin
with an angle within 2^-24 pi + 2^-53 |t f| and two sines' units in the last
place, in fp32: within 2^-21 (|x| + |x'|), and one rounding to bf16, 2^-8 of
the value.  Attention: a probability and the output are each rounded to bf16,
off by at most 2^-8 of the value.  The sum takes the rounded probabilities, so
their errors move an output by sum p e (v - o): independent ones by 2^-8 times
spread = sqrt(sum p^2 (v - o)^2), and up to four keys' that agree by twice
that.  A row's error over its channels is then within 2^-8 (|o| + 2 spread);
the fp32 part (scores, sums, joins of parts) gets 2^-12 of |o| + |v|.
"""
import numpy as np
import pytest

import kv16_ref as R
from helpers import build_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def _i32(a):
    import torch
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def _bf(x):
    import torch
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def _np(x):
    return x.double().cpu().numpy()


# ------------------------------------------------------------------- append

ROPES = [dict(rot=None), dict(rot=64), dict(rot=48, theta=5e5), dict(rot=16, neighbours=True), dict(rot=64, neighbours=True, theta=1e6)]


def _near(got, want, err):
    """got (bf16) within a rounding of want, itself known to err."""
    a, b = _np(got), np.asarray(want)
    bad = np.abs(a - b) > 2.0 ** -8 * np.abs(b) + err * (1 + 2.0 ** -8) + 2.0 ** -133
    assert not bad.any(), (int(bad.sum()), a[bad][:4], b[bad][:4])


def _turned(x, pos, r, D):
    """A turned row and how far fp32 may be from it."""
    rot = r["rot"]
    if rot is None:
        return np.asarray(x, np.float64), np.zeros(np.shape(x))
    y = R.turn(x, pos, rot, r.get("theta", 1e4), r.get("neighbours", False), r.get("freq"))
    err, a, i = np.zeros(np.shape(x)), np.abs(np.asarray(x, np.float64)), np.arange(rot // 2)
    lo, hi = (2 * i, 2 * i + 1) if r.get("neighbours", False) else (i, i + rot // 2)
    err[..., lo] = err[..., hi] = 2.0 ** -21 * (a[..., lo] + a[..., hi])
    return y, err


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rope", ROPES, ids=str)
@pytest.mark.parametrize("n,heads,kv_heads,D,page", [(1, 4, 4, 64, 16), (7, 6, 2, 128, 32), (129, 7, 1, 64, 64), (700, 9, 3, 128, 128)])
def test_append_turns_and_keeps(n, heads, kv_heads, D, page, rope, dtype):
    """Queries and keys turned, keys and values kept in their slots, from rows of a fused projection."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    g = np.random.default_rng(n * 31 + D)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n_rows, W = n + 5, (heads + 2 * kv_heads) * D
    qkv = torch.as_tensor(g.standard_normal((n_rows, W + 16)).astype(np.float32)).to(tdt).cuda()
    q, k, v = qkv[:, :heads * D], qkv[:, heads * D:(heads + kv_heads) * D], qkv[:, (heads + kv_heads) * D:W]
    rows = g.integers(0, n_rows, n) if n > 1 else None
    pos = g.integers(0, 1 << 20, n)
    pos[0] = (1 << 31) - 1
    n_pages = -(-n // page) + 2
    slots = g.permutation(n_pages * page)[:n]
    slots[g.random(n) < 0.3] = -1
    kp, vp = LA.KV16Cache.empty_pages(n_pages, kv_heads, D, page)
    kp.fill_(7), vp.fill_(-7)
    cache = LA.KV16Cache(kp, vp, 4)
    k_out = torch.full((n + 1, kv_heads * D + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    q_out = torch.full((n + 1, heads * D), 3.0, dtype=torch.bfloat16, device="cuda")
    r = LA.Rope(rope["rot"], rope.get("theta", 1e4), rope.get("neighbours", False)) if rope["rot"] else None
    cache.append(k, v, _i32(slots), rows=None if rows is None else _i32(rows), positions=_i32(pos) if r else None, rope=r,
                 k_out=k_out[:n, :kv_heads * D], q=q, q_out=q_out[:n]) if rows is not None else \
        cache.append(k[:n], v[:n], _i32(slots), positions=_i32(pos) if r else None, rope=r, k_out=k_out[:n, :kv_heads * D],
                     q=q[:n], q_out=q_out[:n])
    cache.check()
    src = np.arange(n) if rows is None else rows
    kx, kerr = _turned(_np(k)[src].reshape(n, kv_heads, D), pos, rope, D)
    qx, qerr = _turned(_np(q)[src].reshape(n, heads, D), pos, rope, D)
    _near(q_out[:n].reshape(n, heads, D), qx, qerr)
    _near(k_out[:n, :kv_heads * D].reshape(n, kv_heads, D), kx, kerr)
    assert (k_out[n:] == 3).all() and (k_out[:, kv_heads * D:] == 3).all() and (q_out[n:] == 3).all()
    left = np.ones((n_pages, page), bool)
    for i, s in enumerate(slots):
        if s >= 0:
            left[s // page, s % page] = False
            # the same bits in both places, and values as they are
            assert torch.equal(kp[s // page, :, s % page], k_out[i, :kv_heads * D].reshape(kv_heads, D))
            assert torch.equal(vp[s // page, :, s % page], v[src[i]].reshape(kv_heads, D).to(torch.bfloat16))
    left = torch.as_tensor(left, device="cuda")
    assert (kp.transpose(1, 2)[left] == 7).all() and (vp.transpose(1, 2)[left] == -7).all()


@pytest.mark.parametrize("n", [1, 1216, 1217, 2500])
@pytest.mark.parametrize("what", ["k", "q"])
def test_append_turns_a_single_head(what, n):
    """A call that moves one head, of few tokens and of many."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    D, g = 64, np.random.default_rng(n)
    c = LA.KV16Cache(*LA.KV16Cache.empty_pages(2, 1, D, 16), max_pages=2)
    x, pos, out = _bf(g.standard_normal((n, D))), g.integers(0, 4096, n), torch.zeros((n, D), dtype=torch.bfloat16, device="cuda")
    to = dict(k_out=out) if what == "k" else dict(q=x, q_out=out)
    c.append(x, None, None, positions=_i32(pos), rope=LA.Rope(D), **to)
    c.check()
    y, err = _turned(_np(x)[:, None], pos, dict(rot=D), D)
    _near(out, y[:, 0], err[:, 0])


def test_append_given_frequencies_and_far_positions():
    """Angles of far positions lose nothing: the last position of 31 bits, negative ones, frequencies of one's own."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    D, n = 128, 64
    g = np.random.default_rng(5)
    freq = np.concatenate([[1.0, 0.0, -0.5, 3.0], g.random(60)])
    pos = np.concatenate([[2 ** 31 - 1, -1, 0, -2 ** 31, 2 ** 30 + 1], g.integers(-2 ** 31, 2 ** 31, n - 5)])
    x = g.standard_normal((n, D)).astype(np.float32)
    kp, vp = LA.KV16Cache.empty_pages(1, 1, D, 16)
    cache = LA.KV16Cache(kp, vp, 1)
    k = torch.as_tensor(x).cuda()
    out = torch.empty((n, D), dtype=torch.bfloat16, device="cuda")
    cache.append(k, None, None, positions=_i32(pos), rope=LA.Rope(D, freq=freq), k_out=out)
    want, err = _turned(x.reshape(n, 1, D), pos, dict(rot=D, freq=freq), D)
    # turn's last bit times 2^31 positions is 2^-33 of a circle; a double's 53 bits of the frequency, 2^-22 radians of 2^31
    _near(out.reshape(n, 1, D), want, err + 2.0 ** -21 * np.abs(x.reshape(n, 1, D)).max())


@pytest.mark.parametrize("neighbours", [False, True])
def test_append_in_place(neighbours):
    """q_out = q and k_out = k inside one projection's rows."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    n, H, Hkv, D = 300, 8, 2, 128
    g = np.random.default_rng(6)
    qkv = _bf(g.standard_normal((n, (H + 2 * Hkv) * D)))
    was = qkv.clone()
    q, k, v = qkv[:, :H * D], qkv[:, H * D:(H + Hkv) * D], qkv[:, (H + Hkv) * D:]
    kp, vp = LA.KV16Cache.empty_pages(20, Hkv, D, 16)
    cache = LA.KV16Cache(kp, vp, 4)
    pos, rope = _i32(np.arange(n)), LA.Rope(D, neighbours=neighbours)
    other_k, other_q = torch.empty_like(k), torch.empty_like(q)
    cache.append(k, v, _i32(np.arange(n)), positions=pos, rope=rope, k_out=other_k, q=q, q_out=other_q)
    assert torch.equal(qkv, was)
    cache.append(k, v, _i32(np.arange(n)), positions=pos, rope=rope, k_out=k, q=q, q_out=q)
    assert torch.equal(q, other_q) and torch.equal(k, other_k) and torch.equal(v, was[:, (H + Hkv) * D:])


def test_append_bad_indexes_leave_their_rows_out():
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    n, D = 6, 64
    kp, vp = LA.KV16Cache.empty_pages(2, 1, D, 16)
    k = _bf(np.ones((4, D)))
    for rows, slots in (([0, 1, 4, 2, -1, 3], [0, 1, 2, 3, 4, 5]), ([0, 1, 2, 2, 3, 3], [0, 1, 32, 3, 2 ** 31 - 1, 5])):
        kp.zero_(), vp.zero_()
        cache = LA.KV16Cache(kp, vp, 1)
        out = torch.zeros((n, D), dtype=torch.bfloat16, device="cuda")
        cache.append(k, k, _i32(slots), rows=_i32(rows), k_out=out)
        with pytest.raises(LA.LAError) as e:
            cache.check()
        assert e.value.code == LA.LA_ERR_ARG
        assert out[:, 0].tolist() == [1, 1, 0, 1, 0, 1]
        assert kp[0, 0, :6, 0].tolist() == [1, 1, 0, 1, 0, 1] and vp[0, 0, :6, 0].tolist() == [1, 1, 0, 1, 0, 1]
        assert int(kp[1].abs().sum()) == 0


def test_append_keeps_nan_and_infinity():
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    kp, vp = LA.KV16Cache.empty_pages(1, 1, 64, 16)
    x = np.zeros((1, 64), np.float32)
    x[0, 3], x[0, 5], x[0, 40] = np.nan, np.inf, 3.4e38
    k = torch.as_tensor(x).cuda()
    LA.KV16Cache(kp, vp, 1).append(k, k, _i32([2]), positions=_i32([0]), rope=LA.Rope(32))
    for p in (kp, vp):
        assert torch.isnan(p[0, 0, 2, 3]) and torch.isinf(p[0, 0, 2, 40])   # past the largest bf16
    assert torch.isinf(vp[0, 0, 2, 5]) and not torch.isfinite(kp[0, 0, 2, 5])


def test_append_offsets_past_32_bits():
    """Slots whose elements lie past 2^32 from the pages' start."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    D, Hkv, page = 128, 40, 128
    n_pages = 2 ** 32 // (Hkv * page * D) + 3
    kp = torch.empty((n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    k, v = (_bf(np.random.default_rng(i).standard_normal((3, Hkv * D))) for i in range(2))
    slots = [n_pages * page - 1, 5, (n_pages - 2) * page + 17]
    LA.KV16Cache(kp, vp, 4).append(k, v, _i32(slots))
    for i, s in enumerate(slots):
        assert torch.equal(kp[s // page, :, s % page].flatten(), k[i]) and torch.equal(vp[s // page, :, s % page].flatten(), v[i])


# ---------------------------------------------------------------- attention

def _case(lens, prefixes, heads, kv_heads, D, page, W, N, G, seed=0, level=1.0, spare=3, ws_fill=None):
    """A batch over a cache whose unwritten slots hold NaN.  prefixes: (length, sequences) in order; a length
    of None leaves the sequences without one before the next."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    g = np.random.default_rng(seed)
    T, B = 1 + (W + G) * (N - 1), len(lens)
    at, spans = 0, []
    for n, count in prefixes:
        spans.append((at, at + count, n))
        at += count
    assert at <= B
    # prefix_first needs neighbours to touch: gaps become prefixes of length 0
    held = [max(0, n) for n in lens] + [n for _, _, n in spans]
    need = [-(-n // page) for n in held]
    n_pages = sum(need) + spare
    order, used, rows = g.permutation(n_pages), 0, []
    for k in need:
        rows.append(order[used: used + k])
        used += k
    pages = [torch.full((n_pages, kv_heads, page, D), -1, dtype=torch.int16, device="cuda").view(torch.bfloat16) for _ in range(2)]
    for i, x in enumerate(pages):
        for n, row in zip(held, rows):
            if n:
                blk = torch.full((len(row) * page, kv_heads, D), float("nan"), device="cuda")
                blk[:n] = torch.as_tensor(g.standard_normal((n, kv_heads, D)).astype(np.float32)).cuda() * (level if i == 0 else 1)
                x[torch.as_tensor(row, device="cuda")] = blk.to(torch.bfloat16).reshape(len(row), page, kv_heads, D).transpose(1, 2)
    mp, pmp = max([1] + need[:B]), max([1] + need[B:])
    table, ptable = np.full((B, mp), -1), np.full((len(spans), pmp), -1)
    for b in range(B):
        table[b, :need[b]] = rows[b]
    for p in range(len(spans)):
        ptable[p, :need[B + p]] = rows[B + p]
    qkv = _bf(g.standard_normal((B * T, (heads + 2 * kv_heads) * D)))
    c = dict(q=qkv[:, :heads * D], k=qkv[:, heads * D:(heads + kv_heads) * D], v=qkv[:, (heads + kv_heads) * D:],
             lens=list(lens), table=table, ptable=ptable, spans=spans, W=W, N=N, G=G, T=T, H=heads, D=D, page=page)
    c["cache"] = LA.KV16Cache(pages[0], pages[1], mp)
    c["first"] = [s[0] for s in spans] + [at]
    c["d"] = dict(lens=_i32(lens), table=_i32(table), plens=_i32([n for _, _, n in spans]), ptable=_i32(ptable), first=_i32(c["first"]))
    c["out"] = torch.full((B * T, heads * D), 123.0, dtype=torch.bfloat16, device="cuda")
    c["ws"] = torch.full((max(16, c["cache"].attention_bytes(B, heads, W, N, G, prefixes=len(spans), prefix_pages=pmp)),), 255,
                         dtype=torch.uint8, device="cuda")
    return c


def _call(c, **kw):
    d = c["d"]
    shared = dict(prefix_lens=d["plens"], prefix_table=d["ptable"], prefix_first=d["first"]) if c["spans"] else {}
    c["cache"].attention(c["q"], c["k"], c["v"], d["lens"], d["table"], c["W"], c["N"], c["G"], out=c["out"], workspace=c["ws"],
                         **{**shared, **kw})
    return c["out"]


def _want(c):
    return R.attend(c["cache"].k_pages, c["cache"].v_pages, c["q"], c["k"], c["v"], c["lens"], c["table"], c["W"], c["N"], c["G"],
                    [(lo, hi, n, c["ptable"][p]) for p, (lo, hi, n) in enumerate(c["spans"])])


def _compare(c, got, want=None):
    import torch
    o, spread = want or _want(c)
    B, T, H, D = o.shape
    got = got.double().reshape(B, T, H, D)
    for b, n in enumerate(c["lens"]):
        if n < 0:
            assert (got[b] == 123).all(), b
            continue
        assert torch.equal(torch.isnan(got[b]), torch.isnan(o[b])), b
        fin = torch.isfinite(o[b])
        assert torch.equal(torch.where(fin, 0.0, got[b]).nan_to_num(0.5), torch.where(fin, 0.0, o[b]).nan_to_num(0.5)), b
        err = torch.where(fin, got[b] - o[b], 0.0).norm(dim=-1)
        size = torch.where(fin, o[b], 0.0).norm(dim=-1)
        tol = 2.0 ** -8 * (size + 2 * spread[b].norm(dim=-1)) + 2.0 ** -12 * (size + D ** 0.5)
        assert (err <= tol).all(), (b, (err / tol).max().item())


SHAPES = [  # lens, prefixes, heads, kv heads, D, page, (W, N, G)
    ([1, 5], [(33, 2)], 4, 4, 64, 16, (0, 2, 0)),
    ([0], [(1, 1)], 1, 1, 128, 16, (0, 2, 0)),
    ([0, 0, 0], [], 2, 1, 64, 128, (0, 2, 0)),
    ([15, 16, 17, 127, 128, 129, 0, 1], [(128, 8)], 8, 2, 128, 16, (0, 2, 0)),
    ([112, 113, 111, 240], [(129, 3)], 3, 3, 64, 32, (0, 2, 0)),                   # the step's key beside 112 others, or not
    ([300, 2, 77, 64, 5], [(1000, 2), (0, 1), (513, 1)], 21, 3, 128, 64, (0, 2, 0)),
    ([40] * 20, [(700, 9), (31, 0), (128, 11)], 14, 2, 64, 16, (0, 2, 0)),
    ([9, 200, 31], [(257, 3)], 10, 2, 128, 128, (2, 4, 2)),                        # 13 rows x 5 heads
    ([100, 0, 511], [(640, 2)], 8, 1, 128, 64, (7, 5, 7)),                         # 57 rows x 8 heads: several tiles
    ([17, 300], [(511, 2)], 3, 3, 128, 16, (15, 5, 15)),                           # 121 rows
    ([0, 50, 129], [(1024, 3)], 4, 2, 64, 32, (0, 100, 1)),                        # a chain of 100 rows
    ([3, 70], [(90, 2)], 2, 2, 128, 16, (0, 128, 1)),                              # 128 rows
    ([60, 60], [(60, 2)], 128, 1, 64, 16, (0, 2, 0)),                              # 128 heads of one KV head
    ([20], [(45, 1)], 128, 1, 128, 16, (3, 3, 2)),
    ([5, 6], [(7, 2)], 100, 1, 64, 16, (1, 4, 1)),                                 # 100 heads: a row a tile
    ([30, -1, 40, -7, 0], [(200, 3)], 6, 2, 128, 32, (1, 3, 1)),                   # sequences that are none
    ([-1, -1], [(77, 2)], 2, 2, 64, 16, (0, 2, 0)),
    ([2000, 3], [(5000, 2)], 2, 1, 128, 128, (0, 2, 0)),
    ([700, 1300, 64], [(4000, 3)], 16, 2, 64, 64, (5, 4, 5)),
    ([1] * 130, [(300, 130)], 5, 5, 64, 16, (0, 2, 0)),                            # 130 rows: a tile and two
    ([4] * 70, [(300, 70)], 8, 2, 128, 16, (0, 2, 0)),                             # 280 rows: a pair and one
    ([10, 250, 33, 70], [], 8, 2, 128, 32, (7, 5, 7)),                             # no prefixes
    ([128 - 16, 128 - 57, 71 + 128], [(100, 1)], 4, 1, 64, 16, (7, 5, 7)),         # the step beside a tile's rest
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attention(i):
    lens, prefixes, H, Hkv, D, page, (W, N, G) = SHAPES[i]
    c = _case(lens, prefixes, H, Hkv, D, page, W, N, G, seed=i)
    got = _call(c)
    c["cache"].check()
    _compare(c, got)


@pytest.mark.parametrize("seed", range(12))
def test_attention_drawn(seed):
    """Sizes drawn over the whole range."""
    g = np.random.default_rng(1000 + seed)
    log = lambda lo, hi: int(round(np.exp(g.uniform(np.log(lo), np.log(hi)))))
    Hkv, group, page, D = log(1, 9), int(g.choice([1, 2, 3, 5, 8, 12])), int(g.choice([16, 32, 64, 128])), int(g.choice([64, 128]))
    W, N, G = [(0, 2, 0), (int(g.integers(1, 8)), int(g.integers(2, 5)), int(g.integers(0, 8))), (0, int(g.integers(2, 100)), 1)][seed % 3]
    B = log(1, 24)
    lens = g.integers(0, log(2, 900), B)
    cuts = np.sort(g.integers(0, B + 1, 3))
    prefixes = [(log(1, 3000), int(n)) for n in np.diff(np.concatenate([[0], cuts]))]
    c = _case(lens.tolist(), prefixes, Hkv * group, Hkv, D, page, W, N, G, seed=seed)
    got = _call(c)
    c["cache"].check()
    _compare(c, got)


@pytest.mark.parametrize("level", [1e-3, 30.0, 2000.0])
def test_attention_flat_and_sharp(level):
    """Scores from almost equal to almost one key a row, the largest found early or late."""
    c = _case([300, 40, 600], [(900, 2)], 8, 2, 128, 32, 2, 4, 2, seed=3, level=level)
    got = _call(c)
    _compare(c, got)


def test_attention_rising_scores():
    """Keys whose scores grow along the sequence by more than the fp32 range of exp2 in all."""
    import torch
    c = _case([500, 20], [(1500, 2)], 4, 2, 64, 16, 0, 2, 0, seed=4)
    q = c["q"]
    q.copy_(torch.ones_like(q))
    kp = c["cache"].k_pages
    for p, n in [(c["ptable"][0], 1500), (c["table"][0], 500)]:
        for t in range(n):
            kp[int(p[t // 16]), :, t % 16] = 0.05 * t if p is c["ptable"][0] else 75 + 0.1 * t
    _compare(c, _call(c))


def test_attention_nan_and_infinity_stay_with_their_rows():
    """A step row's NaN or infinity reaches the rows that see it, a sequence's those of the sequence, a prefix's
    those behind it."""
    import torch
    for where in ("v_step", "k_step", "v_tail", "v_prefix"):
        c = _case([30, 140, 20], [(200, 2)], 8, 2, 128, 16, 2, 3, 2, seed=5)
        T = c["T"]
        if where == "v_step":
            c["v"][T + 2, 5] = float("nan")            # sequence 1: a window row, a candidate's row
            c["v"][T + 6, 130] = float("inf")
            c["v"][2 * T + 1, 7] = float("-inf")
        elif where == "k_step":
            c["k"][T + 3, 5] = float("nan")
        elif where == "v_tail":
            c["cache"].v_pages[int(c["table"][1, 2]), 1, 3, 9] = float("nan")
        else:
            c["cache"].v_pages[int(c["ptable"][0, 5]), 0, 3, 9] = float("inf")
        got, want = _call(c), _want(c)
        assert not torch.isfinite(want[0]).all()
        _compare(c, got, want)


MANY = [  # prefixes worth reading by themselves, many entries, many prefixes: lens, prefixes, heads, kv heads, D, page, (W, N, G)
    ([7, -1, 130, 0, 64, 33, 2, 1, 90, 5], [(3000, 6), (0, 1), (2111, 3)], 4, 2, 128, 64, (3, 3, 3)),       # 26 rows a sequence
    ([3, 40, 0, -2, 17, 200, 8, 1] * 2, [(2500, 16)], 8, 1, 128, 32, (1, 5, 0)),                           # 40 rows, all with one
    ([20, 0, 61, 7, 5, 128, 300, 9, -1], [(6000, 2), (5000, 3), (-1, 1)], 8, 2, 64, 128, (2, 5, 1)),         # 52; a length below 0
    ([int(n) for n in np.random.default_rng(1).integers(-1, 40, 420)], [(170, 201), (40, 199), (3, 1)], 1, 1, 64, 16, (0, 2, 0)),
    ([int(n) for n in np.random.default_rng(2).integers(-1, 40, 400)], [(100, 30), (170, 333)], 2, 1, 64, 16, (2, 5, 0)),   # 18 rows
    ([int(n) for n in np.random.default_rng(3).integers(-1, 90, 400)], [], 2, 2, 64, 32, (0, 2, 0)),
    ([5, 0, 31, -1, 77, 16, 2, 50] * 5, [(20 * i, 1) for i in range(36)], 2, 1, 64, 16, (0, 2, 0)),          # 36 prefixes, read per sequence
    ([5, 0, 31, -1, 77, 16, 2, 50] * 5, [(13 * i, 1) for i in range(36)], 40, 1, 64, 16, (0, 2, 0)),         # and by many rows
    ([9, 1, 60] * 17, [(30 + 20 * i, 1) for i in range(42)], 4, 2, 128, 32, (0, 2, 0)),                      # 42 by themselves
]


@pytest.mark.parametrize("i", range(len(MANY)))
def test_attention_many(i):
    lens, prefixes, H, Hkv, D, page, (W, N, G) = MANY[i]
    c = _case(lens, [(max(n, 0), k) for n, k in prefixes], H, Hkv, D, page, W, N, G, seed=40 + i)
    c["d"]["plens"].copy_(_i32([n for n, _ in prefixes]))
    got = _call(c)
    c["cache"].check()
    _compare(c, got)


def test_attention_bad_values_beside_shared_prefixes():
    """Prefixes read by themselves: bad pages, lengths over their bounds, prefix_first out of order."""
    import lossless_lookahead_decoding_gb300 as LA

    def refused(c):
        with pytest.raises(LA.LAError) as e:
            c["cache"].check()
        return e.value.code == LA.LA_ERR_ARG

    for rows in ((0, 2, 0), (3, 3, 2)):
        new = lambda: _case([30, 40, 50, 6, 77, 8], [(4000, 3), (3000, 2)], 4, 2, 128, 64, *rows, seed=17)
        c = new()
        for t, p, j in (("table", 0, 0), ("ptable", 0, 3), ("ptable", 1, 46), ("table", 4, 1)):
            for bad in (-1, 10 ** 6):
                c[t][p, j] = bad
        for t in ("table", "ptable"):
            c["d"][t].copy_(_i32(c[t]))
        got = _call(c)
        assert refused(c)
        _compare(c, got)
        c = new()
        got = _call(c, max_len=60, max_prefix_len=3999)
        for b in (0, 1, 2, 4):
            c["lens"][b] = -1
        assert refused(c)
        _compare(c, got)
        for first in ([0, 4, 3], [-1, 2, 3], [0, 4, 7], [2 ** 31 - 1, 0, -2 ** 31]):
            c = new()
            c["d"]["first"].copy_(_i32(first))
            assert (_call(c) == 123).all() and refused(c)


def test_attention_more_keys_than_a_schedule_holds():
    """64 sequences x 64 heads over 7.9 M keys each (one page named again and again) are refused on the device."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    B, H, D, page, mp = 64, 64, 64, 128, 61440
    c = LA.KV16Cache(*LA.KV16Cache.empty_pages(1, H, D, page), max_pages=mp)
    x = torch.zeros((B, H * D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 123.0)
    table = torch.zeros((B, mp), dtype=torch.int32, device="cuda")
    ws = torch.empty(c.attention_bytes(B, H, 0, 2, 0), dtype=torch.uint8, device="cuda")
    c.attention(x, x, x, _i32([page * mp] * B), table, 0, 2, 0, out=out, workspace=ws)
    with pytest.raises(LA.LAError) as e:
        c.check()
    assert e.value.code == LA.LA_ERR_ARG and (out == 123).all()
    c.attention(x, x, x, _i32([300] * B), table, 0, 2, 0, out=out, workspace=ws)
    c.check()
    assert (out == 0).all()


def test_attention_buffers_at_odd_16_byte_places():
    """q, k_step, v_step, out and the workspace at 16 bytes past other boundaries; what lies beside them stays."""
    import torch
    for shape in (([30, 400, 5], [(200, 2)], 4, 2, 128, 32, 0, 2, 0), ([30, 400, 5], [(200, 2)], 4, 2, 64, 32, 5, 4, 5),
                  ([30, 40, 5, 9], [(5000, 4)], 4, 2, 128, 32, 2, 3, 2)):
        c = _case(*shape, seed=18)
        want = _call(c).clone()

        def moved(x, fill):
            room = torch.full((x.numel() * x.element_size() + 48,), fill, dtype=torch.uint8, device="cuda")
            return room, room[16:-32].view(x.dtype).view(x.shape)

        for name in ("q", "k", "v"):
            c[name] = moved(c[name].contiguous(), 255)[1].copy_(c[name])
        (oroom, c["out"]), (wroom, c["ws"]) = moved(c["out"], 77), moved(c["ws"], 78)
        assert torch.equal(_call(c), want)
        assert (oroom[:16] == 77).all() and (oroom[-32:] == 77).all() and (wroom[:16] == 78).all() and (wroom[-32:] == 78).all()
        c["cache"].check()


def test_attention_prefixes_in_gaps():
    """Sequences before the first prefix and behind the last have none."""
    c = _case([12, 40, 9, 77, 30, 5], [(150, 2), (33, 1)], 4, 2, 64, 16, 1, 3, 1, seed=6)
    c["spans"] = [(lo + 2, hi + 2, n) for lo, hi, n in c["spans"]]
    c["d"]["first"].copy_(_i32([2, 4, 5]))
    _compare(c, _call(c))


def test_attention_bad_values_on_the_device():
    """Lengths over their bound, prefix_first out of order, pages outside the pool: nothing else is touched."""
    import lossless_lookahead_decoding_gb300 as LA
    E = LA.LA_ERR_ARG

    def code(c):
        with pytest.raises(LA.LAError) as e:
            c["cache"].check()
        return e.value.code

    new = lambda: _case([30, 40, 50], [(100, 2)], 4, 2, 64, 16, 1, 3, 1, seed=7)
    c = new()
    c["d"]["lens"][1] = 10 ** 6
    got = _call(c)
    c["lens"][1] = -1
    assert code(c) == E
    _compare(c, got)
    c = new()
    got = _call(c, max_len=45)
    c["lens"][2] = -1
    assert code(c) == E
    _compare(c, got)
    c = new()
    got = _call(c, max_prefix_len=99)
    c["lens"][0] = c["lens"][1] = -1
    assert code(c) == E
    _compare(c, got)
    c = new()
    got = _call(c, max_len=50, max_prefix_len=100)
    c["cache"].check()
    _compare(c, got)
    for first in ([2, 1], [-1, 2], [0, 4], [2 ** 31 - 1, -2 ** 31]):
        c = new()
        c["d"]["first"].copy_(_i32(first))
        assert (_call(c) == 123).all() and code(c) == E
    c = new()
    for t, p, j in (("table", 0, 1), ("ptable", 0, 3), ("table", 2, 3)):
        for bad in (-1, 10 ** 6):
            c[t][p, j] = bad
        c["d"][t].copy_(_i32(c[t]))
    got = _call(c)
    assert code(c) == E
    _compare(c, got)


def test_attention_strides_and_single_rows():
    """Rows apart, one sequence, views of three dimensions."""
    import torch
    c = _case([44], [(60, 1)], 6, 2, 128, 16, 0, 2, 0, seed=8)
    wide = torch.full((1, 4000), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + 768] = c["q"]
    want = _want(c)
    c["q"] = wide[:, 8:8 + 768].unflatten(-1, (6, 128))
    _compare(c, _call(c), want)


def test_attention_equal_calls_give_equal_bits_in_graphs_and_streams():
    """Captured and replayed over other lengths; two streams with a workspace each; the workspace's old bytes do not count."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    c = _case([300, 40, 129, 5], [(700, 3)], 8, 2, 128, 32, 2, 4, 2, seed=9)
    first = _call(c).clone()
    c["ws"].random_(0, 255)
    assert torch.equal(_call(c), first)
    other = torch.empty_like(c["ws"])
    outs = [torch.empty_like(c["out"]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    d = c["d"]
    for _ in range(20):
        for s, o, w in zip(streams, outs, (c["ws"], other)):
            with torch.cuda.stream(s):
                c["cache"].attention(c["q"], c["k"], c["v"], d["lens"], d["table"], 2, 4, 2, out=o, workspace=w,
                                     prefix_lens=d["plens"], prefix_table=d["ptable"], prefix_first=d["first"])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(c)
    c["out"].fill_(123)
    graph.replay()
    assert torch.equal(c["out"], first)
    for lens, plen in (([10, 299, 0, -1], 699), ([300, 0, 1, 2], 1), ([1, 1, 1, 1], 0)):
        c["lens"], c["spans"] = lens, [(0, 3, plen)]
        d["lens"].copy_(_i32(lens)), d["plens"].copy_(_i32([plen]))
        c["out"].fill_(123)
        graph.replay()
        _compare(c, c["out"])
        if lens[1] > 64:
            # (its table names two pages: the others count as no keys, and say so)
            with pytest.raises(LA.LAError):
                c["cache"].check()
        c["cache"].check()


@pytest.mark.parametrize("heads,kv_heads,D,W,N,G", [(32, 32, 128, 0, 2, 0), (16, 16, 64, 0, 2, 0), (8, 8, 128, 3, 3, 3)])
def test_attention_many_times_under_load(heads, kv_heads, D, W, N, G):
    """A batch whose prefix and sequences contend for memory, so that loads end in other orders: equal bits every time."""
    import torch
    g = np.random.default_rng(12)
    c = _case(g.integers(1, 256, 100).tolist(), [(1000, 60), (777, 40)], heads, kv_heads, D, 64, W, N, G, seed=12)
    first = _call(c).clone()
    c["cache"].check()
    _compare(c, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(20):
            _call(c)
    for _ in range(10):
        graph.replay()
        assert torch.equal(c["out"], first)
    c["cache"].check()


def test_attention_pages_past_32_bits():
    """Pages whose elements lie past 2^32 from the arrays' start."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    c = _case([100, 30], [(260, 2)], 40, 40, 128, 128, 0, 2, 0, seed=10)
    n_pages = 2 ** 32 // (40 * 128 * 128) + 12
    small, shift = c["cache"], n_pages - c["cache"].k_pages.shape[0]
    want = _want(c)
    big = [torch.empty((n_pages, 40, 128, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    big[0][shift:], big[1][shift:] = small.k_pages, small.v_pages
    c["cache"] = LA.KV16Cache(big[0], big[1], small.max_pages)
    for t in ("table", "ptable"):
        c["d"][t] += shift
    _compare(c, _call(c), want)


def test_prompt_then_steps():
    """The calls as they are used: a system prompt planned, written and attended to in blocks, two chats behind it,
    single tokens and a lookahead step whose accepted rows are committed; every output against one causal pass."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    H, Hkv, D, page, mp, n_pages = 4, 2, 64, 16, 16, 64
    g = np.random.default_rng(11)
    kp, vp = LA.KV16Cache.empty_pages(n_pages, Hkv, D, page)
    kp.fill_(float("nan")), vp.fill_(float("nan"))
    cache, rope = LA.KV16Cache(kp, vp, mp), LA.Rope(D)
    free, n_free = _i32(g.permutation(n_pages)), _i32([n_pages])
    # rows 0: the prompt, 1 and 2: the chats
    lens, table = _i32([0, 0, 0]), _i32(np.full((3, mp), -1))
    kept = [[], [], []]                                    # rows of q, k, v of every token, as they come
    width = (H + 2 * Hkv) * D

    def step(seqs, W, N, G, positions, keep, prefix):
        """One call for sequences `seqs` (table rows), T rows each; keep: rows of each that stay."""
        T = 1 + (W + G) * (N - 1)
        B = len(seqs)
        raw = _bf(g.standard_normal((B * T, width)))
        q, k, v = raw[:, :H * D], raw[:, H * D:(H + Hkv) * D], raw[:, (H + Hkv) * D:]
        turned_k, turned_q = torch.empty_like(k).contiguous(), torch.empty_like(q).contiguous()
        cache.append(k, v, None, positions=_i32(positions), rope=rope, k_out=turned_k, q=q, q_out=turned_q)
        out = torch.empty((B * T, H * D), dtype=torch.bfloat16, device="cuda")
        sl = slice(seqs[0], seqs[-1] + 1)
        shared = dict(prefix_lens=lens[0:1].clone(), prefix_table=table[0:1], prefix_first=_i32([0, B])) if prefix else {}
        ws = torch.empty(cache.attention_bytes(B, H, W, N, G, prefixes=int(prefix), prefix_pages=mp), dtype=torch.uint8, device="cuda")
        cache.attention(turned_q, turned_k, v, lens[sl], table[sl], W, N, G, out=out, workspace=ws, **shared)
        n_new = np.zeros(3, np.int32)
        n_new[seqs] = [len(x) for x in keep]
        slots = _i32(np.zeros(int(n_new.sum())))
        cache.plan(lens, _i32(n_new), free, n_free, table, slots, lens, n_free)
        rows = np.concatenate([i * T + np.asarray(x) for i, x in enumerate(keep)]).astype(int)
        cache.append(turned_k, v, slots, rows=_i32(rows))
        cache.check()
        for i, s in enumerate(seqs):
            see = R.sees(W, N, G)
            hist = ([kept[0]] if prefix else []) + [kept[s]]
            hk = [r for h in hist for r in h]
            for r in range(T):
                mine = hk + [(_np(turned_k[i * T + j]), _np(v[i * T + j])) for j in range(T) if see[r, j]]
                K, V = (np.array([m[x] for m in mine]).reshape(-1, Hkv, D) for x in range(2))
                qq = _np(turned_q[i * T + r]).reshape(H, D)
                for h in range(H):
                    s_ = K[:, h // (H // Hkv)] @ qq[h] / np.sqrt(D)
                    p = np.exp(s_ - s_.max())
                    p /= p.sum()
                    vv = V[:, h // (H // Hkv)]
                    o = p @ vv
                    spread = np.sqrt((p[:, None] ** 2 * (vv - o) ** 2).sum(0))
                    tol = 2.0 ** -8 * (np.linalg.norm(o) + 2 * np.linalg.norm(spread)) + 2.0 ** -12 * (np.linalg.norm(o) + 8)
                    assert np.linalg.norm(_np(out[i * T + r]).reshape(H, D)[h] - o) <= tol
            kept[s] += [(_np(turned_k[i * T + j]), _np(v[i * T + j])) for j in keep[i]]

    step([0], 0, 50, 1, np.arange(50), [range(50)], False)             # the system prompt, two blocks
    step([0], 0, 21, 1, 50 + np.arange(21), [range(21)], False)
    step([1, 2], 0, 9, 1, np.tile(71 + np.arange(9), 2), [range(9), range(4)], True)   # the chats' prompts (one is shorter)
    step([1, 2], 0, 2, 0, [80, 75], [[0], [0]], True)                  # a single token each
    pos = lambda p: [p] + [p + 1 + l + c for l in range(2) for c in range(2)] + [p + 1 + i for _ in range(2) for i in range(2)]
    step([1, 2], 2, 3, 2, pos(81) + pos(76), [[0, 5, 6], [0]], True)   # a lookahead step: a candidate accepted, or none
    assert lens.tolist() == [71, 13, 6]
    done = _i32([0, 1, 1])
    cache.release(done, lens, table, free, n_free)
    assert lens.tolist() == [71, 0, 0] and int(n_free) == n_pages - 5


# ------------------------------------------------- scores far from 0, nearly equal

def _level(c, exp, sign=1, seed=0):
    """Scores sign 2^exp (C + 0 or 1) of each KV head, C a whole number of 20 bits: exact in fp32, in whatever order
    they are summed, so that the 64-bit reference has the same."""
    import torch
    g = np.random.default_rng(seed)
    Hkv, D = c["cache"].n_kv_heads, c["D"]
    c["q"].copy_(torch.full_like(c["q"], sign * 2.0 ** exp))
    base = g.integers(128, 256, (Hkv, 3)) * 2.0 ** np.array([0, 6, 12])

    def keys(shape):                                 # [..., Hkv, D]
        k = np.zeros((*shape, Hkv, D))
        k[..., :3], k[..., 3] = base, g.integers(0, 2, (*shape, Hkv))
        return _bf(k)

    kp = c["cache"].k_pages                          # [n_pages, Hkv, page, D]; unwritten slots stay NaN
    n_pages, _, page, _ = kp.shape
    kp.copy_(torch.where(torch.isnan(kp), kp, keys((n_pages, page)).transpose(1, 2)))
    c["k"].copy_(keys((len(c["k"]),)).flatten(1))


LEVELS = [  # lens, prefixes, heads, kv heads, D, page, (W, N, G)
    ([300, 40, 0], [(600, 2)], 8, 8, 128, 32, (0, 2, 0)),              # a row a sequence and KV head
    ([300, 40, 0], [(600, 2)], 8, 4, 64, 16, (1, 4, 1)),               # 14
    ([300, 40], [(600, 2)], 12, 6, 128, 16, (2, 4, 2)),                # 26: both streams have the same rows
    ([300, 40], [(700, 2)], 24, 6, 64, 64, (7, 5, 7)),                 # 228: a stream has its own
    ([30, 140, 7, 61] * 3, [(4000, 7), (3500, 5)], 12, 6, 128, 64, (0, 2, 0)),   # prefixes by themselves
    ([30, 140, 7, 61] * 3, [(4000, 7), (3500, 5)], 12, 6, 64, 128, (3, 3, 3)),
]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exp", [0, 7, 11])
@pytest.mark.parametrize("i", range(len(LEVELS)))
def test_attention_nearly_equal_scores_far_from_zero(i, exp, sign):
    """Scores of up to 2^28 (as powers of two of a weight) whose reference is off by several powers of two itself."""
    lens, prefixes, H, Hkv, D, page, (W, N, G) = LEVELS[i]
    c = _case(lens, prefixes, H, Hkv, D, page, W, N, G, seed=60 + i)
    _level(c, exp, sign, seed=i)
    got = _call(c)
    c["cache"].check()
    _compare(c, got)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exp", [14, 20, 45, 100])
@pytest.mark.parametrize("i", range(len(LEVELS)))
def test_attention_finite_scores_of_any_size(i, exp, sign):
    """Scores of 2^31 to 2^118: what fp32 makes of their product with log2(e) / sqrt(D) is off by more than exp2 can hold."""
    test_attention_nearly_equal_scores_far_from_zero(i, exp, sign)


@pytest.mark.parametrize("bits", [0.3, 0.6, 2.0, 40.0, -0.6])
@pytest.mark.parametrize("i", range(len(LEVELS)))
def test_attention_scores_that_rise_along_the_keys(i, bits):
    """Every key weighs 2^bits times the one before it, so that references move in either half of a tile, in many of
    them, and parts differ by hundreds of powers of two."""
    import math
    lens, prefixes, H, Hkv, D, page, (W, N, G) = LEVELS[i]
    c = _case(lens, prefixes, H, Hkv, D, page, W, N, G, seed=70 + i, level=0.5)
    step = np.float32(bits * math.log(2) * math.sqrt(D))

    def put(row, at, t):                                # position t as 256 a + b, each exact in bf16 but for the step
        kp[int(row[at // page]), :, at % page, 0] = float(step * 256 * (t // 256))
        kp[int(row[at // page]), :, at % page, 1] = float(step * (t % 256))

    kp = c["cache"].k_pages.cpu()
    for p, (_, _, n) in enumerate(c["spans"]):
        for t in range(n):
            put(c["ptable"][p], t, t)
    for b, n in enumerate(lens):
        before = sum(m for lo, hi, m in c["spans"] if lo <= b < hi)
        for t in range(n):
            put(c["table"][b], t, before + t)
    c["cache"].k_pages.copy_(kp)
    q = c["q"].reshape(-1, H, D).clone()
    q[..., :2] = 1
    c["q"] = q.flatten(1)
    got = _call(c)
    c["cache"].check()
    # A score far from 0 is known to 2^-23 of itself for each of its D / 16 + 1 sums in fp32, its weight to as much, in
    # nats: sum p e (v - o) is at most e (|v| + |o|) more.
    far = abs(bits) * math.log(2) * (max(lens) + max(m for _, _, m in c["spans"])) + 10
    e = (D // 16 + 1) * 2.0 ** -23 * far
    o, spread = _want(c)
    _compare(c, got, (o, spread + 2.0 ** 7 * e * (4 + o.abs())))


@pytest.mark.parametrize("heads,kv_heads,D,W,N,G", [(16, 16, 128, 0, 2, 0), (16, 8, 64, 1, 4, 1), (8, 8, 128, 2, 4, 2)])
def test_attention_sees_what_the_calls_before_it_wrote(heads, kv_heads, D, W, N, G):
    """Lengths, prefixes and rows written on the same stream right before each call, without a wait in between: as if
    everything were waited for, in a graph too."""
    import torch
    g = np.random.default_rng(21)
    B = 24
    c = _case([200] * B, [(4000, 14), (3000, 10)], heads, kv_heads, D, 64, W, N, G, seed=21)
    d, each = c["d"], []
    for _ in range(12):
        cut = int(g.integers(1, B))
        each.append((_i32(g.integers(-1, 201, B)), _i32(g.integers(1, 3001, 2)), _i32([0, cut, B]),
                     _bf(g.standard_normal(tuple(c["q"].shape))), torch.full_like(c["out"], 123.0)))

    def write(x):
        for to, what in zip((d["lens"], d["plens"], d["first"], c["q"]), x):
            to.copy_(what)
        c["out"].fill_(123)

    def run(wait):
        for x in each:
            write(x)
            if wait:
                torch.cuda.synchronize()
            _call(c)
            if wait:
                torch.cuda.synchronize()
            x[4].copy_(c["out"])

    run(True)
    want = [x[4].clone() for x in each]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(False)
    for again in (lambda: run(False), graph.replay):
        for _ in range(5):
            for x in each:
                x[4].fill_(7)
            again()
            for x, y in zip(each, want):
                assert torch.equal(x[4], y)
    c["cache"].check()
    c["lens"], c["spans"] = each[0][0].tolist(), [(0, int(each[0][2][1]), int(each[0][1][0])), (int(each[0][2][1]), B, int(each[0][1][1]))]
    write(each[0])
    _compare(c, _call(c))


def test_attention_more_keys_than_a_count_holds_behind_a_prefix():
    """64 sequences of 2^30 tokens each (one page named again and again) behind a prefix read by itself: their blocks
    pass 2^31, and every row is left alone; the same buffers then do for lengths that fit."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    B, D, page, mp = 64, 64, 128, 1 << 23
    c = LA.KV16Cache(*LA.KV16Cache.empty_pages(2, 1, D, page), max_pages=mp)
    c.v_pages.fill_(3)
    x = torch.zeros((B, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 123.0)
    table, ptable = torch.zeros((B, mp), dtype=torch.int32, device="cuda"), torch.ones((1, 24), dtype=torch.int32, device="cuda")
    ws = torch.empty(c.attention_bytes(B, 1, 0, 2, 0, prefixes=1, prefix_pages=24), dtype=torch.uint8, device="cuda")

    def call(n):
        c.attention(x, x, x + 3, _i32([n] * B), table, 0, 2, 0, out=out, workspace=ws, prefix_lens=_i32([3000]), prefix_table=ptable,
                    prefix_first=_i32([0, B]))

    call(page * mp)
    with pytest.raises(LA.LAError) as e:
        c.check()
    assert e.value.code == LA.LA_ERR_ARG and (out == 123).all()
    call(300)
    c.check()
    assert (out == 3).all()
