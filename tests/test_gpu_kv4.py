"""The paged 4-bit KV cache on the GPU, through KV4Cache and the C ABI, against
the 64-bit reference of kv4_ref.

Tolerances.  Codes, scales, slots, tables and lengths: equal.  fp32 values:
equal (a code times an 8-bit scale has 12 bits); bf16 values: the rounding of
those.  Attention: bf16 probabilities and the bf16 output round by at most
2^-8 of the value each (half of bf16's eps); a row's error over its channels
is then within 2^-8 (|o| + spread), spread = sqrt(sum p^2 v^2) (independent
roundings of the probabilities); the fp32 part (scores within
(D + 4) 2^-24 143 s sum|q| / sqrt(D), typically 2^-12) gets a tenth of that.
"""
import numpy as np
import pytest

import kv4_ref as R
from helpers import build_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def _i32(a):
    import torch
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def _cache(n_pages, heads, D, page, max_pages, fill=0):
    import lossless_lookahead_decoding_gb300 as LA
    pages = LA.KV4Cache.empty_pages(n_pages, heads, D, page)
    pages.fill_(fill)
    return LA.KV4Cache(pages, page, max_pages)


# --------------------------------------------------------- append and read

def _hard_vectors(D, g, f32):
    """Vectors where a quantiser goes wrong, as float32 [n, D]."""
    v = [np.zeros(D), np.full(D, 3.0), np.full(D, -2.5), np.full(D, -0.0)]
    ties = (np.arange(D) % 31 - 15) / 2.0                     # scale 1, every code border hit exactly
    v += [ties, ties * 0.3125, -ties, ties * 2.0 ** -120, ties * 2.0 ** 100]
    v += [np.where(np.arange(D) == 3, 3.3e38, -3.3e38), np.where(np.arange(D) == 0, 3.3e38, 1e-40)]
    v += [np.where(np.arange(D) == 5, 1.0, 2.0 ** -30), np.where(np.arange(D) == 5, -1.0, 2.0 ** -30)]
    v += [np.where(np.arange(D) % 2 == 0, 2.0 ** -133, -(2.0 ** -133)), np.arange(D) * 2.0 ** -133]
    v += [np.arange(D) - 200.0, np.arange(D) + 1.0]
    for _ in range(40):
        v.append(g.standard_normal(D) * np.exp(4 * g.standard_normal()))
    for _ in range(20):                                       # few bits: many exact ties
        v.append(g.integers(-8, 9, D) / 4.0 * 2.0 ** g.integers(-3, 4))
    x = np.array(v)
    for bad in (np.nan, np.inf, -np.inf):
        y = g.standard_normal(D)
        y[g.integers(0, D)] = bad
        x = np.concatenate([x, y[None]])
    with np.errstate(over="ignore"):
        x = x.astype(np.float32)
    if f32:
        return x
    import torch
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("f32", [False, True])
def test_append_is_exact_on_hard_vectors(D, f32):
    import torch
    g = np.random.default_rng(D + f32)
    x = _hard_vectors(D, g, f32)
    n = len(x)
    dt = torch.float32 if f32 else torch.bfloat16
    c = _cache(-(-n // 32), 1, D, 32, 1)
    k = torch.from_numpy(x).cuda().to(dt)
    v = k.flip(0).contiguous()
    c.append(k, v, _i32(np.arange(n)))
    got = R.unpack(c.pages.cpu().numpy(), D)
    for part, xs in zip(got, (x, x[::-1])):
        codes, s, z = (a.reshape(-1, *a.shape[3:])[:n] for a in part)
        for i in range(n):
            ce, se, ze = R.quantise_exact(xs[i])
            assert (s[i] == se or (np.isnan(s[i]) and np.isnan(se))) and z[i] == ze, (i, s[i], se, z[i], ze)
            assert np.array_equal(codes[i], ce), (i, codes[i], ce)
    c.check()


@pytest.mark.parametrize("D,heads,page,f32,extra", [(128, 3, 16, False, 0), (64, 5, 64, False, 64), (128, 8, 128, True, 256),
                                                    (64, 1, 32, True, 8), (128, 1, 64, False, 8)])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 37])
def test_append_and_read_through_scattered_slots(D, heads, page, f32, extra, n):
    """Random slots, skipped ones (-1), a row map, strided rows; untouched bytes
    and rows stay as they were; fp32 and bf16 values."""
    import torch
    g = np.random.default_rng(n * 100 + D + heads)
    dt = torch.float32 if f32 else torch.bfloat16
    n_pages = 4 + n // page
    c = _cache(n_pages, heads, D, page, n_pages, fill=0xA5)
    before = c.pages.cpu().numpy()
    slots = g.permutation(n_pages * page)[:n]
    slots[g.random(n) < 0.2] = -1
    rows = g.integers(0, n + 3, n)
    kv = torch.randn((n + 3, 2 * heads * D + extra), generator=torch.Generator().manual_seed(n)).cuda().to(dt)
    k, v = kv[:, : heads * D], kv[:, heads * D: 2 * heads * D]
    c.append(k, v, _i32(slots), rows=_i32(rows))
    c.check()
    pages = c.pages.cpu().numpy()
    want = before.copy()
    live = [i for i in range(n) if slots[i] >= 0]
    if live:
        f = lambda t: t.double().cpu().numpy().reshape(n + 3, heads, D)[rows[live]]  # noqa: E731
        packed = R.pack(f(k), f(v), n_pages, page, slots[live], fill=0)
        mask = R.pack(f(k) * 0, f(v) * 0, n_pages, page, slots[live], fill=255) != 255
        # bytes that belong to the tokens: everything pack() wrote (zero vectors write 0x00 and 0x4300)
        want[mask] = packed[mask]
    assert np.array_equal(pages, want)
    for odt in (torch.float32, torch.bfloat16):
        ko = torch.full((n, heads * D + 8), 7.0, dtype=odt, device="cuda")
        vo = torch.full((n, heads * D + 8), 7.0, dtype=odt, device="cuda")
        c.read(_i32(slots), ko[:, : heads * D], vo[:, : heads * D])
        for x, o in ((k, ko), (v, vo)):
            ref = np.full((n, heads * D + 8), 7.0)
            if live:
                cd, s, z = R.quantise(x.double().cpu().numpy().reshape(n + 3, heads, D)[rows[live]])
                ref[live, : heads * D] = ((cd - z[..., None]) * s[..., None]).reshape(len(live), -1)
            ref = torch.from_numpy(ref).to(odt)
            assert torch.equal(o.cpu(), ref)
    c.check()


def test_append_and_read_report_bad_indexes_and_touch_nothing():
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    c = _cache(2, 2, 64, 16, 2, fill=9)
    k = torch.ones((3, 128), dtype=torch.bfloat16, device="cuda")
    for slots, rows in (([32, -1, 1 << 30], None), ([-1, 0, -5], [0, 3, 1]), ([0, -1, -1], [-1, 0, 0])):
        c.append(k, k, _i32(slots), rows=None if rows is None else _i32(rows))
        with pytest.raises(LA.LAError) as e:
            c.check()
        assert e.value.code == LA.LA_ERR_ARG
        c.check()
        assert (c.pages == 9).all()
    out = torch.full((3, 128), 5.0, device="cuda")
    c.read(_i32([32, -1, -7]), out, out.clone())
    with pytest.raises(LA.LAError):
        c.check()
    assert (out == 5).all()
    with pytest.raises(ValueError):
        c.append(k, k[:2], _i32([0]))
    with pytest.raises(ValueError):
        c.append(k.half(), k.half(), _i32([0]))
    with pytest.raises(ValueError):
        c.append(k, k, _i32([0]).long())
    with pytest.raises(LA.LAError):
        c.append(k, k, _i32([0, 1, 2, 3]))  # four slots, three rows


def test_read_past_32_bit_byte_offsets():
    """A pool of more than 4 GB: the last page's tokens land and come back."""
    import torch
    heads, D, page = 64, 128, 128
    n_pages = (5 << 30) // (heads * 8 * 2176)
    c = _cache(n_pages, heads, D, page, n_pages)
    slots = _i32([0, n_pages * page - 1, n_pages // 2 * page + 77])
    k = torch.randn((3, heads * D), device="cuda")
    v = torch.randn((3, heads * D), device="cuda")
    c.append(k, v, slots)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    c.read(slots, ko, vo)
    c.check()
    for x, o in ((k, ko), (v, vo)):
        cd, s, z = R.quantise(x.double().cpu().numpy().reshape(3, heads, D))
        assert np.array_equal(o.double().cpu().numpy(), ((cd - z[..., None]) * s[..., None]).reshape(3, -1))


# --------------------------------------------------------- plan and release

def _plan_case(B, page, lo, hi, new_hi, stride, seed, spare=3, extra_slots=0):
    g = np.random.default_rng(seed)
    lens, new = g.integers(lo, hi + 1, B), g.integers(0, new_hi + 1, B)
    lens[g.random(B) < 0.1] = -1
    mp = -(-(hi + new_hi) // page) + 1
    used = [max(0, -(-int(n) // page)) for n in lens]
    need = sum(-(-int(n + k) // page) - -(-int(n) // page) for n, k in zip(lens, new) if n >= 0)
    order = g.permutation(sum(used) + need + spare)
    table, at = np.full((B, mp), -7), 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    n_slots = B * stride if stride else int(sum(k for n, k in zip(lens, new) if n >= 0)) + extra_slots
    return lens, new, order[at:], need + spare, table, n_slots, len(order)


@pytest.mark.parametrize("B,page,lo,hi,new_hi,stride,extra", [
    (1, 16, 0, 0, 1, 0, 0), (1, 64, 17, 17, 300, 0, 5), (8, 16, 0, 60, 5, 8, 0), (37, 32, 0, 100, 40, 0, 3),
    (1000, 128, 0, 3000, 6, 6, 0), (1025, 64, 0, 700, 3, 3, 0), (8192, 16, 0, 40, 9, 0, 1), (300, 64, 0, 500, 400, 0, 2),
    (5, 16, 0, 9, 0, 0, 0), (5, 16, 0, 9, 0, 4, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_against_the_walk(B, page, lo, hi, new_hi, stride, extra, in_place):
    import torch
    lens, new, free, n_free, table, n_slots, n_pages = _plan_case(B, page, lo, hi, new_hi, stride, B + page, extra_slots=extra)
    want = R.plan(lens, new, free, n_free, table, n_slots, stride, page)
    c = _cache(n_pages, 1, 64, page, table.shape[1])
    d_lens, d_new, d_free, d_nf, d_table = _i32(lens), _i32(new), _i32(free), _i32([n_free]), _i32(table)
    slots = torch.full((n_slots,), 99, dtype=torch.int32, device="cuda")
    nl = d_lens if in_place else torch.full((B,), 99, dtype=torch.int32, device="cuda")
    left = d_nf if in_place else torch.full((1,), 99, dtype=torch.int32, device="cuda")
    c.plan(d_lens, d_new, d_free, d_nf, d_table, slots, nl, left, stride=stride)
    c.check()
    assert np.array_equal(slots.cpu().numpy(), want[0])
    assert np.array_equal(d_table.cpu().numpy(), want[1])
    assert np.array_equal(nl.cpu().numpy(), want[2]) and int(left) == want[3]


@pytest.mark.parametrize("what", ["pages", "slots", "stride", "row", "negative", "free"])
@pytest.mark.parametrize("big", [False, True])
def test_plan_is_all_or_nothing(what, big):
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    B, page, stride = (400, 16, 0) if big else (6, 16, 0)
    lens, new, free, n_free, table, n_slots, n_pages = _plan_case(B, page, 1, 50, 60 if big else 9, stride, 3, spare=0)
    lens = np.maximum(lens, 0)
    new[1] = 30
    lens, new = np.minimum(lens, 50), new
    table = np.where(table < 0, 0, table)
    need = sum(-(-int(n + k) // page) - -(-int(n) // page) for n, k in zip(lens, new))
    free, n_free, n_slots = np.arange(need), need, int(new.sum())
    mp = table.shape[1] + 2
    table = np.concatenate([table, np.zeros((B, 2), int)], 1)
    code = LA.LA_ERR_CAPACITY
    if what == "pages":
        n_free -= 1
    elif what == "slots":
        n_slots -= 1
    elif what == "stride":
        stride, n_slots = 29, 29 * B
        new = np.minimum(new, 29)
        new[1] = 30
    elif what == "row":
        lens[2] = mp * page - 3
        new[2] = 4
    elif what == "negative":
        new[B - 1] = -1
        code = LA.LA_ERR_ARG
    else:
        n_free = -1
        code = LA.LA_ERR_ARG
    c = _cache(8, 1, 64, page, mp)
    d = [_i32(x) for x in (lens, new, free, [n_free], table)]
    slots = torch.full((n_slots,), 99, dtype=torch.int32, device="cuda")
    nl, left = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    c.plan(*d, slots, nl, left, stride=stride)
    with pytest.raises(LA.LAError) as e:
        c.check()
    assert e.value.code == code
    assert (slots == -1).all() and np.array_equal(nl.cpu().numpy(), lens) and int(left) == n_free
    assert np.array_equal(d[4].cpu().numpy(), table)


@pytest.mark.parametrize("B", [1, 7, 1500])
def test_release_gives_pages_back_in_order(B):
    import lossless_lookahead_decoding_gb300 as LA
    g = np.random.default_rng(B)
    page, mp = 16, 9
    lens = g.integers(-1, mp * page + 1, B)
    done = g.integers(0, 2, B)
    used = [max(0, -(-int(n) // page)) for n in lens]
    order = g.permutation(sum(used) + 4)
    table, at = np.full((B, mp), -1), 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    free = np.concatenate([order[at:], np.full(sum(used), -3)])
    stack = list(order[at:])
    for b in range(B):
        if done[b]:
            stack += table[b, :used[b]].tolist()
    c = _cache(len(order), 1, 64, page, mp)
    d_lens, d_free, d_nf = _i32(lens), _i32(free), _i32([4])
    c.release(_i32(done), d_lens, _i32(table), d_free, d_nf)
    c.check()
    assert int(d_nf) == len(stack) and d_free.cpu().numpy()[:len(stack)].tolist() == stack
    assert np.array_equal(d_lens.cpu().numpy(), np.where((done != 0) & (lens > 0), 0, lens))
    # given back once more: there are not that many pages
    if sum(u for u, x in zip(used, done) if x) > 0:
        d_lens, before = _i32(lens), d_free.clone()
        c.release(_i32(np.ones(B)), d_lens, _i32(table), d_free, _i32([len(order) - sum(used) + 1]))
        with pytest.raises(LA.LAError):
            c.check()
        assert np.array_equal(d_lens.cpu().numpy(), lens) and bool((d_free == before).all())


# ---------------------------------------------------------------- attention

def _attend_case(H, Hkv, D, W, N, G, lens, page, seed, extra=0, spread=1.0):
    """Device inputs of one call and the host copies of the cached vectors."""
    import torch
    g = np.random.default_rng(seed)
    B, T = len(lens), 1 + (W + G) * (N - 1)
    need = [max(0, -(-n // page)) for n in lens]
    n_pages = sum(need) + 2
    order = g.permutation(n_pages)
    mp = max(1, max(need)) + 1
    table, at, slots = np.full((B, mp), -1), 0, []
    for b, (n, u) in enumerate(zip(lens, need)):
        table[b, :u] = order[at:at + u]
        at += u
        pos = np.arange(max(n, 0))
        slots.append(table[b, pos // page] * page + pos % page)
    total = sum(max(n, 0) for n in lens)
    kc, vc = g.standard_normal((2, total, Hkv, D)) * spread
    c = _cache(n_pages, Hkv, D, page, mp, fill=255)  # unwritten bytes: NaN scales
    if total:
        t = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
        c.append(t(kc.reshape(total, -1)), t(vc.reshape(total, -1)), _i32(np.concatenate(slots)))
    vals = []
    for x in (kc, vc):
        cd, s, z = R.quantise(x.astype(np.float32)) if total else (np.zeros((0, Hkv, D)), np.zeros((0, Hkv)), np.zeros((0, Hkv)))
        vals.append((cd - z[..., None]) * s[..., None])
    qkv = torch.from_numpy(g.standard_normal((B * T, (H + 2 * Hkv) * D + extra)).astype(np.float32)).cuda().to(torch.bfloat16)
    return c, qkv, _i32(lens), _i32(table), vals


def _call(c, qkv, lens, table, H, W, N, G, out=None, ws=None, max_len=0):
    import torch
    D, Hkv = c.head_dim, c.n_kv_heads
    if out is None:
        out = torch.full((qkv.shape[0], H * D), 77.0, dtype=torch.bfloat16, device="cuda")
    if ws is None:
        ws = torch.full((c.attention_bytes(lens.shape[0], H, W, N, G, max_len),), 255, dtype=torch.uint8, device="cuda")
    c.attention(qkv[:, : H * D], qkv[:, H * D: (H + Hkv) * D], qkv[:, (H + Hkv) * D: (H + 2 * Hkv) * D], lens, table, W, N, G,
                out=out, workspace=ws, max_len=max_len)
    return out


def _verify(out, qkv, lens, vals, H, Hkv, D, W, N, G, only=None):
    T, at = 1 + (W + G) * (N - 1), 0
    x = qkv.double().cpu().numpy()[:, : (H + 2 * Hkv) * D].reshape(len(lens), T, H + 2 * Hkv, D)
    got = out.double().cpu().numpy().reshape(len(lens), T, H, D)
    for b, n in enumerate(lens):
        if n < 0:
            assert (got[b] == 77).all()
            continue
        if only is None or b in only:
            want, spread = R.attention(x[b, :, :H], x[b, :, H:H + Hkv], x[b, :, H + Hkv:], vals[0][at:at + n], vals[1][at:at + n],
                                       W, N, G)
            err = np.linalg.norm(got[b] - want, axis=-1)
            tol = 1.1 * 2.0 ** -8 * (np.linalg.norm(want, axis=-1) + spread)
            assert np.isfinite(got[b]).all() and (err <= tol).all(), (b, n, float((err / tol).max()), np.unravel_index(np.argmax(err / tol), err.shape))
        at += max(n, 0)


SHAPES = [  # heads, KV heads, head_dim
    (1, 1, 64), (4, 4, 64), (8, 8, 128), (16, 2, 128), (6, 2, 64), (20, 1, 128), (9, 3, 128), (40, 8, 128)]
STEPS = [(0, 2, 0), (1, 2, 0), (0, 2, 1), (4, 3, 4), (2, 4, 2), (15, 5, 15), (7, 5, 7), (5, 2, 0), (0, 6, 3), (0, 17, 1),
         (0, 128, 1), (31, 2, 31), (127, 2, 0)]
LENS = [[0], [1], [15], [16], [17], [129], [0, 1, 64, -1, 33], [300, 5, 0, 127, 128]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention_single_tokens(shape, lens):
    H, Hkv, D = shape
    page = 16 << (len(lens) % 4)
    c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, 0, 2, 0, lens, page, 7, extra=8)
    out = _call(c, qkv, dl, dt, H, 0, 2, 0)
    c.check()
    _verify(out, qkv, lens, vals, H, Hkv, D, 0, 2, 0)


@pytest.mark.parametrize("lens", [[0], [21], [130, 0, -1, 16]], ids=str)
@pytest.mark.parametrize("step", STEPS, ids=str)
@pytest.mark.parametrize("shape", [(4, 4, 64), (4, 2, 128), (8, 1, 128)], ids=str)
def test_attention_step_rows(shape, step, lens):
    H, Hkv, D = shape
    c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, *step, lens, 32, 11)
    out = _call(c, qkv, dl, dt, H, *step)
    c.check()
    _verify(out, qkv, lens, vals, H, Hkv, D, *step)


@pytest.mark.parametrize("case", [
    dict(H=32, Hkv=32, D=128, step=(15, 5, 15), lens=[2048], page=64),
    dict(H=64, Hkv=8, D=128, step=(7, 5, 7), lens=[1111], page=16),
    dict(H=64, Hkv=8, D=128, step=(0, 2, 0), lens=[9000, 3, 0, 700, -1, 8191], page=128),
    dict(H=4, Hkv=1, D=64, step=(0, 2, 0), lens=[20011], page=32),
    dict(H=32, Hkv=32, D=128, step=(0, 2, 0), lens=list(range(0, 480, 4)), page=16),
    dict(H=12, Hkv=12, D=64, step=(2, 4, 2), lens=[513, 40, 1000, 0, 77, 250], page=64),
], ids=lambda c: f"{c['H']}x{c['Hkv']}x{c['D']}-{c['step']}-{len(c['lens'])}")
def test_attention_large(case):
    """Items split over workers and joined, ragged batches; a few sequences of
    each are compared."""
    H, Hkv, D, step, lens = case["H"], case["Hkv"], case["D"], case["step"], case["lens"]
    c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, *step, lens, case["page"], 5)
    out = _call(c, qkv, dl, dt, H, *step)
    c.check()
    _verify(out, qkv, lens, vals, H, Hkv, D, *step, only=set(range(0, len(lens), max(1, len(lens) // 9))))
    # equal calls, equal bits, whatever the workspace held; a bound on the lengths changes the split only
    import torch
    assert torch.equal(out, _call(c, qkv, dl, dt, H, *step))
    other = _call(c, qkv, dl, dt, H, *step, max_len=max(lens))
    _verify(other, qkv, lens, vals, H, Hkv, D, *step, only={0})


def test_attention_scores_of_any_size():
    """Scores far apart (one key takes all), all equal, and growing along the
    context (the running maximum moves in every tile)."""
    import torch
    H = Hkv = 2
    D, n = 128, 400
    for mode in range(3):
        c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, 0, 2, 0, [n], 16, 3)
        k = np.zeros((n, Hkv, D))
        if mode == 0:
            k[137] = 40.0
        elif mode == 2:
            k += np.arange(n)[:, None, None] * 0.25
        slots = dt[0].cpu().numpy()[np.arange(n) // 16] * 16 + np.arange(n) % 16
        t = lambda a: torch.from_numpy(a.reshape(n, -1).astype(np.float32)).cuda()  # noqa: E731
        c.append(t(k), t(vals[1]), _i32(slots))
        new = []
        for x in (k, vals[1]):
            cd, s, z = R.quantise(x.astype(np.float32))
            new.append((cd - z[..., None]) * s[..., None])
        qkv[:, : H * D] = qkv[:, : H * D].abs()
        out = _call(c, qkv, dl, dt, H, 0, 2, 0)
        _verify(out, qkv, [n], new, H, Hkv, D, 0, 2, 0)


@pytest.mark.parametrize("shape", [(4, 4, 64), (4, 2, 128), (64, 4, 128)], ids=str)
def test_attention_hidden_nonfinite_rows_reach_no_other_row(shape):
    """NaN and infinities in the step rows of one candidate, in K, V or both:
    rows that see them are not finite, the others as if they were not there."""
    import torch
    H, Hkv, D = shape
    W, N, G = 2, 3, 3
    T = 1 + (W + G) * (N - 1)
    lens = [37]
    bad = 1 + W * (N - 1) + 2  # first row of candidate 1
    sees = [i for i in range(T) if bad in R.visible(W, N, G, i)]
    for which in ("k", "v"):
        for value in (float("nan"), float("inf"), float("-inf")):
            c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, W, N, G, lens, 16, 13)
            clean = _call(c, qkv, dl, dt, H, W, N, G)
            at = (H + (0 if which == "k" else Hkv)) * D
            poisoned = qkv.clone()
            poisoned[bad, at + 3: at + Hkv * D: D] = value
            out = _call(c, poisoned, dl, dt, H, W, N, G)
            rest = [i for i in range(T) if i not in sees]
            assert torch.equal(out[rest], clean[rest]), (which, value)
            o = out.float().reshape(T, H, D)[sees]
            if which == "v":
                assert (~torch.isfinite(o[:, :, 3])).all()
                keep = [d for d in range(D) if d != 3]
                assert torch.equal(o[:, :, keep], clean.float().reshape(T, H, D)[sees][:, :, keep])
            elif value != value:
                assert torch.isnan(o).all()


def test_attention_bad_pages_and_lengths():
    """A page index outside the pool counts as no keys, a length over its bound
    leaves the sequence's rows alone; both are reported, nothing else moves."""
    import lossless_lookahead_decoding_gb300 as LA
    H, Hkv, D, lens = 8, 4, 128, [40, 50, 33]
    for step in ((0, 2, 0), (4, 3, 4), (15, 5, 15)):
        c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, *step, lens, 16, 21)
        for bad in (-1, c.pages.shape[0], 1 << 30):
            dt2 = dt.clone()
            dt2[1, 1] = bad
            out = _call(c, qkv, dl, dt2, H, *step)
            with pytest.raises(LA.LAError) as e:
                c.check()
            assert e.value.code == LA.LA_ERR_ARG
            _verify(out, qkv, lens, vals, H, Hkv, D, *step, only={0, 2})
            short = [x.copy() for x in vals]
            keep = np.r_[0:40 + 16, 40 + 32:len(short[0])]
            _verify(out, qkv, [40, 34, 33], [x[keep] for x in short], H, Hkv, D, *step, only={1})
        long = [40, c.max_pages * 16 + 1, 33]
        out = _call(c, qkv, _i32(long), dt, H, *step)
        with pytest.raises(LA.LAError):
            c.check()
        T = qkv.shape[0] // 3
        assert (out[T:2 * T] == 77).all()
        keep = np.r_[0:40, 90:123]
        _verify(out, qkv, [40, -1, 33], [x[keep] for x in vals], H, Hkv, D, *step)
        out = _call(c, qkv, dl, dt, H, *step, max_len=45)
        with pytest.raises(LA.LAError):
            c.check()
        _verify(out, qkv, [40, -1, 33], [x[keep] for x in vals], H, Hkv, D, *step)


def test_attention_refuses_wrong_tensors():
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    H, Hkv, D = 4, 2, 64
    c, qkv, dl, dt, _ = _attend_case(H, Hkv, D, 0, 2, 0, [20, 30], 16, 1)
    out = torch.zeros((2, H * D), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(c.attention_bytes(2, H, 0, 2, 0), dtype=torch.uint8, device="cuda")
    q, k, v = qkv[:, : H * D], qkv[:, H * D: (H + Hkv) * D], qkv[:, (H + Hkv) * D:]
    for bad in [dict(q=q.float()), dict(q=q[:1]), dict(k=k[:, :64]), dict(v=v.cpu()), dict(out=out.float()), dict(out=out.t()),
                dict(dl=dl.long()), dict(dt=dt[:, :1]), dict(dt=dt.t()), dict(W=3)]:
        a = {**dict(q=q, k=k, v=v, dl=dl, dt=dt, out=out, W=0), **bad}
        with pytest.raises(ValueError):
            c.attention(a["q"], a["k"], a["v"], a["dl"], a["dt"], a["W"], 2, 0, out=a["out"], workspace=ws)
    if ws.numel():
        with pytest.raises(LA.LAError):
            c.attention(q, k, v, dl, dt, 0, 2, 0, out=out, workspace=ws[:-16])
    odd = torch.zeros((2, (H + 2 * Hkv) * D + 4), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(LA.LAError):  # rows that are not 16-byte aligned
        c.attention(odd[:, : H * D], odd[:, H * D: (H + Hkv) * D], odd[:, (H + Hkv) * D: (H + 2 * Hkv) * D], dl, dt, 0, 2, 0,
                    out=out, workspace=ws)


@pytest.mark.parametrize("shape,step,lens", [
    ((8, 8, 128), (0, 103, 1), [30]), ((8, 8, 64), (0, 40, 1), [3, 700, 0]), ((8, 2, 128), (15, 5, 15), [300]),
    ((8, 8, 128), (7, 5, 7), [129] * 11), ((32, 4, 128), (0, 2, 0), [777, 30]), ((16, 16, 64), (2, 4, 2), [500, 31])], ids=str)
def test_attention_error_is_that_of_the_output(shape, step, lens):
    """Over many rows of normal data the error is little more than the output's
    rounding to bf16.  That one: uniform within half a step, relative 2^-8 / m
    at a mantissa m in [1, 2), and m log-uniform: rms 2^-8 / sqrt(3) sqrt(3 /
    (8 ln 2)) = 1.66e-3.  The fp16 roundings of probabilities, values and keys
    (rms 2^-11 / sqrt(3) or less of p v each, the keys' times scores of
    order 1) add in squares 3 (2.8e-4)^2: 1.73e-3.  Bound: 1.2 times the first."""
    H, Hkv, D = shape
    c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, *step, lens, 32, 17)
    out = _call(c, qkv, dl, dt, H, *step)
    c.check()
    T = 1 + (step[0] + step[2]) * (step[1] - 1)
    x = qkv.double().cpu().numpy().reshape(len(lens), T, H + 2 * Hkv, D)
    got, at, num, den = out.double().cpu().numpy().reshape(len(lens), T, H, D), 0, 0.0, 0.0
    for b, n in enumerate(lens):
        want, _ = R.attention(x[b, :, :H], x[b, :, H:H + Hkv], x[b, :, H + Hkv:], vals[0][at:at + n], vals[1][at:at + n], *step)
        num, den, at = num + ((got[b] - want) ** 2).sum(), den + (want ** 2).sum(), at + n
    bound = 1.2 * 2.0 ** -8 / np.sqrt(3) * np.sqrt(3 / (8 * np.log(2)))
    assert np.sqrt(num / den) <= bound, (np.sqrt(num / den), bound)


@pytest.mark.parametrize("step,H", [((0, 16, 1), 1), ((0, 16, 1), 2), ((7, 3, 0), 1)], ids=str)
def test_attention_rows_past_32_bit_offsets(step, H):
    """Step rows so far apart that row offsets pass 2^31 elements."""
    import torch
    D, W, N, G = 64, *step
    T, ld = 1 + (W + G) * (N - 1), 1 << 28
    c, qkv, dl, dt, vals = _attend_case(H, 1, D, *step, [70], 16, 23)
    far = torch.empty((T - 1) * ld + (H + 2) * D, dtype=torch.bfloat16, device="cuda").as_strided((T, (H + 2) * D), (ld, 1))
    far.copy_(qkv)
    out = _call(c, far, dl, dt, H, *step, out=torch.full((T, H * D), 77.0, dtype=torch.bfloat16, device="cuda"))
    c.check()
    assert torch.equal(out, _call(c, qkv, dl, dt, H, *step))
    _verify(out, qkv, [70], vals, H, 1, D, *step)


@pytest.mark.parametrize("heads,D", [(2, 64), (9, 128), (13, 64), (40, 128)])
def test_append_and_read_many_heads(heads, D):
    """Numbers of heads that leave parts of the last workers idle."""
    import torch
    n, page = 101, 16
    g = np.random.default_rng(heads)
    c = _cache(9, heads, D, page, 9, fill=0x5A)
    slots = g.permutation(9 * page)[:n]
    k, v = (torch.from_numpy(g.standard_normal((n, heads, D)).astype(np.float32)).cuda().to(torch.bfloat16) for _ in range(2))
    c.append(k, v, _i32(slots))
    want = R.pack(*(x.double().cpu().numpy() for x in (k, v)), 9, page, slots, fill=0x5A)
    assert np.array_equal(c.pages.cpu().numpy(), want)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    c.read(_i32(slots), ko, vo)
    c.check()
    for x, o in ((k, ko), (v, vo)):
        cd, s, z = R.quantise(x.double().cpu().numpy())
        assert torch.equal(o.cpu(), torch.from_numpy((cd - z[..., None]) * s[..., None]).to(torch.bfloat16))


def test_plan_reports_pages_outside_the_pool():
    """A page index outside the pool, held or newly taken: its tokens get no
    slot (and none of another page's), the rest as ever."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    for bad in (-1, 6, 1 << 28, -(1 << 28)):
        c = _cache(6, 1, 64, 16, 4)
        lens, new = [20, 10, 0], [3, 10, 17]
        table = np.array([[0, 1, -1, -1], [2, -1, -1, -1], [-1] * 4])
        free = np.array([3, bad, 4])
        for held in (False, True):
            tb, fr = table.copy(), free.copy()
            if held:
                tb[0, 1], fr[1] = bad, 5
            slots = torch.full((33,), 99, dtype=torch.int32, device="cuda")
            nl, left, dt = _i32([0] * 3), _i32([0]), _i32(tb)
            c.plan(_i32(lens), _i32(new), _i32(fr), _i32([3]), dt, slots, nl, left)
            with pytest.raises(LA.LAError) as e:
                c.check()
            assert e.value.code == LA.LA_ERR_ARG
            got = slots.cpu().numpy()
            # pages taken from the top: sequence 1 gets 4, sequence 2 gets fr[1], then 3
            want = np.r_[(-1, -1, -1) if held else (20, 21, 22), 42:48, 64:68,
                         np.arange(80, 96) if held else np.full(16, -1), 48, [-1] * 3]
            assert np.array_equal(got, want), (bad, held, got)
            assert nl.cpu().numpy().tolist() == [23, 20, 17] and int(left) == 0


@pytest.mark.parametrize("case", [
    dict(H=4, Hkv=2, D=64, step=(0, 2, 0), lens=[40000, 3, 200, 0, -1, 1111], page=16),
    dict(H=4, Hkv=4, D=128, step=(2, 4, 2), lens=[30001, 0, 77, -1, 2050], page=128),
    dict(H=32, Hkv=32, D=64, step=(0, 2, 0), lens=[1000 - 50 * i for i in range(20)], page=32),
    dict(H=32, Hkv=32, D=64, step=(0, 2, 2), lens=[1500 - 170 * i for i in range(9)] + [0, -1, 16], page=64, runs=False),
    dict(H=48, Hkv=48, D=64, step=(0, 2, 2), lens=[3000 - 300 * i for i in range(10)] + [0, -1, 16], page=64),
    dict(H=2, Hkv=2, D=64, step=(15, 5, 15), lens=[33000, 12, 129, -1], page=64),
], ids=lambda c: f"{c['H']}x{c['Hkv']}x{c['D']}-{c['step']}-{len(c['lens'])}")
def test_attention_equal_runs(case):
    """Shapes whose items are cut into equal runs and joined from parts (and one
    that takes them whole), on two streams at once with a workspace each; the
    workspace's bytes do not matter."""
    import torch
    H, Hkv, D, step, lens = case["H"], case["Hkv"], case["D"], case["step"], case["lens"]
    c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, *step, lens, case["page"], 31)
    assert (c.attention_bytes(len(lens), H, *step) > 0) == case.get("runs", True)
    out = _call(c, qkv, dl, dt, H, *step)
    c.check()
    _verify(out, qkv, lens, vals, H, Hkv, D, *step, only=set(range(0, len(lens), max(1, len(lens) // 6))))
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.full_like(out, 77.0) for _ in range(2)]
    ws = [torch.zeros(c.attention_bytes(len(lens), H, *step), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, w in zip(streams, outs, ws):
            with torch.cuda.stream(s):
                _call(c, qkv, dl, dt, H, *step, out=o, ws=w)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 100, 225, 449, 897, 1800])
@pytest.mark.parametrize("shape", [(3, 3, 64), (16, 2, 128), (40, 40, 128), (130, 65, 64), (200, 200, 64)], ids=str)
def test_attention_one_sequence(shape, n):
    """Single tokens over lengths around the tiles that a cluster's warps take,
    for every cluster size; without a workspace where none is asked for."""
    H, Hkv, D = shape
    c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, 0, 2, 0, [n], 64, 37)
    out = _call(c, qkv, dl, dt, H, 0, 2, 0)
    c.check()
    _verify(out, qkv, [n], vals, H, Hkv, D, 0, 2, 0)


def _store(c, dt, n, k, v):
    """Tokens 0..n-1 of sequence 0 from [n, heads, D] arrays; the values held."""
    import torch
    slots = dt[0].cpu().numpy()[np.arange(n) // c.page] * c.page + np.arange(n) % c.page
    t = lambda a: torch.from_numpy(a.reshape(n, -1).astype(np.float32)).cuda()  # noqa: E731
    c.append(t(k), t(v), _i32(slots))
    vals = []
    for x in (k, v):
        cd, s, z = R.quantise(x.astype(np.float32))
        vals.append((cd - z[..., None]) * s[..., None])
    return vals


@pytest.mark.parametrize("step", [(0, 2, 0), (2, 4, 2), (7, 5, 7)], ids=str)
@pytest.mark.parametrize("big", [2.0 ** 10, 2.0 ** 14, 2.0 ** 40, 2.0 ** -40])
@pytest.mark.parametrize("first", [True, False])
def test_attention_values_of_very_different_size(step, big, first):
    """Whole tiles of keys without a value (V = 0) next to large or small ones: they
    still take their share of the weights."""
    H, Hkv, D, n = 4, 2, 128, 384
    c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, *step, [n], 64, 41)
    g = np.random.default_rng(41)
    k, v = g.standard_normal((2, n, Hkv, D))
    v *= big
    v[:256] *= first
    if first:
        v[128:256] = 0
    qkv[:, (H + Hkv) * D: (H + 2 * Hkv) * D] *= big
    held = _store(c, dt, n, k, v)
    out = _call(c, qkv, dl, dt, H, *step)
    c.check()
    _verify(out, qkv, [n], held, H, Hkv, D, *step)


@pytest.mark.parametrize("step", [(0, 2, 0), (2, 4, 2), (7, 5, 7)], ids=str)
def test_attention_nonfinite_cache_and_queries(step):
    """A cached vector with a NaN makes its head's rows NaN and no others; a
    query row with a NaN is NaN in its head, every other row as before."""
    import torch
    H, Hkv, D, n = 4, 2, 64, 300
    T = 1 + (step[0] + step[2]) * (step[1] - 1)
    c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, *step, [n, 40], 32, 43)
    clean = _call(c, qkv, dl, dt, H, *step)
    bad = qkv.clone()
    bad[T - 1, 2 * D + 5] = float("nan")
    out = _call(c, bad, dl, dt, H, *step).reshape(2 * T, H, D)
    assert torch.isnan(out[T - 1, 2]).all()
    out[T - 1, 2] = clean.reshape(2 * T, H, D)[T - 1, 2]
    assert torch.equal(out.reshape(2 * T, -1), clean)
    for part in range(2):
        k, v = (x[:n].copy() for x in vals)
        (k, v)[part][171, 1, 9] = np.nan
        with np.errstate(invalid="ignore"):
            slots = dt[0].cpu().numpy()[171 // 32] * 32 + 171 % 32
        t = lambda a: torch.from_numpy(a[171:172].reshape(1, -1).astype(np.float32)).cuda()  # noqa: E731
        c.append(t(k), t(v), _i32([slots]))
        out = _call(c, qkv, dl, dt, H, *step).reshape(2 * T, H, D)
        assert torch.isnan(out[:T, 2:]).all()
        assert torch.equal(out[:T, :2], clean.reshape(2 * T, H, D)[:T, :2]) and torch.equal(out[T:].reshape(T, -1), clean[T:])
        c.append(t(vals[0]), t(vals[1]), _i32([slots]))
        assert torch.equal(_call(c, qkv, dl, dt, H, *step), clean)


@pytest.mark.parametrize("D", [64, 128])
def test_read_of_hard_vectors(D):
    """Scales from the smallest subnormal to the largest, NaN: fp32 exact, bf16
    rounded once."""
    import torch
    x = _hard_vectors(D, np.random.default_rng(D), True)
    n = len(x)
    c = _cache(-(-n // 16), 1, D, 16, 1)
    k = torch.from_numpy(x).cuda()
    c.append(k, k, _i32(np.arange(n)))
    want = np.full((n, D), np.nan)
    for i in range(n):
        cd, s, z = R.quantise_exact(x[i])
        if not np.isnan(s):
            want[i] = (cd.astype(np.float64) - z) * float(s)
    with np.errstate(over="ignore"):
        w32 = torch.from_numpy(want.astype(np.float32))
    for dt, ref in ((torch.float32, w32), (torch.bfloat16, torch.from_numpy(want).to(torch.bfloat16))):
        ko, vo = torch.zeros((n, D), dtype=dt, device="cuda"), torch.zeros((n, D), dtype=dt, device="cuda")
        c.read(_i32(np.arange(n)), ko, vo)
        for o in (ko.cpu(), vo.cpu()):
            assert torch.equal(torch.isnan(o), torch.isnan(ref))
            assert torch.equal(torch.nan_to_num(o, 0.0), torch.nan_to_num(ref, 0.0))
    c.check()


@pytest.mark.parametrize("step,B", [((0, 2, 0), 9000), ((0, 17, 1), 2000)], ids=str)
def test_attention_many_sequences(step, B):
    lens = [b % 23 - 1 for b in range(B)]
    c, qkv, dl, dt, vals = _attend_case(1, 1, 64, *step, lens, 16, 47)
    out = _call(c, qkv, dl, dt, 1, *step)
    c.check()
    _verify(out, qkv, lens, vals, 1, 1, 64, *step, only=set(range(0, B, B // 40)) | {B - 1})


# ------------------------------------------------------- all of them together

def _serve(graph, steps=6):
    """A ragged batch decoded for some steps: attention over the cache, accepted
    rows planned and appended, one sequence ended and its pages given back.
    Checked against a host copy of the cache after every step."""
    import torch
    H, Hkv, D, page, mp, n_pages = 8, 2, 128, 16, 12, 60
    W, N, G = 2, 3, 2
    T, cap = 1 + (W + G) * (N - 1), N
    B = 4
    g = torch.Generator(device="cuda").manual_seed(5)
    host = np.random.default_rng(5)
    c = _cache(n_pages, Hkv, D, page, mp, fill=255)
    lens = _i32([0] * B)
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    free, n_free = _i32(host.permutation(n_pages)), _i32([n_pages])
    mirror = [[np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))] for _ in range(B)]

    def grow(k, v, rows, counts, starts):
        for b, n in enumerate(counts):
            idx = rows[starts[b]: starts[b] + n]
            for i, x in enumerate((k, v)):
                cd, s, z = R.quantise(x.double().cpu().numpy().reshape(-1, Hkv, D)[idx])
                mirror[b][i] = np.concatenate([mirror[b][i], (cd - z[..., None]) * s[..., None]])

    # prompts: one packed plan and append
    prompts = [33, 1, 64, 17]
    slots = torch.zeros(sum(prompts) + 3, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((sum(prompts), Hkv * D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    c.plan(lens, _i32(prompts), free, n_free, table, slots, lens, n_free)
    c.append(k, v, slots[: sum(prompts)])
    grow(k, v, np.arange(sum(prompts)), prompts, np.cumsum([0] + prompts[:-1]))
    # fixed buffers of a step (what a captured graph replays on)
    qkv = torch.zeros((B * T, (H + 2 * Hkv) * D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((B * T, H * D), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(max(16, c.attention_bytes(B, H, W, N, G)), dtype=torch.uint8, device="cuda")
    n_acc, rows = _i32([0] * B), _i32([0] * (B * cap))
    sl = torch.zeros(B * cap, dtype=torch.int32, device="cuda")
    q_, k_, v_ = qkv[:, : H * D], qkv[:, H * D: (H + Hkv) * D], qkv[:, (H + Hkv) * D:]

    def step():
        c.attention(q_, k_, v_, lens, table, W, N, G, out=out, workspace=ws)
        c.plan(lens, n_acc, free, n_free, table, sl, lens, n_free, stride=cap)
        c.append(k_, v_, sl, rows=rows)

    side = torch.cuda.Stream()
    cg = None
    if graph:
        side.wait_stream(torch.cuda.current_stream())
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg, stream=side):
            step()
    for it in range(steps):
        acc = host.integers(0, cap + 1, B)
        picked = np.concatenate([b * T + np.r_[np.sort(host.permutation(T)[:cap])] for b in range(B)])
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        n_acc.copy_(_i32(acc))
        rows.copy_(_i32(picked))
        now = lens.cpu().numpy().tolist()
        assert now == [len(m[0]) for m in mirror]
        if graph:
            cg.replay()
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        c.check()
        vals = [np.concatenate([m[i] for m in mirror]) for i in range(2)]
        _verify(out, qkv, now, vals, H, Hkv, D, W, N, G)
        grow(k_, v_, picked, acc, [b * cap for b in range(B)])
        if it == 2:
            before, gone = int(n_free), -(-int(lens[2]) // page)
            c.release(_i32([0, 0, 1, 0]), lens, table, free, n_free)
            assert int(n_free) == before + gone and int(lens[2]) == 0
            mirror[2] = [np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))]
    held = [table[b, : -(-int(lens[b]) // page)].cpu().numpy() for b in range(B)]
    everyone = np.concatenate(held + [free.cpu().numpy()[: int(n_free)]])
    assert sorted(everyone.tolist()) == list(range(n_pages))  # no page lost, none twice


def test_serving_loop_on_a_side_stream():
    _serve(False)


def test_serving_loop_replayed_from_a_graph():
    _serve(True)


def test_two_graphs_with_their_own_workspaces_run_side_by_side():
    import torch
    H, Hkv, D, step = 16, 2, 128, (0, 2, 0)
    cases = [_attend_case(H, Hkv, D, *step, [n, 77, 3000], 64, s) for n, s in ((2500, 1), (999, 2))]
    want = [_call(c, qkv, dl, dt, H, *step) for c, qkv, dl, dt, _ in cases]
    graphs, outs, keep = [], [], []
    for c, qkv, dl, dt, _ in cases:
        out = torch.zeros_like(want[0])
        ws = torch.zeros(c.attention_bytes(3, H, *step), dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        cg = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(cg, stream=s):
            for _ in range(5):
                _call(c, qkv, dl, dt, H, *step, out=out, ws=ws)
        graphs.append((cg, s))
        outs.append(out)
        keep.append(ws)
    torch.cuda.synchronize()
    for _ in range(20):
        for cg, s in graphs:
            with torch.cuda.stream(s):
                cg.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("step", [(4, 3, 4), (0, 64, 1)], ids=str)
def test_calls_on_two_streams_with_their_own_workspaces(step):
    """Many rows per KV head: calls that overlap on two streams (some shapes need no workspace)."""
    import torch
    H, Hkv, D = 16, 8, 128
    cases = [_attend_case(H, Hkv, D, *step, [n] + [77, 300] * 8, 64, s) for n, s in ((900, 1), (1500, 2))]
    want = [_call(c, qkv, dl, dt, H, *step) for c, qkv, dl, dt, _ in cases]
    outs = [torch.zeros_like(w) for w in want]
    ws = [torch.zeros(c.attention_bytes(17, H, *step), dtype=torch.uint8, device="cuda") for c, *_ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for (c, qkv, dl, dt, _), o, w, s in zip(cases, outs, ws, streams):
            with torch.cuda.stream(s):
                _call(c, qkv, dl, dt, H, *step, out=o, ws=w)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing has to run before a capture: kernels are set up while it goes on."""
    import os
    import subprocess
    import sys
    code = """
import torch, lossless_lookahead_decoding_gb300 as LA
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
c = LA.KV4Cache(LA.KV4Cache.empty_pages(4, 2, 128, 16), 16, 4)
lens, new, free, nf, table = i32([0]), i32([5]), i32([3, 2, 1, 0]), i32([4]), i32([[-1] * 4])
slots = i32([0] * 8)
k = torch.randn((8, 256), device="cuda").to(torch.bfloat16)
q, q2 = torch.randn((1, 512), device="cuda").to(torch.bfloat16), torch.randn((40, 512), device="cuda").to(torch.bfloat16)
k2 = torch.randn((40, 256), device="cuda").to(torch.bfloat16)
o, o2 = torch.zeros_like(q), torch.zeros_like(q2)
b = [torch.empty(max(16, c.attention_bytes(1, 4, 0, n, g)), dtype=torch.uint8, device="cuda") for n, g in ((2, 0), (40, 1))]
torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    c.plan(lens, new, free, nf, table, slots, lens, nf, stride=8)
    c.append(k, k, slots)
    c.attention(q, k[:1], k[:1], lens, table, 0, 2, 0, out=o, workspace=b[0])
    c.attention(q2, k2, k2, lens, table, 0, 40, 1, out=o2, workspace=b[1])
gr.replay()
torch.cuda.synchronize()
c.check()
assert int(lens) == 5 and int(nf) == 3 and bool(o.any()) and bool(o2.any())
gr.replay()
torch.cuda.synchronize()
c.check()
assert int(lens) == 10 and int(nf) == 3
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=300)


# ------------------------------------- many rows, sequences without cached tokens

EMPTY_BETWEEN = [  # heads, KV heads, head_dim, step, lens: more than 152 items, so equal runs of them
    (8, 8, 64, (0, 128, 1), [0] + [64] * 40),
    (5, 5, 128, (0, 128, 1), ([0, 0, 11, 0, 300, 0, 0, 0, 5] + [0] * 9 + [129, 0, 250]) * 3),
    (32, 32, 64, (0, 17, 1), ([0] * 7 + [3, 0, 0, 40, 1]) * 3),
    (8, 1, 128, (2, 4, 2), [0, 0, 0, 0, 0, 7] * 30 + [0] * 20 + [200, 0, 0, 0, 13]),
    (64, 4, 128, (7, 5, 7), [0, 30, 0, 0, 400, 0]),
]


@pytest.mark.parametrize("case", EMPTY_BETWEEN, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}-{c[3]}-{len(c[4])}")
def test_attention_empty_sequences_between_others(case):
    """First blocks of prompts in a batch with running sequences: items that hold
    the step's own rows only, many in a row, before, between and after others."""
    import torch
    H, Hkv, D, step, lens = case
    c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, *step, lens, 16, 61)
    out = _call(c, qkv, dl, dt, H, *step)
    c.check()
    _verify(out, qkv, lens, vals, H, Hkv, D, *step)
    for _ in range(3):
        assert torch.equal(out, _call(c, qkv, dl, dt, H, *step))
    c.check()


@pytest.mark.parametrize("case", EMPTY_BETWEEN[:3], ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}-{c[3]}-{len(c[4])}")
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_attention_nonfinite_values_of_empty_sequences(case, value):
    """A value that is not finite in the last own row of sequences without cached
    tokens reaches that row and channel alone: everything else is as with a zero
    in its place, bit for bit."""
    import torch
    H, Hkv, D, step, lens = case
    T = 1 + (step[0] + step[2]) * (step[1] - 1)
    c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, *step, lens, 16, 67)
    rows = torch.tensor([b * T + T - 1 for b, n in enumerate(lens) if n == 0], device="cuda")
    at = (H + Hkv) * D + torch.arange(Hkv, device="cuda") * D + 3
    qkv[rows[:, None], at[None]] = 0.0
    clean = _call(c, qkv, dl, dt, H, *step)
    _verify(clean, qkv, lens, vals, H, Hkv, D, *step)
    odd = qkv.clone()
    odd[rows[:, None], at[None]] = value
    out = _call(c, odd, dl, dt, H, *step)
    c.check()
    touched = torch.arange(H, device="cuda") * D + 3
    assert not torch.isfinite(out[rows[:, None], touched[None]]).any()
    out[rows[:, None], touched[None]] = clean[rows[:, None], touched[None]]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_new", [3, 20000])
def test_plan_refuses_more_free_pages_than_there_are(n_new, in_place):
    """A page count over n_pages: nothing is planned; the count itself is allowed."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    page, n_pages = 128, 200
    c = _cache(n_pages, 1, 64, page, n_pages)
    free = np.r_[np.arange(n_pages), np.zeros(8, int)]
    for n_free in (n_pages + 1, n_pages + 8, 1 << 30, n_pages):
        lens, nf = _i32([0]), _i32([n_free])
        table = torch.full((1, n_pages), -7, dtype=torch.int32, device="cuda")
        slots = torch.full((n_new,), 99, dtype=torch.int32, device="cuda")
        nl, left = (lens, nf) if in_place else (_i32([5]), _i32([5]))
        c.plan(lens, _i32([n_new]), _i32(free), nf, table, slots, nl, left)
        if n_free == n_pages:
            c.check()
            pages = -(-n_new // page)
            assert int(nl) == n_new and int(left) == n_pages - pages
            assert table[0, :pages].tolist() == list(range(n_pages - 1, n_pages - 1 - pages, -1)) and int(slots[0]) == (n_pages - 1) * page
            continue
        with pytest.raises(LA.LAError) as e:
            c.check()
        assert e.value.code == LA.LA_ERR_ARG
        assert bool((slots == -1).all()) and bool((table == -7).all()) and int(nl) == 0 and int(left) == n_free


def test_plan_refuses_an_output_over_the_free_pages():
    """KV4Cache knows how long the stack's buffer is; neighbours in one buffer are fine."""
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    c = _cache(6, 1, 64, 16, 4)
    buf = torch.zeros(40, dtype=torch.int32, device="cuda")
    free, lens, new = buf[:6], _i32([0, 5]), _i32([2, 12])
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    free.copy_(torch.arange(6))
    other = dict(table=table, slots=_i32([9] * 14), new_lens=_i32([9, 9]), left=_i32([9]))
    table[1, 0] = 5
    for bad in (dict(slots=buf[5:19]), dict(slots=buf[2:16]), dict(table=buf[4:12].view(2, 4)), dict(new_lens=buf[5:7]),
                dict(left=buf[3:4])):
        a = {**other, **bad}
        with pytest.raises((ValueError, LA.LAError)):
            c.plan(lens, new, free, _i32([5]), a["table"], a["slots"], a["new_lens"], a["left"])
    assert free.tolist() == list(range(6))
    c.plan(lens, new, free, _i32([5]), table, buf[6:20], buf[20:22], buf[22:23])
    c.check()
    assert buf[6:23].tolist() == [64, 65, *range(85, 96), 48, 2, 17, 3] and table[:, 0].tolist() == [4, 5] and int(table[1, 1]) == 3


@pytest.mark.parametrize("f32", [False, True])
def test_single_rows_of_any_stride(f32):
    """One token whose k is a tensor of its own and whose v (and q) are views into
    a projection: a single row has no stride to differ in."""
    import torch
    H = Hkv = 2
    D, n = 64, 20
    c, qkv, dl, dt, vals = _attend_case(H, Hkv, D, 0, 2, 0, [n], 16, 71, extra=8)
    want = _call(c, qkv, dl, dt, H, 0, 2, 0)
    q, v = qkv[:, :H * D], qkv[:, 2 * H * D: 3 * H * D]
    k = v.new_empty((1, H * D)).copy_(qkv[:, H * D: 2 * H * D])
    assert k.stride(0) != v.stride(0)
    ws = torch.zeros(max(16, c.attention_bytes(1, H, 0, 2, 0)), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    c.attention(q, k, v, dl, dt, 0, 2, 0, out=out, workspace=ws)
    assert torch.equal(out, want)
    dtype = torch.float32 if f32 else torch.bfloat16
    k, x = k.to(dtype), torch.cat([v, v, v[:, :8]], 1).to(dtype)
    v = x[:, H * D: 2 * H * D]
    assert k.stride(0) != v.stride(0)
    slot = dt[0, :1] * 16 + 3
    c.append(k, v, slot)
    ko, vo = torch.zeros_like(k), torch.zeros_like(x)[:, :H * D]
    c.read(slot, ko, vo)
    c.check()
    for a, b in ((k, ko), (v, vo)):
        cd, s, z = R.quantise(a.double().cpu().numpy().reshape(1, Hkv, D))
        ref = torch.from_numpy(((cd - z[..., None]) * s[..., None]).reshape(1, -1)).to(dtype)
        assert torch.equal(b.cpu(), ref)
