"""The paged 4-bit KV cache's entry points on the host: sizing and the calls
they refuse before anything reaches a GPU, and the test reference's own pins."""
import ctypes as C
from fractions import Fraction as F

import numpy as np
import pytest

import kv4_ref as R
from helpers import build_lib

FAKE = 1 << 20  # never dereferenced: every call here is refused


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def _desc(**kw):
    import lossless_lookahead_decoding_gb300 as LA
    f = dict(n_kv_heads=8, head_dim=128, page=64, n_pages=100, max_pages=16, pages=FAKE, status=None)
    f.update(kw)
    return LA.la_kv4_desc(**f)


def _attn(**kw):
    import lossless_lookahead_decoding_gb300 as LA
    f = dict(q=FAKE, k_step=FAKE, v_step=FAKE, out=FAKE, lens=FAKE, table=FAKE, batch=2, n_heads=64, W=0, N=2, G=0,
             q_ld=64 * 128, kv_ld=8 * 128, max_len=0, workspace=None, ws_bytes=0)
    f.update(kw)
    return LA.la_kv4_attn(**f)


BAD_DESC = [dict(head_dim=96), dict(head_dim=0), dict(n_kv_heads=0), dict(n_kv_heads=1025), dict(page=8), dict(page=48),
            dict(page=256), dict(n_pages=0), dict(n_pages=1 << 25), dict(max_pages=0), dict(max_pages=1 << 25)]


def test_page_bytes():
    import lossless_lookahead_decoding_gb300 as LA
    assert LA.la_kv4_page_bytes(_desc()) == 8 * 4 * (16 * 128 + 128)
    assert LA.la_kv4_page_bytes(_desc(head_dim=64, page=16, n_kv_heads=3)) == 3 * (16 * 64 + 128)
    assert LA.lib().la_kv4_page_bytes(None) == 0
    for bad in BAD_DESC:
        assert LA.la_kv4_page_bytes(_desc(**bad)) == 0, bad


def test_append_and_read_refusals():
    import lossless_lookahead_decoding_gb300 as LA
    E = LA.LA_ERR_ARG
    ok = dict(k=FAKE, v=FAKE, dtype=LA.LA_BF16, ld=1024, n_rows=5, rows=None, slots=FAKE, n=5)

    def append(desc=None, **kw):
        a = {**ok, **kw}
        return LA.la_kv4_append(desc or _desc(), a["k"], a["v"], a["dtype"], a["ld"], a["n_rows"], a["rows"], a["slots"], a["n"])

    def read(desc=None, **kw):
        a = {**ok, **kw}
        return LA.la_kv4_read(desc or _desc(), a["slots"], a["n"], a["k"], a["v"], a["dtype"], a["ld"])

    for bad in BAD_DESC + [dict(pages=None), dict(pages=FAKE + 8), dict(status=FAKE + 2)]:
        assert append(_desc(**bad)) == E and read(_desc(**bad)) == E, bad
    for bad in [dict(k=None), dict(v=None), dict(slots=None), dict(k=FAKE + 2), dict(v=FAKE + 8), dict(dtype=2), dict(ld=1023),
                dict(ld=1020), dict(ld=1028), dict(n=-1), dict(dtype=LA.LA_FP32, ld=1026)]:
        assert append(**bad) == E and read(**bad) == E, bad
    assert append(n_rows=4) == E and append(n_rows=-1) == E  # without `rows`, row i is read for slot i
    assert append(n=0) == 0 and read(n=0) == 0               # nothing to do, nothing launched


def test_plan_and_release_refusals():
    import lossless_lookahead_decoding_gb300 as LA
    E = LA.LA_ERR_ARG
    p = [FAKE + 0x10000 * i for i in range(8)]
    ok = dict(lens=p[0], n_new=p[1], batch=4, free=p[2], n_free=p[3], table=p[4], slots=p[5], n_slots=32, stride=8,
              new_lens=p[6], left=p[7])

    def plan(desc=None, **kw):
        a = {**ok, **kw}
        return LA.la_kv4_plan(desc or _desc(), a["lens"], a["n_new"], a["batch"], a["free"], a["n_free"], a["table"],
                              a["slots"], a["n_slots"], a["stride"], a["new_lens"], a["left"])

    for bad in BAD_DESC:
        assert plan(_desc(**bad)) == E, bad
    for bad in [dict(lens=None), dict(n_new=None), dict(free=None), dict(n_free=None), dict(table=None), dict(slots=None),
                dict(new_lens=None), dict(left=None), dict(batch=-1), dict(batch=8193), dict(n_slots=-1), dict(stride=-1),
                dict(n_slots=31), dict(n_slots=40),
                # outputs over inputs or over each other
                dict(new_lens=p[0] + 4), dict(new_lens=p[1]), dict(slots=p[0]), dict(slots=p[1] - 64), dict(slots=p[4] + 8),
                dict(slots=p[6] - 4), dict(table=p[0] - 16), dict(table=p[1]), dict(table=p[6] - 252), dict(left=p[0]),
                dict(left=p[5] + 4), dict(left=p[4] + 252), dict(left=p[6] + 12), dict(left=p[1] + 4)]:
        assert plan(**bad) == E, bad

    def release(desc=None, **kw):
        a = {**ok, **kw}
        return LA.la_kv4_release(desc or _desc(), a["n_new"], a["batch"], a["lens"], a["table"], a["free"], a["n_free"])

    for bad in BAD_DESC:
        assert release(_desc(**bad)) == E, bad
    for bad in [dict(lens=None), dict(n_new=None), dict(free=None), dict(n_free=None), dict(table=None), dict(batch=-1),
                dict(batch=8193)]:
        assert release(**bad) == E, bad
    assert release(batch=0) == 0


def test_attention_refusals_and_sizing():
    import lossless_lookahead_decoding_gb300 as LA
    E = LA.LA_ERR_ARG
    d, a = _desc(), _attn(batch=400)
    need = LA.la_kv4_attention_bytes(d, a)
    assert need > 0  # many sequences of any lengths: items are split
    for bad in BAD_DESC + [dict(pages=None), dict(pages=FAKE + 4), dict(status=FAKE + 1)]:
        assert LA.la_kv4_attention(_desc(**bad), _attn(batch=400, workspace=FAKE, ws_bytes=need)) == E, bad
    shapes = [dict(batch=-1), dict(batch=65536), dict(n_heads=0), dict(n_heads=12), dict(W=-1), dict(G=-1), dict(N=1), dict(N=129),
              dict(W=40, N=5), dict(W=127, N=3), dict(max_len=-1), dict(W=64, G=64, N=2)]
    for bad in shapes:
        assert LA.la_kv4_attention_bytes(d, _attn(**bad)) == 0, bad
    for bad in shapes + [dict(q=None), dict(k_step=None), dict(v_step=None), dict(out=None), dict(lens=None), dict(table=None),
                         dict(q=FAKE + 2), dict(k_step=FAKE + 8), dict(v_step=FAKE + 4), dict(out=FAKE + 8),
                         dict(q_ld=64 * 128 - 8), dict(q_ld=64 * 128 + 4), dict(kv_ld=1016), dict(kv_ld=1028),
                         dict(workspace=None), dict(ws_bytes=need - 1), dict(workspace=FAKE + 8)]:
        assert LA.la_kv4_attention(d, _attn(**{**dict(batch=400, workspace=FAKE, ws_bytes=need), **bad})) == E, bad
    assert LA.lib().la_kv4_attention(None, C.byref(a), None) == E and LA.lib().la_kv4_attention(C.byref(d), None, None) == E
    assert LA.la_kv4_attention(d, _attn(batch=0)) == 0
    # the widest steps and longest chains are accepted
    for good in [dict(W=127, N=2, G=0), dict(W=0, N=128, G=1), dict(W=15, N=5, G=15), dict(batch=65535)]:
        assert LA.la_kv4_attention_bytes(d, _attn(**{**dict(batch=400), **good})) > 0, good


def test_reference_quantiser_pins():
    """bf16_up, ties and the clamp on numbers worked by hand."""
    assert R.bf16_up(F(1)) == 1 and R.bf16_up(F(257, 256)) == F(258, 256) and R.bf16_up(F(256, 255)) == F(258, 256)
    assert R.bf16_up(F(1, 2) ** 140) == F(1, 2) ** 133
    c, s, z = R.quantise_exact(np.array([0.0, 15.0, 0.5, 1.5, 2.5]))
    assert (s, z) == (1.0, 0) and c.tolist() == [0, 15, 0, 2, 2]
    c, s, z = R.quantise_exact(np.array([-7.5, 7.5]))  # z = rne(7.5) = 8, 7.5 / 1 -> 8 + 8 = 16 -> 15
    assert (s, z) == (1.0, 8) and c.tolist() == [0, 15]
    assert R.quantise_exact(np.array([0.0, -0.0]))[1:] == (0.0, 0)
    c, s, z = R.quantise_exact(np.array([1.0, np.inf]))
    assert np.isnan(s) and z == 0 and c.tolist() == [0, 0]
    g = np.random.default_rng(0)
    x = g.standard_normal((50, 64)).astype(np.float32) * np.exp(3 * g.standard_normal((50, 1))).astype(np.float32)
    c, s, z = R.quantise(x)
    for i in range(50):
        ce, se, ze = R.quantise_exact(x[i])
        assert (s[i], z[i]) == (se, ze) and np.array_equal(c[i], ce)


def test_reference_pages_round_trip():
    g = np.random.default_rng(1)
    for D, page in ((64, 16), (128, 32)):
        k, v = g.standard_normal((2, 5, 3, D))
        slots = [0, 17, page + 3, 2 * page - 1, 3 * page]
        pages = R.pack(k, v, 4, page, slots)
        for x, (c, s, z) in zip((k, v), R.unpack(pages, D)):
            want = R.quantise(x)
            for i, sl in enumerate(slots):
                assert np.array_equal(c[sl // page, :, sl % page], want[0][i])
                assert np.array_equal(s[sl // page, :, sl % page], want[1][i])
                assert np.array_equal(z[sl // page, :, sl % page], want[2][i])


def test_reference_mask_matches_the_oracle_controller():
    """The listed visibility is the oracle controller's, for windows with every
    candidate present."""
    import oracle as O
    for W, N, G in ((3, 3, 2), (0, 4, 3), (5, 2, 0), (2, 5, 1), (15, 5, 15)):
        k = O.Controller(W, N, G, 64)
        k.init(np.arange(64, dtype=np.int32), seed=1)
        for g in range(G):
            k.insert(3, [(g * 7 + i) % 64 for i in range(N - 1)])
        _, _, vis = k.rows(3, 0)
        for i in range(len(vis)):
            assert np.nonzero(vis[i])[0].tolist() == sorted(R.visible(W, N, G, i)), (W, N, G, i)


def test_plan_and_release_refuse_shared_buffers():
    """The free pages and their number under an output; all of release's buffers."""
    import lossless_lookahead_decoding_gb300 as LA
    E = LA.LA_ERR_ARG
    p = [FAKE + 0x10000 * i for i in range(8)]
    ok = dict(lens=p[0], n_new=p[1], batch=4, free=p[2], n_free=p[3], table=p[4], slots=p[5], n_slots=32, stride=8,
              new_lens=p[6], left=p[7], done=p[1])

    def plan(**kw):
        a = {**ok, **kw}
        return LA.la_kv4_plan(_desc(), a["lens"], a["n_new"], a["batch"], a["free"], a["n_free"], a["table"],
                              a["slots"], a["n_slots"], a["stride"], a["new_lens"], a["left"])

    for bad in [dict(n_free=p[5]), dict(n_free=p[5] + 31 * 4), dict(n_free=p[4] + 63 * 4), dict(n_free=p[6] + 12),
                dict(slots=p[3] - 31 * 4), dict(table=p[3] - 63 * 4), dict(new_lens=p[3] - 12),
                dict(free=p[5] + 31 * 4), dict(slots=p[2]), dict(table=p[2] - 63 * 4), dict(new_lens=p[2] - 4), dict(left=p[2])]:
        assert plan(**bad) == E, bad

    def release(**kw):
        a = {**ok, **kw}
        return LA.la_kv4_release(_desc(), a["done"], a["batch"], a["lens"], a["table"], a["free"], a["n_free"])

    for bad in [dict(lens=p[2]), dict(lens=p[2] + 99 * 4), dict(done=p[2] - 12), dict(table=p[2] + 99 * 4),
                dict(table=p[2] - 63 * 4), dict(n_free=p[2]), dict(n_free=p[2] + 99 * 4), dict(lens=p[4] + 63 * 4),
                dict(lens=p[1] + 4), dict(lens=p[1] - 12), dict(n_free=p[0] + 12), dict(n_free=p[1]), dict(n_free=p[4] + 4)]:
        assert release(**bad) == E, bad


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_index_arrays_are_refused(off):
    """Every int32 array of every call, and the status, at an address that is no int's."""
    import lossless_lookahead_decoding_gb300 as LA
    E = LA.LA_ERR_ARG
    p = [FAKE + 0x10000 * i for i in range(8)]
    for i in range(8):
        a = [x + off * (i == j) for j, x in enumerate(p)]
        assert LA.la_kv4_plan(_desc(), a[0], a[1], 4, a[2], a[3], a[4], a[5], 32, 8, a[6], a[7]) == E, i
    for i in range(5):
        a = [x + off * (i == j) for j, x in enumerate(p)]
        assert LA.la_kv4_release(_desc(), a[0], 4, a[1], a[2], a[3], a[4]) == E, i
    d = _desc(status=FAKE + off)
    assert LA.la_kv4_plan(d, *p[:2], 4, *p[2:6], 32, 8, *p[6:]) == E and LA.la_kv4_release(d, p[0], 4, *p[1:5]) == E
    for rows, slots in ((FAKE + off, FAKE), (None, FAKE + off)):
        assert LA.la_kv4_append(_desc(), FAKE, FAKE, LA.LA_BF16, 1024, 5, rows, slots, 5) == E
    assert LA.la_kv4_read(_desc(), FAKE + off, 5, FAKE, FAKE, LA.LA_BF16, 1024) == E
    ws = dict(workspace=FAKE, ws_bytes=1 << 40)
    assert LA.la_kv4_attention(_desc(), _attn(lens=FAKE + off, **ws)) == E
    assert LA.la_kv4_attention(_desc(), _attn(table=FAKE + off, **ws)) == E
