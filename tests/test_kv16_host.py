"""The paged bf16 KV cache's entry points on the host: sizing, rotations, the
calls they refuse before anything reaches a GPU, and the test reference's pins."""
import ctypes as C

import numpy as np
import pytest

import kv16_ref as R
from helpers import build_lib

FAKE = 1 << 20  # never dereferenced: every call here is refused


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib()


def _desc(**kw):
    import lossless_lookahead_decoding_gb300 as LA
    f = dict(n_kv_heads=8, head_dim=128, page=64, n_pages=100, max_pages=16, k_pages=FAKE, v_pages=FAKE << 8, status=None)
    f.update(kw)
    return LA.la_kv16_desc(**f)


def _rope(**kw):
    import lossless_lookahead_decoding_gb300 as LA
    r = LA.la_rope()
    assert LA.la_rope_init(r, kw.pop("rot", 128)) == LA.LA_OK
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _rows(rope=None, **kw):
    import lossless_lookahead_decoding_gb300 as LA
    f = dict(k=FAKE << 12, v=FAKE << 13, q=FAKE << 14, dtype=LA.LA_BF16, n_rows=5, n_heads=64, k_ld=1024, v_ld=1024, q_ld=8192, n=5, rows=None,
             slots=FAKE << 15, positions=FAKE << 16, k_out=FAKE << 17, q_out=FAKE << 18, k_out_ld=1024, q_out_ld=8192)
    f.update(kw)
    return LA.la_kv16_rows(rope=C.pointer(rope) if rope is not None else None, **f)


def _attn(**kw):
    import lossless_lookahead_decoding_gb300 as LA
    f = dict(q=FAKE, k_step=FAKE, v_step=FAKE, out=FAKE, lens=FAKE, table=FAKE, batch=2, n_heads=64, W=0, N=2, G=0,
             q_ld=64 * 128, k_ld=8 * 128, v_ld=8 * 128, max_len=0, n_prefix=1, prefix_pages=20, max_prefix_len=0, prefix_lens=FAKE,
             prefix_table=FAKE, prefix_first=FAKE, workspace=FAKE, ws_bytes=1 << 40)
    f.update(kw)
    return LA.la_kv16_attn(**f)


BAD_DESC = [dict(head_dim=96), dict(head_dim=0), dict(n_kv_heads=0), dict(n_kv_heads=1025), dict(page=8), dict(page=48),
            dict(page=256), dict(n_pages=0), dict(n_pages=1 << 25), dict(max_pages=0), dict(max_pages=1 << 25)]
BAD_POOL = BAD_DESC + [dict(k_pages=None), dict(v_pages=None), dict(k_pages=FAKE + 8), dict(v_pages=FAKE + 2), dict(status=FAKE + 2)]


def test_page_bytes():
    import lossless_lookahead_decoding_gb300 as LA
    assert LA.la_kv16_page_bytes(_desc()) == 8 * 64 * 128 * 2
    assert LA.la_kv16_page_bytes(_desc(head_dim=64, page=16, n_kv_heads=3)) == 3 * 16 * 64 * 2
    assert LA.lib().la_kv16_page_bytes(None) == 0
    for bad in BAD_DESC:
        assert LA.la_kv16_page_bytes(_desc(**bad)) == 0, bad


def test_rope_turns_of_a_circle():
    """turn[i] / 2^64 of a circle is the frequency to a double's precision, negative ones wrapped."""
    import lossless_lookahead_decoding_gb300 as LA
    r = LA.la_rope()
    assert LA.la_rope_init(r, 64, 1, 5e5) == LA.LA_OK and (r.rot_dim, r.neighbours) == (64, 1)
    two_pi = 8 * np.arctan(np.longdouble(1))
    for i in range(32):
        f = np.longdouble(5e5) ** (-np.longdouble(2 * i) / 64)
        assert abs(np.longdouble(r.turn[i]) / np.longdouble(2) ** 64 - f / two_pi) <= 2.0 ** -50 * (f / two_pi) + 2.0 ** -63
    freq = np.array([2 * np.pi, -1.0, 0.0, 1e6, -1e-9, 7.0, 0.5, -0.25])
    assert LA.la_rope_init(r, 16, 0, -1.0, freq) == LA.LA_OK        # theta does not count then
    for i, f in enumerate(freq):
        want = float(np.mod(np.longdouble(f) / two_pi, np.longdouble(1)))
        off = abs(r.turn[i] / 2.0 ** 64 - want)
        assert min(off, 1 - off) <= 2.0 ** -51 * max(1.0, abs(f)), (i, off)


def test_rope_refusals():
    import lossless_lookahead_decoding_gb300 as LA
    r = LA.la_rope(rot_dim=5)
    for bad in ((0,), (8,), (24,), (144,), (-16,), (64, 2), (64, -1), (64, 0, 0.0), (64, 0, -2.0), (64, 0, float("nan")),
                (64, 0, float("inf")), (16, 0, 1e4, [1.0] * 7), (16, 0, 1e4, [1.0] * 7 + [float("nan")]),
                (16, 0, 1e4, [1.0] * 7 + [1e7]), (128, 0, 1e-7)):
        assert LA.la_rope_init(r, *bad) == LA.LA_ERR_ARG, bad
    assert r.rot_dim == 5                                            # a refused call writes nothing
    assert LA.lib().la_rope_init(None, 64, 0, 1e4, None) == LA.LA_ERR_ARG
    with pytest.raises(ValueError):
        LA.Rope(40)


def test_append_refusals():
    import lossless_lookahead_decoding_gb300 as LA
    E, rope = LA.LA_ERR_ARG, _rope()
    ok = _rows(rope)
    for bad in BAD_POOL:
        assert LA.la_kv16_append(_desc(**bad), ok) == E, bad
    assert LA.lib().la_kv16_append(None, C.byref(ok), None) == E
    assert LA.lib().la_kv16_append(C.byref(_desc()), None, None) == E
    A, i32 = FAKE << 12, FAKE << 15
    for bad in (dict(n=-1), dict(n_rows=-1), dict(dtype=2), dict(n=6), dict(k=None), dict(v=None), dict(q=None), dict(n_heads=0),
                dict(n_heads=16385), dict(k_ld=1016), dict(v_ld=1016), dict(q_ld=8184), dict(k_ld=1028), dict(v_ld=1028), dict(q_ld=8196), dict(k_out_ld=1020),
                dict(k_out_ld=1028), dict(q_out_ld=8188), dict(q_out_ld=4096), dict(positions=None), dict(k=A + 8), dict(v=A + 4),
                dict(q=A + 2), dict(k_out=A + 8), dict(q_out=A + 8), dict(slots=i32 + 2), dict(positions=i32 + 1), dict(rows=i32 + 3),
                dict(dtype=LA.LA_FP32, k_ld=1026)):
        assert LA.la_kv16_append(_desc(), _rows(rope, **bad)) == E, bad
    for bad in (dict(rot_dim=0), dict(rot_dim=40), dict(rot_dim=256), dict(neighbours=2)):
        assert LA.la_kv16_append(_desc(), _rows(_rope(**bad))) == E, bad
    assert LA.la_kv16_append(_desc(head_dim=64), _rows(_rope(rot=128))) == E   # wider than the head


def test_append_overlaps():
    """What is written over anything but its own input, in place, is refused."""
    import lossless_lookahead_decoding_gb300 as LA
    E, rope = LA.LA_ERR_ARG, _rope()
    k, v, q, slots, pos = FAKE << 12, FAKE << 13, FAKE << 14, FAKE << 15, FAKE << 16
    for bad in (dict(q_out=k), dict(q_out=v), dict(k_out=v), dict(k_out=q), dict(k_out=FAKE << 18), dict(q_out=slots), dict(k_out=pos),
                dict(q_out=FAKE), dict(k_out=FAKE << 8), dict(k=FAKE), dict(v=FAKE << 8), dict(q_out=q + 16), dict(k_out=k + 1024),
                dict(q_out=q, q_out_ld=8200), dict(k_out=k, rows=FAKE << 19), dict(q_out=q, dtype=LA.LA_FP32),
                dict(slots=FAKE), dict(positions=FAKE << 8)):
        assert LA.la_kv16_append(_desc(), _rows(rope, **bad)) == E, bad
    assert LA.la_kv16_append(_desc(v_pages=FAKE), _rows(rope)) == E
    assert LA.la_kv16_append(_desc(status=FAKE << 18), _rows(rope)) == E
    # one matrix of rows: columns apart are apart, columns over each other are not
    ld = 64 * 128 + 2 * 1024
    one = dict(q=q, k=q + 64 * 128 * 2, v=q + (64 * 128 + 1024) * 2, q_ld=ld, k_ld=ld, v_ld=ld, k_out_ld=ld, q_out_ld=ld)
    assert LA.la_kv16_append(_desc(), _rows(rope, **one, q_out=q, k_out=q + 64 * 128 * 2 - 256)) == E


def test_nothing_to_do_is_no_error():
    import lossless_lookahead_decoding_gb300 as LA
    assert LA.la_kv16_append(_desc(), _rows(_rope(), n=0)) == LA.LA_OK
    assert LA.la_kv16_append(_desc(), _rows(None, slots=None, k_out=None, q_out=None)) == LA.LA_OK
    assert LA.la_kv16_attention(_desc(), _attn(batch=0)) == LA.LA_OK


BAD_SHAPES = [dict(batch=-1), dict(batch=8193), dict(n_heads=0), dict(n_heads=12), dict(n_heads=8 * 129), dict(W=-1), dict(G=-1), dict(N=1),
              dict(N=129), dict(W=128), dict(G=128), dict(W=10, N=9, G=6), dict(max_len=-1), dict(n_prefix=-1), dict(n_prefix=8193),
              dict(prefix_pages=0), dict(prefix_pages=1 << 25), dict(max_prefix_len=-1)]


def test_attention_refusals():
    import lossless_lookahead_decoding_gb300 as LA
    E = LA.LA_ERR_ARG
    for bad in BAD_POOL:
        assert LA.la_kv16_attention(_desc(**bad), _attn()) == E, bad
    for bad in BAD_SHAPES:
        assert LA.la_kv16_attention(_desc(), _attn(**bad)) == E, bad
        assert LA.la_kv16_attention_bytes(_desc(), _attn(**bad)) == 0, bad
    for bad in (dict(q=None), dict(k_step=None), dict(v_step=None), dict(out=None), dict(lens=None), dict(table=None), dict(prefix_lens=None),
                dict(prefix_table=None), dict(prefix_first=None), dict(q=FAKE + 8), dict(k_step=FAKE + 2), dict(v_step=FAKE + 4),
                dict(out=FAKE + 8), dict(lens=FAKE + 1), dict(table=FAKE + 2), dict(prefix_lens=FAKE + 2), dict(prefix_table=FAKE + 3),
                dict(prefix_first=FAKE + 1), dict(q_ld=8184), dict(q_ld=8196), dict(k_ld=1016), dict(k_ld=1028), dict(v_ld=1016), dict(v_ld=1028)):
        assert LA.la_kv16_attention(_desc(), _attn(**bad)) == E, bad
    assert LA.lib().la_kv16_attention(None, C.byref(_attn()), None) == E
    assert LA.lib().la_kv16_attention(C.byref(_desc()), None, None) == E


def test_attention_bytes_grow_with_the_rows():
    import lossless_lookahead_decoding_gb300 as LA
    need = LA.la_kv16_attention_bytes(_desc(), _attn(workspace=None, ws_bytes=0))
    more = LA.la_kv16_attention_bytes(_desc(), _attn(batch=200))
    assert more >= need
    if need:
        for bad in (dict(workspace=None), dict(workspace=FAKE + 8), dict(ws_bytes=need - 1)):
            assert LA.la_kv16_attention(_desc(), _attn(**bad)) == LA.LA_ERR_ARG, bad


def test_attention_needs_a_workspace_where_items_are_split():
    """None for few short sequences, which a team each holds; some for longer ones, more for more rows to join; and what
    is less, missing or misaligned is refused."""
    import lossless_lookahead_decoding_gb300 as LA
    E, bytes_of = LA.LA_ERR_ARG, lambda **kw: LA.la_kv16_attention_bytes(_desc(), _attn(**kw))
    assert bytes_of(n_prefix=0, max_len=64) == 0 and bytes_of(n_prefix=0, max_len=64, W=7, N=5, G=7) == 0
    # results of 200 sequences' rows, of the prefix's and of their own keys, are to be joined
    assert bytes_of(batch=200) >= bytes_of() + 2 * 200 * 64 * 128 * 4
    for rows in (dict(), dict(W=0, N=17, G=1), dict(W=7, N=5, G=7)):
        need = bytes_of(**rows)
        assert need > 0
        for bad in (dict(workspace=None), dict(workspace=FAKE + 8), dict(ws_bytes=need - 1), dict(ws_bytes=0)):
            assert LA.la_kv16_attention(_desc(), _attn(**rows, **bad)) == E, (rows, bad)


def test_python_refusals_need_no_gpu():
    import torch
    import lossless_lookahead_decoding_gb300 as LA
    z = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    for k, v in ((z, z), (z.float(), z), (z[0], z)):
        with pytest.raises(ValueError):
            LA.KV16Cache(k, v, 1)


def test_reference_mask_and_turn():
    """The mask's rows as the branches say, a quarter turn, and a turn's inverse."""
    see = R.sees(2, 3, 1)                                  # rows: 0 | 1 2 | 3 4 | 5 6
    assert [np.nonzero(r)[0].tolist() for r in see] == [[0], [0, 1], [0, 1, 2], [0, 1, 3], [0, 1, 2, 4], [0, 5], [0, 5, 6]]
    assert (R.sees(0, 6, 1) == np.tril(np.ones((6, 6), bool))).all() and R.sees(0, 2, 0).shape == (1, 1)
    x = np.zeros((1, 1, 64))
    x[0, 0, 0] = 1
    y = R.turn(x, [1], 64, freq=np.full(32, np.pi / 2))
    assert abs(y[0, 0, 32] - 1) < 1e-15 and abs(y[0, 0, 0]) < 1e-15
    y = R.turn(x, [1], 64, neighbours=True, freq=np.full(32, np.pi / 2))
    assert abs(y[0, 0, 1] - 1) < 1e-15
    x = np.random.default_rng(0).standard_normal((4, 2, 64))
    assert np.allclose(R.turn(R.turn(x, [1, 5, 10 ** 6, 7], 32), [-1, -5, -10 ** 6, -7], 32), x, atol=1e-12)
