"""Argument checks of the attention entry points (no GPU): the status comes before any launch."""
import ctypes

import pytest

from quantised_gguf_weight_gb300 import build as qbuild

FAKE = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def qk():
    qbuild.build()
    from quantised_gguf_weight_gb300 import qk as _qk
    _qk.load()
    return _qk


def cache(qk, pages=FAKE, n=4, heads=2, D=64, page=16):
    return qk._KVCacheQ4(pages, n, heads, D, page)


def test_new_status_string(qk):
    assert qk.load().qk_status_string(10) == b"unknown element type"


def test_norm_rope_statuses(qk):
    names = ("x", "ldx", "x_type", "nq", "nk", "D", "wq", "wk", "eps", "table", "n_pos", "rot", "inter", "pos", "T",
             "y", "ldy", "y_type", "stream")
    ok = dict(x=FAKE, ldx=0, x_type=0, nq=2, nk=1, D=64, wq=None, wk=None, eps=1e-6, table=FAKE, n_pos=8, rot=64,
              inter=0, pos=FAKE, T=3, y=FAKE + 0x10000, ldy=0, y_type=0, stream=None)

    def call(**kw):
        a = dict(ok, **kw)
        return qk.load().qk_norm_rope(*[a[n] for n in names])

    assert call(x=None) == 1 and call(y=None) == 1 and call(table=None) == 1 and call(pos=None) == 1
    for kw in (dict(nq=-1), dict(nq=0, nk=0), dict(D=0), dict(D=63), dict(D=514), dict(T=-1), dict(rot=3),
               dict(rot=66), dict(rot=-2), dict(n_pos=0), dict(ldx=100), dict(ldy=191),
               dict(y=FAKE, y_type=1), dict(y=FAKE, ldy=200)):
        assert call(**kw) == 2, kw
    assert call(x=FAKE + 2) == 3 and call(y=FAKE + 0x10001, y_type=1) == 3 and call(wq=FAKE + 1) == 3
    assert call(table=FAKE + 4) == 3 and call(pos=FAKE + 2) == 3
    assert call(x_type=3) == 10 and call(y_type=-1) == 10
    assert call(T=1 << 40) == 8 and call(nq=70000) == 8
    assert call(T=0, x=None) == 0


def test_cache_statuses(qk):
    read = qk.load().qk_kv_read_q4

    def call(c, slots=FAKE, T=2, k=FAKE, ldk=0, v=FAKE, ldv=0, t=0):
        return read(ctypes.byref(c) if c is not None else None, slots, T, k, ldk, v, ldv, t, None)

    assert call(None) == 1 and call(cache(qk, pages=None)) == 1
    for kw in (dict(n=0), dict(heads=0), dict(D=80), dict(D=0), dict(page=8), dict(page=24), dict(page=0),
               dict(page=2048), dict(page=-16)):
        assert call(cache(qk, **kw)) == 2, kw
    assert call(cache(qk, pages=FAKE + 8)) == 3
    assert call(cache(qk, n=1 << 31)) == 8
    c = cache(qk)
    assert call(c, slots=None) == 1 and call(c, k=None, v=None) == 1
    assert call(c, T=-1) == 2 and call(c, ldk=127) == 2 and call(c, ldv=1) == 2
    assert call(c, slots=FAKE + 4) == 3 and call(c, k=FAKE + 2) == 3
    assert call(c, t=7) == 10 and call(c, T=1 << 60) == 8 and call(c, T=0, slots=None) == 0


def test_append_statuses(qk):
    names = ("q", "ldq", "nq", "k", "ldk", "v", "ldv", "t", "wq", "wk", "eps", "table", "n_pos", "rot", "inter",
             "pos", "slots", "T", "qo", "ldqo", "qo_t", "stream")
    ok = dict(q=FAKE, ldq=0, nq=4, k=FAKE, ldk=0, v=FAKE, ldv=0, t=0, wq=None, wk=None, eps=0.0, table=FAKE,
              n_pos=9, rot=64, inter=0, pos=FAKE, slots=FAKE, T=2, qo=FAKE + 0x10000, ldqo=0, qo_t=0, stream=None)

    def call(c=cache(qk), **kw):
        a = dict(ok, **kw)
        return qk.load().qk_kv_append_q4(ctypes.byref(c), *[a[n] for n in names])

    assert call(k=None) == 1 and call(v=None) == 1 and call(slots=None) == 1 and call(qo=None) == 1
    for kw in (dict(nq=0), dict(T=-1), dict(ldq=255), dict(ldk=127), dict(ldv=127), dict(ldqo=3), dict(rot=96),
               dict(qo=FAKE, qo_t=2)):
        assert call(**kw) == 2, kw
    assert call(slots=FAKE + 4) == 3 and call(k=FAKE + 1, t=1) == 3 and call(q=FAKE + 2) == 3
    assert call(t=5) == 10 and call(qo_t=5) == 10
    assert call(T=1 << 40) == 8 and call(cache(qk, D=72)) == 2 and call(T=0, k=None) == 0


def test_attn_statuses(qk):
    names = ("q", "ldq", "t", "nq", "pt", "ldp", "maxp", "lens", "qs", "B", "T", "maxq", "maxlen", "scale", "window",
             "out", "ldo", "ot", "ws", "wsb", "stream")
    ok = dict(q=FAKE, ldq=0, t=0, nq=4, pt=FAKE, ldp=8, maxp=0, lens=FAKE, qs=None, B=2, T=2, maxq=1, maxlen=0,
              scale=0.1, window=0, out=FAKE, ldo=0, ot=0, ws=None, wsb=0, stream=None)

    def call(c=cache(qk), **kw):
        a = dict(ok, **kw)
        return qk.load().qk_attn_q4(ctypes.byref(c), *[a[n] for n in names])

    for n in ("q", "pt", "lens", "out"):
        assert call(**{n: None}) == 1, n
    for kw in (dict(nq=3), dict(nq=0), dict(B=-1), dict(T=-1), dict(maxq=-1), dict(maxlen=-1), dict(window=-1),
               dict(ldp=-1), dict(maxp=9), dict(ldq=255), dict(ldo=1), dict(T=3), dict(scale=float("nan"))):
        assert call(**kw) == 2, kw
    assert call(q=FAKE + 2) == 3 and call(out=FAKE + 1, ot=1) == 3 and call(pt=FAKE + 2) == 3
    assert call(lens=FAKE + 1) == 3 and call(qs=FAKE + 2) == 3
    assert call(ws=FAKE + 16, wsb=1 << 20) == 7
    assert call(t=3) == 10 and call(ot=3) == 10
    assert call(nq=131072 * 2, ldq=0) == 8 and call(B=1 << 31, T=1 << 31) == 8
    assert call(T=0, B=0, q=None) == 0


def test_rope_table_statuses(qk):
    f = qk.load().qk_rope_table

    def call(t=FAKE, n=8, rot=64, base=1e4, s=1.0, ff=None, ctx=0, bf=32.0, bs=1.0, amp=1.0):
        return f(t, n, rot, base, s, ff, ctx, bf, bs, amp, None)

    assert call(t=None) == 1
    for kw in (dict(n=0), dict(rot=0), dict(rot=5), dict(base=1.0), dict(s=0.0), dict(ctx=-1), dict(ctx=4, bf=0.0),
               dict(ctx=4, bs=-1.0), dict(base=float("nan"))):
        assert call(**kw) == 2, kw
    assert call(t=FAKE + 4) == 3 and call(ff=FAKE + 2) == 3 and call(rot=8192) == 8


def test_workspace_bytes_of_nothing(qk):
    f = qk.load().qk_attn_q4_workspace_bytes
    assert f(0, 8, 2, 64, 1, 100) == 0 and f(1, 8, 0, 64, 1, 100) == 0 and f(1, 7, 2, 64, 1, 100) == 0
