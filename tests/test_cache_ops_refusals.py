"""The calls around the cache (norms and rotary positions, rows read back,
differential heads) reject bad host-side arguments with their documented codes
before anything is enqueued, and the rope table holds what it says (no GPU needed)."""
import ctypes
import math
from fractions import Fraction

from tests.test_abi import _desc, _tq4_desc, K  # noqa: F401

DUMMY = 4096


def rows(K, heads=4, ts=1024, hs=256, dtype=0, ptr=DUMMY):
    return K.RowsDesc(ptr, dtype, heads, ts, hs)


def norm(K, eps=1e-6, offset=0.0, dtype=0, ptr=DUMMY):
    return K.NormDesc(ptr, dtype, eps, offset)


def rope(K, rot=64, inter=0, axes=1, ptr=DUMMY, reserved=0):
    return K.RopeDesc(rot, inter, axes, reserved, ptr)


def p(x):
    return None if x is None else ctypes.byref(x)


def test_rope_table_words(K):
    L = K.lib()
    freqs = [1.0, 0.25, 1e-4, 0.0, -0.5, 2 * math.pi, 100.0]
    axes = [0, 1, 2, 3, 0, 1, 2]
    n = len(freqs)
    f = (ctypes.c_double * n)(*freqs)
    a = (ctypes.c_int32 * n)(*axes)
    w = (ctypes.c_uint64 * n)()
    assert L.kvq_rope_table(f, a, n, w) == K.OK
    two_pi = Fraction("6.28318530717958647692528676655900577")
    for i in range(n):
        assert w[i] & 3 == axes[i]
        want = (Fraction(freqs[i]) / two_pi) % 1
        got = Fraction(w[i] >> 2, 1 << 62)
        # the double product's rounding (2^-53 of up to 16 turns) and the table's own 2^-63
        off = abs(got - want)
        off = min(off, 1 - off)
        assert off <= Fraction(abs(freqs[i])) / two_pi / (1 << 51) + Fraction(1, 1 << 62)
    assert L.kvq_rope_table(f, None, n, w) == K.OK and all(x & 3 == 0 for x in w)
    for bad in (math.inf, -math.inf, math.nan):
        assert L.kvq_rope_table((ctypes.c_double * 1)(bad), None, 1, w) == K.ERR_INVALID_ARG
    assert L.kvq_rope_table(f, (ctypes.c_int32 * n)(*([4] * n)), n, w) == K.ERR_INVALID_ARG
    assert L.kvq_rope_table(f, (ctypes.c_int32 * n)(*([-1] * n)), n, w) == K.ERR_INVALID_ARG
    assert L.kvq_rope_table(None, None, n, w) == K.ERR_INVALID_ARG
    assert L.kvq_rope_table(f, None, n, None) == K.ERR_INVALID_ARG
    assert L.kvq_rope_table(f, None, 0, w) == K.ERR_INVALID_ARG


def _refuse_rows(K, call):
    """call(rows) for every kind of bad strided tensor."""
    assert call(None) == K.ERR_INVALID_ARG
    assert call(rows(K, ptr=0)) == K.ERR_INVALID_ARG
    assert call(rows(K, dtype=2)) == K.ERR_INVALID_ARG
    assert call(rows(K, ts=-1024)) == K.ERR_INVALID_ARG
    assert call(rows(K, hs=-256)) == K.ERR_INVALID_ARG
    assert call(rows(K, ptr=DUMMY + 2)) == K.ERR_INVALID_ARG            # f32 at an odd half word
    assert call(rows(K, dtype=1, ptr=DUMMY + 1)) == K.ERR_INVALID_ARG
    assert call(rows(K, ts=(1 << 31) + 1)) == K.ERR_UNSUPPORTED


def test_norm_rope_refusals(K):
    L = K.lib()
    x, y = rows(K), rows(K, ptr=8192)

    def call(x=x, y=y, n=4, w=256, nm=None, rp=None, pos=DUMMY, ps=4):
        return L.kvq_norm_rope(p(x), p(y), n, w, p(nm), p(rp), pos, ps, None, None)

    _refuse_rows(K, lambda r: call(x=r))
    _refuse_rows(K, lambda r: call(y=r))
    assert call(n=-1) == K.ERR_INVALID_ARG
    assert call(n=0) == K.OK
    assert call(n=1 << 31) == K.ERR_UNSUPPORTED
    assert call(w=0) == K.ERR_INVALID_ARG
    for w in (32, 96, 250, 576, 1024):
        assert call(w=w) == K.ERR_UNSUPPORTED
    assert call(x=rows(K, heads=3)) == K.ERR_INVALID_ARG                 # heads differ
    assert call(x=rows(K, heads=0), y=rows(K, heads=0)) == K.ERR_INVALID_ARG
    assert call(x=rows(K, heads=16385), y=rows(K, heads=16385, ts=16385 * 256)) == K.ERR_UNSUPPORTED
    assert call(y=rows(K, ptr=8192, hs=0)) == K.ERR_INVALID_ARG          # outputs on top of each other
    assert call(y=rows(K, ptr=8192, ts=256)) == K.ERR_INVALID_ARG
    assert call(y=rows(K, ptr=8192, hs=255)) == K.ERR_INVALID_ARG
    assert call(y=rows(K, dtype=1)) == K.ERR_INVALID_ARG                 # in place with another type
    assert call(y=rows(K, ts=2048)) == K.ERR_INVALID_ARG                 # in place with other strides
    for bad in (norm(K, eps=0.0), norm(K, eps=-1.0), norm(K, eps=math.inf), norm(K, eps=math.nan),
                norm(K, offset=math.nan), norm(K, ptr=0), norm(K, dtype=3), norm(K, ptr=DUMMY + 2)):
        assert call(nm=bad) == K.ERR_INVALID_ARG
    for bad in (rope(K, rot=0), rope(K, rot=63), rope(K, rot=258), rope(K, axes=0), rope(K, axes=5), rope(K, inter=2),
                rope(K, ptr=0), rope(K, ptr=DUMMY + 4), rope(K, reserved=1)):
        assert call(rp=bad) == K.ERR_INVALID_ARG
    assert call(rp=rope(K, rot=40)) == K.ERR_UNSUPPORTED                 # half-split: a multiple of 16
    assert call(rp=rope(K, rot=288), w=512) == K.ERR_UNSUPPORTED
    assert call(rp=rope(K), pos=None) == K.ERR_INVALID_ARG
    assert call(rp=rope(K), pos=DUMMY + 2) == K.ERR_INVALID_ARG
    assert call(rp=rope(K, axes=3), ps=3) == K.ERR_INVALID_ARG           # the axes' positions overlap


def test_norm_rope_store_refusals(K):
    L = K.lib()
    c = _desc(K)
    q, qo, k, v = rows(K, heads=24, ts=6144), rows(K, heads=24, ts=6144, ptr=8192), rows(K), rows(K)

    def call(c=c, q=q, k=k, v=v, n=4, qn=None, kn=None, rp=None, pos=DUMMY, ps=4, slots=DUMMY, qo=qo, rot=1):
        return L.kvq_norm_rope_store(p(c), p(q), p(k), p(v), n, p(qn), p(kn), p(rp), pos, ps, slots, p(qo), rot, None,
                                     None)

    assert call(c=None) == K.ERR_INVALID_ARG
    # fp8 latent rows: 512 + 64, no v, no norm of the queries
    fp8 = _desc(K, fmt=2, Hk=1, D=512, rope=64)
    lk, lq, lo = rows(K, heads=1, ts=576, hs=576), rows(K, heads=16, ts=9216, hs=576), \
        rows(K, heads=16, ts=9216, hs=576, ptr=8192)
    latent = lambda c=fp8, k=lk, v=None, q=lq, qo=lo, **kw: call(c=c, k=k, v=v, q=q, qo=qo, **kw)
    assert latent(n=0) == K.OK
    assert latent(c=_desc(K, fmt=2, Hk=1, D=256, rope=64)) == K.ERR_UNSUPPORTED
    assert latent(c=_desc(K, fmt=2, Hk=1, D=512, rope=32)) == K.ERR_UNSUPPORTED
    assert latent(v=lk) == K.ERR_INVALID_ARG
    assert latent(qn=norm(K)) == K.ERR_INVALID_ARG
    assert latent(k=None) == K.ERR_INVALID_ARG
    assert latent(k=rows(K, heads=2, ts=1152, hs=576)) == K.ERR_INVALID_ARG
    assert latent(rp=rope(K, rot=128)) == K.ERR_INVALID_ARG                # wider than the rope part
    assert latent(rp=rope(K, rot=40)) == K.ERR_UNSUPPORTED
    assert latent(qo=rows(K, heads=16, ts=8192, hs=512, ptr=8192)) == K.ERR_INVALID_ARG
    assert call(c=_desc(K, D=32)) == K.ERR_UNSUPPORTED
    assert call(c=_desc(K, fmt=1, D=96)) == K.ERR_UNSUPPORTED
    assert call(c=_tq4_desc(K, signs=None)) == K.ERR_INVALID_ARG
    _refuse_rows(K, lambda r: call(k=r))
    _refuse_rows(K, lambda r: call(v=r))
    bad_q = lambda r: None if r is None else K.RowsDesc(r.data, r.dtype, 24, max(r.tok_stride, -1) and r.tok_stride * 6,
                                                        r.head_stride)
    assert call(q=bad_q(rows(K, ptr=0))) == K.ERR_INVALID_ARG
    assert call(q=bad_q(rows(K, dtype=2))) == K.ERR_INVALID_ARG
    assert call(q=None) == K.ERR_INVALID_ARG                              # an output without queries
    assert call(qo=None) == K.ERR_INVALID_ARG
    assert call(q=rows(K, heads=0), qo=rows(K, heads=0)) == K.ERR_INVALID_ARG
    assert call(qo=rows(K, heads=12, ts=6144, ptr=8192)) == K.ERR_INVALID_ARG
    assert call(qo=rows(K, heads=24, ts=6144, dtype=1, ptr=8192)) == K.ERR_INVALID_ARG   # rotated queries are fp32
    assert call(qo=rows(K, heads=24, ts=1024, ptr=8192)) == K.ERR_INVALID_ARG            # overlapping tokens
    assert call(q=rows(K, heads=24, ts=6144, ptr=8192, dtype=1)) == K.ERR_INVALID_ARG    # in place, other type
    assert call(rot=2) == K.ERR_INVALID_ARG
    assert call(n=-1) == K.ERR_INVALID_ARG
    assert call(n=0) == K.OK
    assert call(slots=None) == K.ERR_INVALID_ARG
    assert call(k=rows(K, heads=2)) == K.ERR_INVALID_ARG                  # not the cache's heads
    assert call(qn=norm(K, eps=0.0)) == K.ERR_INVALID_ARG
    assert call(kn=norm(K, eps=0.0)) == K.ERR_INVALID_ARG
    assert call(rp=rope(K, rot=260)) == K.ERR_INVALID_ARG


def test_load_refusals(K):
    L = K.lib()
    c = _desc(K)
    k, v = rows(K), rows(K, ptr=1 << 20)

    def call(c=c, slots=DUMMY, n=4, rb=1, k=k, v=v):
        return L.kvq_load(p(c), slots, n, rb, p(k), p(v), None, None)

    def seqs(c=c, bt=DUMMY, mp=4, B=2, cu=DUMMY, n=4, rb=1, k=k, v=v):
        return L.kvq_load_seqs(p(c), bt, mp, B, None, cu, n, rb, p(k), p(v), None, None)

    for f in (call, seqs):
        assert f(c=None) == K.ERR_INVALID_ARG
        assert f(c=_desc(K, D=48)) == K.ERR_UNSUPPORTED
        assert f(k=None, v=None) == K.ERR_INVALID_ARG
        for bad in (rows(K, ptr=0), rows(K, dtype=7), rows(K, heads=3), rows(K, hs=0), rows(K, ts=512), rows(K, ts=-1)):
            assert f(k=bad) == K.ERR_INVALID_ARG
            assert f(v=bad) == K.ERR_INVALID_ARG
        assert f(rb=2) == K.ERR_INVALID_ARG
        for fmt in (1, 3):
            assert f(c=_desc(K, fmt=fmt)) == K.ERR_INVALID_ARG             # nothing to rotate back
        assert f(n=-1) == K.ERR_INVALID_ARG
        assert f(n=0) == K.OK
        assert f(n=1 << 31) == K.ERR_UNSUPPORTED
        fp8 = _desc(K, fmt=2, Hk=1, D=512, rope=64)
        latent = rows(K, heads=1, ts=576, hs=576)
        assert f(c=fp8, rb=0, k=latent) == K.ERR_INVALID_ARG               # v must be NULL
        assert f(c=fp8, rb=0, k=rows(K, heads=1, ts=512, hs=512), v=None) == K.ERR_INVALID_ARG   # rows of 576
        assert f(c=fp8, rb=1, k=latent, v=None) == K.ERR_INVALID_ARG
    assert call(slots=None) == K.ERR_INVALID_ARG
    assert seqs(bt=None) == K.ERR_INVALID_ARG
    assert seqs(cu=None) == K.ERR_INVALID_ARG
    assert seqs(mp=0) == K.ERR_INVALID_ARG
    assert seqs(B=-1) == K.ERR_INVALID_ARG
    assert seqs(B=0) == K.OK                                               # no sequences: nothing is written


def test_differential_refusals(K):
    L = K.lib()
    c = _desc(K)
    ws = L.kvq_decode_workspace_size(p(c), 2, 24, 1000, 0)

    def merge(c=c, wsp=DUMMY, wsb=ws, B=2, Hq=24, lens=DUMMY, msl=1000, nsel=0, rb=1, lam=DUMMY, ls=12, nm=None, sc=1.0,
              out=DUMMY, od=0):
        return L.kvq_merge_diff(p(c), wsp, wsb, B, Hq, lens, msl, nsel, rb, lam, ls, p(nm), sc, out, od, None)

    assert merge(c=None) == K.ERR_INVALID_ARG
    assert merge(c=_desc(K, fmt=2, Hk=1, D=512, rope=64), Hq=16, rb=0) == K.ERR_UNSUPPORTED
    assert merge(c=_desc(K, D=128)) == K.ERR_UNSUPPORTED
    assert merge(Hq=12) == K.ERR_UNSUPPORTED          # three query heads to a KV head: a pair would straddle two
    assert merge(Hq=25) == K.ERR_INVALID_ARG
    assert merge(Hq=40) == K.ERR_UNSUPPORTED
    assert merge(B=-1) == K.ERR_INVALID_ARG
    assert merge(B=0) == K.OK
    assert merge(B=65536, wsb=1 << 50) == K.ERR_UNSUPPORTED
    assert merge(nsel=4097) == K.ERR_INVALID_ARG
    assert merge(c=_desc(K, fmt=3)) == K.ERR_INVALID_ARG                   # nothing to rotate back
    assert merge(wsp=None) == K.ERR_INVALID_ARG
    assert merge(wsp=DUMMY + 8) == K.ERR_INVALID_ARG
    assert merge(wsb=ws - 1) == K.ERR_WORKSPACE_TOO_SMALL
    assert merge(lens=None) == K.ERR_INVALID_ARG

    def heads(x=DUMMY, n=4, Hq=24, w=256, lam=DUMMY, ls=12, nm=None, sc=1.0, out=DUMMY, od=0):
        return L.kvq_diff_heads(x, n, Hq, w, lam, ls, p(nm), sc, out, od, None)

    assert heads(x=None) == K.ERR_INVALID_ARG
    assert heads(x=DUMMY + 2) == K.ERR_INVALID_ARG
    assert heads(n=-1) == K.ERR_INVALID_ARG
    assert heads(n=0) == K.OK
    assert heads(Hq=0) == K.ERR_INVALID_ARG
    assert heads(Hq=23) == K.ERR_INVALID_ARG
    assert heads(w=96) == K.ERR_UNSUPPORTED
    wp = L.kvq_prefill_diff_workspace_size(p(c), 4, 24, 40)
    assert wp >= 4 * 24 * 258 * 4

    def prefill(c=c, q=DUMMY, dt=0, n=4, Hq=24, q0=40, bt=DUMMY, mp=4, lam=DUMMY, ls=12, nm=None, sc=1.0, wsp=DUMMY,
                wsb=wp, out=DUMMY, od=0):
        return L.kvq_prefill_diff(p(c), q, dt, n, Hq, q0, bt, mp, 0.1, lam, ls, p(nm), sc, wsp, wsb, out, od, None, None)

    assert prefill(c=None) == K.ERR_INVALID_ARG
    assert prefill(c=_desc(K, fmt=1)) == K.ERR_UNSUPPORTED
    assert prefill(c=_tq4_desc(K)) == K.ERR_UNSUPPORTED
    assert prefill(c=_desc(K, D=128)) == K.ERR_UNSUPPORTED
    assert prefill(Hq=12) == K.ERR_UNSUPPORTED
    assert prefill(Hq=40) == K.ERR_UNSUPPORTED
    assert prefill(Hq=26) == K.ERR_INVALID_ARG
    assert prefill(n=-1) == K.ERR_INVALID_ARG
    assert prefill(n=0) == K.OK
    assert prefill(q0=-1) == K.ERR_INVALID_ARG
    assert prefill(q0=61) == K.ERR_INVALID_ARG                             # past the block table
    assert prefill(n=1 << 27, Hq=32, mp=1 << 30) == K.ERR_UNSUPPORTED
    assert prefill(q=None) == K.ERR_INVALID_ARG
    assert prefill(q=DUMMY + 2) == K.ERR_INVALID_ARG
    assert prefill(dt=2) == K.ERR_INVALID_ARG
    assert prefill(bt=None) == K.ERR_INVALID_ARG
    assert prefill(mp=0) == K.ERR_INVALID_ARG
    assert prefill(wsp=None) == K.ERR_INVALID_ARG
    assert prefill(wsp=DUMMY + 16) == K.ERR_INVALID_ARG
    assert prefill(wsb=wp - 1) == K.ERR_WORKSPACE_TOO_SMALL
    assert L.kvq_prefill_diff_workspace_size(p(c), 4, 12, 40) == 0
    assert L.kvq_prefill_diff_workspace_size(None, 4, 24, 40) == 0
    for f in (merge, heads, prefill):
        assert f(lam=None) == K.ERR_INVALID_ARG
        assert f(lam=DUMMY + 1) == K.ERR_INVALID_ARG
        assert f(ls=-1) == K.ERR_INVALID_ARG
        assert f(ls=11) == K.ERR_INVALID_ARG
        assert f(nm=norm(K, eps=0.0)) == K.ERR_INVALID_ARG
        assert f(sc=math.inf) == K.ERR_INVALID_ARG
        assert f(sc=math.nan) == K.ERR_INVALID_ARG
        assert f(out=None) == K.ERR_INVALID_ARG
        assert f(out=DUMMY + 2) == K.ERR_INVALID_ARG
        assert f(od=2) == K.ERR_INVALID_ARG
