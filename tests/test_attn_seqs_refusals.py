"""Rows of several sequences over the paged cache (kvq_decode_local, kvq_attn_seqs): bad
host-side arguments are rejected with their documented codes before anything is enqueued
(no GPU needed)."""
import math

from tests.test_abi import _desc, K  # noqa: F401
from tests.test_cache_ops_refusals import DUMMY, _refuse_rows, p, rows

BIG = 1 << 40


def q_rows(K, **kw):
    return rows(K, **{"heads": 24, "ts": 24 * 256, "hs": 256, **kw})


def shared(K, call, two):
    """What both calls refuse; two: of their rows."""
    assert call(c=None) == K.ERR_INVALID_ARG
    assert call(c=_desc(K, fmt=2, Hk=1, D=512, rope=64)) == K.ERR_UNSUPPORTED
    assert call(c=_desc(K, fmt=7)) == K.ERR_INVALID_ARG
    for D in (32, 96, 512):
        assert call(c=_desc(K, fmt=1, D=D), q=q_rows(K), out=q_rows(K, ptr=8192)) == K.ERR_UNSUPPORTED
    assert call(c=_desc(K, ps=24)) == K.ERR_UNSUPPORTED
    assert call(q=None) == K.ERR_INVALID_ARG
    assert call(out=None) == K.ERR_INVALID_ARG
    _refuse_rows(K, lambda r: call(q=r if r is None else q_rows(K, ptr=r.data, dtype=r.dtype, **(
        {"ts": r.tok_stride} if r.tok_stride != 1024 else {"hs": r.head_stride} if r.head_stride != 256 else {}))))
    assert call(q=q_rows(K, heads=23)) == K.ERR_INVALID_ARG           # heads are no multiple of the KV heads
    assert call(q=q_rows(K, heads=0)) == K.ERR_INVALID_ARG
    assert call(out=q_rows(K, heads=20, ptr=8192)) == K.ERR_INVALID_ARG
    assert call(out=q_rows(K)) == K.ERR_INVALID_ARG                   # over the queries
    assert call(out=q_rows(K, ptr=8192, hs=0)) == K.ERR_INVALID_ARG   # on top of each other
    assert call(out=q_rows(K, ptr=8192, ts=256)) == K.ERR_INVALID_ARG
    wide = dict(heads=4 * 65, ts=4 * 65 * 256)
    assert call(q=rows(K, **wide), out=rows(K, ptr=8192, **wide)) == K.ERR_UNSUPPORTED  # 65 heads a KV head
    for name in ("lens", "tables"):
        assert call(**{name: None}) == K.ERR_INVALID_ARG
        assert call(**{name: DUMMY + 2}) == K.ERR_INVALID_ARG
    assert call(status=DUMMY + 1) == K.ERR_INVALID_ARG
    assert call(pages=0) == K.ERR_INVALID_ARG
    assert call(max_len=-1) == K.ERR_INVALID_ARG
    assert call(max_len=64 * 16 + 1) == K.ERR_INVALID_ARG             # more than the tables hold
    assert call(max_len=1 << 29, pages=1 << 26) == K.ERR_UNSUPPORTED
    assert call(window=-1) == K.ERR_INVALID_ARG
    assert call(sinks=-1) == K.ERR_INVALID_ARG
    for bad in (math.nan, math.inf, -math.inf):
        assert call(scale=bad) == K.ERR_INVALID_ARG
    assert call(c=_desc(K, pages=1 << 27)) == K.ERR_UNSUPPORTED   # rows of the pool past 2^31
    assert call(seqs=-1) == K.ERR_INVALID_ARG
    assert call(seqs=0) == K.OK
    assert call(seqs=65536, **two(65536)) == K.ERR_UNSUPPORTED


def test_decode_local_refusals(K):
    L = K.lib()

    def call(c=_desc(K), q=q_rows(K), seqs=4, lens=DUMMY, tables=DUMMY, pages=64, max_len=1024, window=100, sinks=4,
             scale=0.1, ws=DUMMY, ws_bytes=BIG, out=q_rows(K, ptr=8192), status=None):
        return L.kvq_decode_local(p(c), p(q), seqs, lens, tables, pages, max_len, window, sinks, scale, ws, ws_bytes,
                                  p(out), status, None)

    shared(K, call, lambda n: {})


def test_attn_seqs_refusals(K):
    L = K.lib()

    def call(c=_desc(K), q=q_rows(K), n=40, seqs=4, cu=DUMMY, lens=DUMMY, tables=DUMMY, pages=64, max_rows=20, max_len=1024,
             window=0, sinks=0, scale=0.1, ws=DUMMY, ws_bytes=BIG, out=q_rows(K, ptr=8192), status=None):
        return L.kvq_attn_seqs(p(c), p(q), n, seqs, cu, lens, tables, pages, max_rows, max_len, window, sinks, scale, ws,
                               ws_bytes, p(out), status, None)

    shared(K, call, lambda n: {})
    assert call(n=-1) == K.ERR_INVALID_ARG
    assert call(n=0) == K.OK
    assert call(n=1 << 29) == K.ERR_UNSUPPORTED
    assert call(max_rows=-1) == K.ERR_INVALID_ARG
    assert call(max_rows=0) == K.OK
    assert call(cu=None) == K.ERR_INVALID_ARG
    assert call(cu=DUMMY + 2) == K.ERR_INVALID_ARG


def test_workspace(K):
    L = K.lib()
    c = _desc(K)
    one = L.kvq_attn_workspace_size(p(c), 1, 1, 24, 1, 1024, 0, 0)
    long = L.kvq_attn_workspace_size(p(c), 1, 1, 24, 1, 1 << 20, 0, 0)
    assert long >= one
    assert L.kvq_attn_workspace_size(p(c), 1, 1, 24, 1, 1 << 20, 256, 4) == L.kvq_attn_workspace_size(p(c), 1, 1, 24, 1, 4096, 256, 4)
    for bad in ((-1, 1, 24, 1, 1024), (1, -1, 24, 1, 1024), (1, 1, 23, 1, 1024), (1, 1, 24, -1, 1024), (1, 1, 24, 1, -1)):
        assert L.kvq_attn_workspace_size(p(c), *bad, 0, 0) == 0
    assert L.kvq_attn_workspace_size(None, 1, 1, 24, 1, 1024, 0, 0) == 0
    # a workspace that is too small, missing or off its 32 bytes (a long sequence needs one)
    if long:
        q, out = q_rows(K), q_rows(K, ptr=8192)

        def call(ws, size):
            return L.kvq_decode_local(p(c), p(q), 1, DUMMY, DUMMY, 1 << 16, 1 << 20, 0, 0, 0.1, ws, size, p(out), None, None)

        assert call(DUMMY, long - 1) == K.ERR_WORKSPACE_TOO_SMALL
        assert call(None, long) == K.ERR_INVALID_ARG
        assert call(DUMMY + 16, long) == K.ERR_INVALID_ARG
