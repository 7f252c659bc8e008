"""The workspace of the calls over several sequences, for shapes that need one on a GPU of any
size, as the host sees it without one (no GPU needed)."""
import random

from tests.test_abi import _desc, K  # noqa: F401
from tests.test_attn_seqs_refusals import q_rows
from tests.test_cache_ops_refusals import DUMMY, p


def need(K, c, n, seqs, max_rows, max_len, window=0, sinks=0):
    return K.lib().kvq_attn_workspace_size(p(c), n, seqs, 24, max_rows, max_len, window, sinks)


def test_ragged_sequences_need_one(K):
    c = _desc(K)
    # two sequences of a million tokens: many pieces each, whatever the number of SMs
    size = need(K, c, 2, 2, 1, 1 << 20)
    # partials of a row and head for every piece, and their references and sums
    ranges = size // (2 * 24 * 258 * 4)
    assert 2 <= ranges <= 32 and size >= ranges * 2 * 24 * 258 * 4
    assert need(K, c, 2, 2, 1, 16) == 0
    for bad in ((-1, 2, 1, 1 << 20), (2, -1, 1, 1 << 20), (2, 2, -1, 1 << 20), (2, 2, 1, -1), (2, 65536, 1, 1 << 20),
                (2, 2, 1, 1 << 29)):
        assert need(K, c, *bad) == 0
    assert need(K, None, 2, 2, 1, 1 << 20) == 0 and need(K, _desc(K, D=512), 2, 2, 1, 1 << 20) == 0


def test_bad_workspaces_are_refused(K):
    L, c = K.lib(), _desc(K)
    size = need(K, c, 2, 2, 1, 1 << 20)
    q, out = q_rows(K), q_rows(K, ptr=8192)

    def local(ws, n):
        return L.kvq_decode_local(p(c), p(q), 2, DUMMY, DUMMY, 1 << 16, 1 << 20, 0, 0, 0.1, ws, n, p(out), None, None)

    def chunk(ws, n):
        return L.kvq_attn_seqs(p(c), p(q), 2, 2, DUMMY, DUMMY, DUMMY, 1 << 16, 1, 1 << 20, 0, 0, 0.1, ws, n, p(out), None, None)

    for call in (local, chunk):
        for n in (0, 1, size - 1):
            assert call(DUMMY, n) == K.ERR_WORKSPACE_TOO_SMALL
        assert call(None, size) == K.ERR_INVALID_ARG
        for off in (1, 4, 16):
            assert call(DUMMY + off, size) == K.ERR_INVALID_ARG


def test_bound_covers_smaller_calls(K):
    """Whatever part of a batch a call has; sizes themselves do not grow with it."""
    rng = random.Random(3)
    L = K.lib()

    def log(hi):
        return min(hi, int(hi ** rng.random()))

    for _ in range(300):
        c = _desc(K, fmt=rng.choice([0, 1, 3, 4]), D=rng.choice([64, 128, 256]))
        seqs, rows, length = 1 + log(300), 1 + log(500), log(1 << 20)
        n = rng.randint(1, seqs * rows)
        window, sinks = rng.choice([(0, 0), (log(8192), rng.choice([0, 4, 100]))])
        bound = L.kvq_attn_workspace_bound(p(c), n, seqs, 24, rows, length, window, sinks)
        for _ in range(30):
            b, r = 1 + log(seqs - 1) if seqs > 1 else 1, 1 + log(rows - 1) if rows > 1 else 1
            m = min(n, rng.choice([b * r, rng.randint(1, b * r)]))
            assert L.kvq_attn_workspace_size(p(c), m, b, 24, r, log(length), window, sinks) <= bound
            assert L.kvq_attn_workspace_size(p(c), m, b, 24, r, length, window, sinks) <= bound
            assert L.kvq_attn_workspace_size(p(c), m, b, 24, r, min(length, window), window, sinks) <= bound
    assert L.kvq_attn_workspace_bound(None, 1, 1, 24, 1, 1024, 0, 0) == 0
    assert L.kvq_attn_workspace_bound(p(_desc(K, D=512)), 1, 1, 24, 1, 1024, 0, 0) == 0
    assert L.kvq_attn_workspace_bound(p(_desc(K)), 0, 0, 24, 1, 1024, 0, 0) == 0
