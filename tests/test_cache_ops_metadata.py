"""Slots, tables, lengths and status words off their four bytes are refused before
anything is enqueued (no GPU needed)."""
import ctypes

import pytest

from tests.test_abi import K, _desc  # noqa: F401
from tests.test_cache_ops_refusals import DUMMY, p, rows

OFF = DUMMY + 2


@pytest.mark.parametrize("where", ["status", "slots", "tables", "lengths", "starts", "scales"])
def test_metadata_off_its_words(K, where):
    L, c, bad = K.lib(), _desc(K), K.ERR_INVALID_ARG
    x, y, kv = rows(K), rows(K, ptr=8192), rows(K, ptr=1 << 20)
    at = {where: OFF}.get
    status, slots, tables, lengths, starts = (at(n, DUMMY) for n in ("status", "slots", "tables", "lengths", "starts"))
    if where == "status":
        assert L.kvq_norm_rope(p(x), p(y), 4, 256, None, None, None, 0, status, None) == bad
    if where in ("status", "slots"):
        assert L.kvq_norm_rope_store(p(c), None, p(x), p(kv), 4, None, None, None, None, 0, slots, None, 0, status,
                                     None) == bad
        assert L.kvq_load(p(c), slots, 4, 1, p(x), p(kv), status, None) == bad
    if where in ("status", "tables", "lengths", "starts"):
        assert L.kvq_load_seqs(p(c), tables, 4, 2, starts, lengths, 4, 1, p(x), p(kv), status, None) == bad
    if where == "lengths":
        ws = L.kvq_decode_workspace_size(p(c), 2, 24, 1000, 0)
        assert L.kvq_merge_diff(p(c), DUMMY, ws, 2, 24, lengths, 1000, 0, 1, DUMMY, 12, None, 1.0, DUMMY, 0, None) == bad
    if where in ("status", "tables"):
        ws = L.kvq_prefill_diff_workspace_size(p(c), 4, 24, 40)
        assert L.kvq_prefill_diff(p(c), DUMMY, 0, 4, 24, 40, tables, 4, 0.1, DUMMY, 12, None, 1.0, DUMMY, ws, DUMMY, 0,
                                  status, None) == bad
    if where == "scales":   # of fp8 rows: fp32
        for k_scale, v_scale in ((OFF, DUMMY), (DUMMY, OFF)):
            fp8 = K.CacheDesc(2, 1, 512, 64, 16, 4, DUMMY, k_scale, DUMMY, v_scale)
            latent = rows(K, heads=1, ts=576, hs=576)
            assert L.kvq_load(p(fp8), DUMMY, 4, 0, p(latent), None, None, None) == bad
            assert L.kvq_store(ctypes.byref(fp8), DUMMY, None, 0, 1, DUMMY, None, None) == bad
