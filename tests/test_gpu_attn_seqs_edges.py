"""decode_local and attn_seqs where calls and values meet in ways that
tests/test_gpu_attn_seqs.py leaves out; its plain 64-bit arithmetic and tolerances."""
import pytest
import torch

from tests.test_gpu_attn_seqs import DEV, FMTS, Batch
from tests.test_gpu_parity import K  # noqa: F401

pytestmark = pytest.mark.gpu

SCALED = [f for f in FMTS if f != "bf16"]


def unseen(b, window, sinks):
    """Slots of the pool that no row of the batch sees [pages, page size]."""
    hidden = torch.ones(b.cache.num_pages, b.ps, dtype=torch.bool, device=DEV)
    for i, (T, n) in enumerate(zip(b.lens, b.rows)):
        key = torch.arange(T, device=DEV)
        if window:
            key = key[(key < sinks) | (key > T - n - window)]
        hidden[b.table[i].long()[key // b.ps], key % b.ps] = False
    return hidden


@pytest.mark.parametrize("fmt", SCALED)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 5), (300, 37)])
def test_large_scales_that_nobody_sees(K, fmt, D, rows, window, sinks):
    """What lies behind a sequence's end, or between sinks and window, does not change how
    the values beside it are rounded."""
    b = Batch(K, fmt, 2, D, 64, [777, 300], [rows, rows], 3, seed=43)
    want = b.attn(window, sinks)
    hidden = unseen(b, window, sinks)
    for s in (b.cache.k_scale, b.cache.v_scale):
        s.transpose(1, 2)[hidden] = 60000.0
    assert torch.equal(b.attn(window, sinks), want)
