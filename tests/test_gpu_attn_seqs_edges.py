"""decode_local and attn_seqs where calls and values meet in ways that
tests/test_gpu_attn_seqs.py leaves out; its plain 64-bit arithmetic and tolerances."""
import math

import pytest
import torch

from tests.test_gpu_attn_seqs import DEV, FMTS, Batch, ints, rnd
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


# ------------------------------------------------------------------ metadata made on the device

def write(dst, src):
    """By a kernel (a copy between tensors of one type may be the copy engine's)."""
    torch.add(src, 0, out=dst)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [[1, 1, 1], [3, 1, 5], [150, 1, 40]])
@pytest.mark.parametrize("last", ["seq_lens", "cu_rows", "block_tables"])
def test_metadata_written_right_before(K, fmt, rows, last):
    """Lengths, row numbers and tables that a kernel writes directly in front of a call, in a
    stream and in a graph, count as if the device had been waited for."""
    b = Batch(K, fmt, 2, 128, 16, [5000, 333, 700], rows, 3, seed=41)
    right = {"seq_lens": ints(b.lens), "cu_rows": ints(b.cu), "block_tables": b.table}
    # what a call that did not wait would see: other lengths, no rows, no pages
    before = {"seq_lens": ints([17, 300, 1]), "cu_rows": ints([0] * 4), "block_tables": torch.full_like(b.table, -1)}
    now = {k: v.clone() for k, v in before.items()}
    out = torch.empty(b.n, 6, 128, device=DEV)
    ws = {w: K.alloc_attn_workspace(b.cache, b.n, 3, 6, max(rows), 5000, w) for w in (0, 600)}

    def call(meta, window):
        if max(rows) == 1 and last != "cu_rows":
            return K.decode_local(b.cache, b.q, meta["seq_lens"], meta["block_tables"], 5000, b.scale, window, out=out,
                                  workspace=ws[window])
        return K.attn_seqs(b.cache, b.q, meta["cu_rows"], meta["seq_lens"], meta["block_tables"], max(rows), 5000, b.scale,
                           window=window, out=out, workspace=ws[window])

    def step(window):
        for name in sorted(right, key=lambda n: n == last):
            write(now[name], right[name])
        call(now, window)
        for name in right:
            write(now[name], before[name])

    for window in (0, 600):
        want = call(right, window).clone()
        torch.cuda.synchronize()
        for _ in range(5):
            out.zero_()
            step(window)
            assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(window)
        for _ in range(5):
            out.zero_()
            graph.replay()
            assert torch.equal(out, want)


# ------------------------------------------------------------------ weights far below a row's largest

class OverSink(Batch):
    """A first token whose score is 18, 20.5 or 23 powers of two above all others' (a head
    each) and whose value is zero: the output is made of the others' weights.

    p of the kernel for many rows (4-bit and TQ4 rows) is fp16 with the row's largest at 2^7 or
    more, so a small one is also off by half a step of fp16's subnormals, 2^-25: 2^-32 of the
    row's largest weight, here next to 1, in the mean square 2^-32 / sqrt(3) for every key."""

    def __init__(self, K, fmt, D, rows, seed):
        T = 6000
        super().__init__(K, fmt, 1, D, 64, [T], [rows], 3, seed=seed, dtype=torch.float32)
        u = torch.sign(rnd((D,), seed, D, "u"))
        k, v = 0.05 * rnd((T, 1, D), seed, D, "keys"), rnd((T, 1, D), seed, D, "values")
        k[0, 0], v[0] = u, 0.0
        pos = torch.arange(T, device=DEV)
        slots = self.table[0].long()[pos // 64] * 64 + pos % 64
        K.store(self.cache, k.to(torch.bfloat16), v.to(torch.bfloat16), slots.to(torch.int32))
        gap = torch.tensor([18.0, 20.5, 23.0], device=DEV)
        self.q = (gap * math.log(2.0) / (self.scale * D))[:, None] * u + 0.1 * rnd((rows, 3, D), seed, D, "q")

    def want(self, window=0, sinks=0):
        out, var = super().want(window, sinks)
        if self.n < 100 or self.fmt == "bf16":
            return out, var
        T = self.lens[0]
        key, p = torch.arange(T, device=DEV), torch.arange(T - self.n, T, device=DEV)[:, None]
        seen = key <= p
        if window:
            seen = seen & ((key > p - window) | (key < sinks))
        _, v = self.kv(0, key)
        return out, var + (seen.double() @ self.turn(v[0], inverse=True) ** 2)[:, None] * 2.0 ** -64 / 3


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 3, 150])
def test_weights_far_below_the_largest(K, fmt, D, rows):
    b = OverSink(K, fmt, D, rows, 45)
    for window, sinks in ((0, 0), (4000, 1)):
        b.check(b.attn(window, sinks), window, sinks)


# ------------------------------------------------------------------ many values that are not numbers

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("rows", [3, 84, 130])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_rows_between_keys_that_are_not_numbers(K, fmt, D, rows, what):
    """Two runs of whole tokens that are not numbers: the rows that see neither keep their
    bits, those that see one are not finite."""
    T, W = 484, 33
    b = Batch(K, fmt, 2, D, 16, [T], [rows], 3, seed=47)
    want = b.attn(W)
    runs = [list(range(T - 84, T - 79)), list(range(T - 24, T - 19))]
    for run, sign in zip(runs, (1, -1)):
        for key in run:
            at = int(b.table[0, key // 16]), slice(None), key % 16
            (b.cache.v if fmt == "bf16" else b.cache.v_scale)[at] = what * sign
    outs = [b.attn(W) for _ in range(3)]
    for got in outs:
        assert torch.equal(got.nan_to_num(777.0), outs[0].nan_to_num(777.0))
    for i, p in enumerate(range(T - rows, T)):
        seen = [any(p - W < key <= p for key in run) for run in runs]
        if not any(seen):
            assert torch.equal(outs[0][i], want[i]), p
        else:  # (an infinite value's product with a weight's second half may be NaN)
            assert not bool(outs[0][i].isfinite().any()), p


# ------------------------------------------------------------------ scores at which 32 bits are coarse

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("rows", [1, 3, 150])
def test_scores_of_any_size(K, fmt, D, rows):
    """One key's score is several times all others': its value is the output, at any size."""
    T, key = 600, 100
    b = Batch(K, fmt, 1, D, 64, [T], [rows], 3, seed=53)
    u = torch.sign(rnd((D,), 53, D, "u"))
    pos = torch.arange(T, device=DEV)
    slots = b.table[0].long()[pos // 64] * 64 + pos % 64
    k, v = rnd((T, 1, D), 53, D, "keys", scale=0.3), rnd((T, 1, D), 53, D, "values", scale=3.0)
    k[key, 0] = 4 * u
    K.store(b.cache, k.to(torch.bfloat16), v.to(torch.bfloat16), slots.to(torch.int32))
    for size in (10, 24, 25, 26, 27, 28, 29, 30, 35, 40, 60):  # the score is about 2^size
        b.q = ((2.0 ** size / (4 * D * b.scale)) * (u + 0.1 * rnd((rows, 3, D), 53, D, "q"))).to(torch.bfloat16)
        b.check(b.attn(), 0, 0)
        b.check(b.attn(520, 2), 520, 2)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("rows", [1, 3, 150])
@pytest.mark.parametrize("first", [True, False])
def test_scores_far_below_the_others(K, fmt, D, rows, first):
    """The first (or the last) keys' scores are millions of powers of two below the others'."""
    T = 1500
    b = Batch(K, fmt, 1, D, 64, [T], [rows], 3, seed=55)
    u = torch.sign(rnd((D,), 55, D, "u"))
    pos = torch.arange(T, device=DEV)
    slots = b.table[0].long()[pos // 64] * 64 + pos % 64
    k, v = rnd((T, 1, D), 55, D, "keys"), rnd((T, 1, D), 55, D, "values")
    far = slice(0, 700) if first else slice(800, T)
    k[far] = -30000 * u * (1 + 0.1 * rnd((T, 1, 1), 55, D, "far")[far])
    K.store(b.cache, k.to(torch.bfloat16), v.to(torch.bfloat16), slots.to(torch.int32))
    b.q = (8 * u + rnd((rows, 3, D), 55, D, "q")).to(torch.bfloat16)
    b.check(b.attn(), 0, 0)
    b.check(b.attn(1300, 64), 1300, 64)


# ------------------------------------------------------------------ scales that need the second pass

@pytest.mark.parametrize("fmt", SCALED)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 5), (300, 37)])
def test_large_scales_that_nobody_sees_beside_many_rows(K, fmt, D, window, sinks):
    """As above: such slots do not send the rows over their keys once more, in other units."""
    b = Batch(K, fmt, 2, D, 64, [777, 300], [150, 150], 3, seed=49, v_scale=1e-5)
    want = b.attn(window, sinks)
    hidden = unseen(b, window, sinks)
    for s in (b.cache.k_scale, b.cache.v_scale):
        s.transpose(1, 2)[hidden] = 60000.0
    assert torch.equal(b.attn(window, sinks), want)


@pytest.mark.parametrize("fmt", SCALED)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("plane", ["k", "v"])
def test_small_scales_beside_large_ones(K, fmt, D, plane):
    """One key with a scale of 60000 among small ones (4-bit rows: of a group of zeros)."""
    T, rows, key = 600, 150, 100
    small = 1e-3 if fmt == "tq4" else 5e-3  # scales of 1e-3 and up
    b = Batch(K, fmt, 1, D, 64, [T], [rows], 3, seed=51, v_scale=small if plane == "v" else 1.0)
    if plane == "k":
        pos = torch.arange(T, device=DEV)
        slots = b.table[0].long()[pos // 64] * 64 + pos % 64
        k = (small * rnd((T, 1, D), 51, D, "small")).to(torch.bfloat16)
        K.store(b.cache, k, rnd((T, 1, D), 51, D, "values", dtype=torch.bfloat16), slots.to(torch.int32))
        b.q = (b.q.float() / small).to(torch.bfloat16)
    at = int(b.table[0, key // 64]), 0, key % 64
    code, scale = (b.cache.k, b.cache.k_scale) if plane == "k" else (b.cache.v, b.cache.v_scale)
    if fmt == "tq4":
        scale[at] = 60000.0
    else:
        scale[(*at, 1)] = 60000.0
        code[at][16:32] = 0x88
    b.check(b.attn(), 0, 0)


class BesideLarge(Batch):
    """The token that nearly all of the weight falls on (16 powers of two above the others) has
    one large value scale, of a group of zeros; its other groups are the output.

    In the kernel for few rows a weight times a value scale is fp16 with the row's largest such
    product (of a token's largest scale) at 2^11 or more, so it is also off by half a step of the
    subnormals, 2^-25: 2^-36 of that product, here next to `large`, and its code multiplies it."""

    def __init__(self, K, fmt, D, rows, large):
        T, key = 600, 100
        super().__init__(K, fmt, 1, D, 64, [T], [rows], 3, seed=57)
        self.large = large
        u = torch.sign(rnd((D,), 57, D, "u"))
        pos = torch.arange(T, device=DEV)
        slots = self.table[0].long()[pos // 64] * 64 + pos % 64
        k, v = 0.05 * rnd((T, 1, D), 57, D, "keys"), rnd((T, 1, D), 57, D, "values")
        k[key, 0] = u
        K.store(self.cache, k.to(torch.bfloat16), v.to(torch.bfloat16), slots.to(torch.int32))
        at = int(self.table[0, key // 64]), 0, key % 64
        self.cache.v_scale[(*at, 1)] = large
        self.cache.v[at][16:32] = 0x88
        self.q = (16 * math.log(2.0) / (self.scale * D) * u + 0.1 * rnd((rows, 3, D), 57, D, "q")).to(torch.bfloat16)

    def want(self, window=0, sinks=0):
        out, var = super().want(window, sinks)
        if self.n < 100:
            key = torch.arange(self.lens[0], device=DEV)
            pg, slot = self.table[0].long()[key // 64], key % 64
            _, v = self.kv(0, key)
            code = v[0] / self.cache.v_scale[pg, 0, slot].double().repeat_interleave(32, -1)
            var = var + self.mix((code ** 2).sum(0)) * (2.0 ** -36 * self.large) ** 2 / 3
        return out, var


@pytest.mark.parametrize("fmt", ["q4_had32", "q4_0"])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("rows", [1, 3, 150])
@pytest.mark.parametrize("large", [17.0, 1000.0, 60000.0])
def test_groups_beside_a_large_scale(K, fmt, D, rows, large):
    b = BesideLarge(K, fmt, D, rows, large)
    b.check(b.attn(), 0, 0)


# ------------------------------------------------------------------ shapes, places and scales that nothing above has

def off_by(x, dtype, by=1):
    """x in a buffer whose rows start `by` elements behind a boundary and end on odd ones."""
    n, h, d = x.shape
    flat = torch.full((n * (h + 1) * (d + 3) + by,), 7.0, dtype=dtype, device=DEV)
    view = flat[by:].view(n, h + 1, d + 3)[:, :h, :d]
    view.copy_(x)
    return view


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 5, 130])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_off_their_boundaries(K, fmt, D, rows, dtype):
    b = Batch(K, fmt, 2, D, 16, [500, 300], [rows, rows], 3, seed=61)
    want = b.attn(90, 3, dtype=dtype)
    place = off_by(torch.zeros_like(want, dtype=torch.float32), dtype)
    q = off_by(b.q, dtype)
    got = K.attn_seqs(b.cache, q, ints(b.cu), ints(b.lens), b.table, rows, 500, b.scale, window=90, sinks=3, out=place)
    assert torch.equal(got, want)
    around = place.as_strided((2 * rows, 7, D + 3), (7 * (D + 3), D + 3, 1))
    assert bool((around[:, 6] == 7).all()) and bool((around[:, :, D:] == 7).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_many_sequences(K, fmt):
    """Hundreds of sequences: the many-row kernel finds its rows over several rounds."""
    g = torch.Generator().manual_seed(63)
    lens = torch.randint(0, 200, (700,), generator=g).tolist()
    rows = [int(r) % (n + 1) for r, n in zip(torch.randint(0, 90, (700,), generator=g), lens)]
    b = Batch(K, fmt, 1, 64, 32, lens, rows, 2, seed=63, pad=0)
    b.check(b.attn(30, 2), 30, 2)
    c = Batch(K, fmt, 1, 64, 32, lens, [1] * 700, 2, seed=64, pad=0)
    c.check(c.local(0), 0, 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [1, 3, 150])
@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30])
def test_other_scales_of_scores(K, fmt, rows, scale):
    b = Batch(K, fmt, 2, 128, 16, [700, 90], [rows, rows], 3, seed=65)
    b.scale = scale
    b.check(b.attn(), 0, 0)
    b.check(b.attn(60, 4), 60, 4)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("rows", [1, 5, 150])
def test_queries_that_are_not_numbers(K, fmt, D, rows):
    """A query's NaN or infinity reaches its own row and head, and nobody else."""
    b = Batch(K, fmt, 2, D, 16, [500, 300], [rows, rows], 3, seed=67)
    want = b.attn(90, 3)
    b.q = b.q.clone()
    b.q[rows - 1, 1, 5], b.q[rows, 4, 0] = math.nan, math.inf
    got = b.attn(90, 3)
    other = torch.ones(2 * rows, 6, dtype=torch.bool, device=DEV)
    other[rows - 1, 1] = other[rows, 4] = False
    assert torch.equal(got[other], want[other])
    assert bool(got[rows - 1, 1].isnan().all()) and not bool(got[rows, 4].isfinite().all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [[1, 1], [3, 0], [150, 7]])
def test_nothing_stored(K, fmt, rows):
    """Sequences without a token: every row sits at a negative position."""
    b = Batch(K, fmt, 2, 128, 16, [0, 0], rows, 3, seed=69)
    for window, sinks in ((0, 0), (5, 3)):
        out = torch.full((b.n, 6, 128), 7.0, device=DEV)
        status = ints([0])
        got = b.attn(window, sinks, out=out, status=status)
        assert bool((got == 0).all()) and int(status) == 0


# ------------------------------------------------------------------ where the work is split otherwise

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [6, 7, 12, 13])
def test_columns_beside_the_limits(K, fmt, D, rows):
    """24, 28, 48 and 52 columns: either side of the numbers at which the kernel for many rows
    takes over from that for few (tests/test_gpu_attn_seqs.py has 32, 36, 40, 64 and 68)."""
    for lens in ([2049], [1501, 700, rows]):
        b = Batch(K, fmt, 2, D, 16, lens, [rows] * len(lens), 4, seed=rows, dtype=torch.float32)
        b.check(b.attn(), 0, 0)
        b.check(b.attn(900, 7), 900, 7)


def test_rows_of_bad_lengths_are_left(K):
    """Every row of a sequence that is not computed is left as it was, and the valid
    sequences' rows keep their bits."""
    b = Batch(K, "q4_had32", 2, 256, 16, [100, 60, 80], [10, 1, 5], 3, seed=21)
    want = b.attn()
    for cu, left, same in (([0, 10, 9, 14], slice(14, 16), slice(0, 9)),  # (the third's rows lie over the first's last)
                           ([-1, 10, 11, 16], slice(0, 10), slice(10, 16)), ([0, 10, 11, 17], slice(11, 16), slice(0, 11)),
                           ([0, 11, 12, 16], slice(0, 11), slice(0, 0))):
        out = torch.full((16, 6, 256), 3.0, device=DEV)
        status = ints([0])
        K.attn_seqs(b.cache, b.q, ints(cu), ints(b.lens), b.table, 10, 100, b.scale, out=out, status=status)
        assert int(status) == K.DEV_BAD_LENGTH
        assert bool((out[left] == 3).all()) and torch.equal(out[same], want[same])
        done = torch.ones(16, dtype=torch.bool, device=DEV)
        done[left] = False
        assert not bool((out[done] == 3).all(-1).any())


# ------------------------------------------------------------------ one workspace for several shapes

@pytest.mark.parametrize("window", [0, 4096])
def test_one_workspace_for_every_batch(K, window):
    lens = [20000, 9000, 300, 7000, 15000, 4000, 12000, 18000] * 4
    b = Batch(K, "q4_had32", 4, 256, 16, lens, [1] * 32, 6, seed=71, pad=0)
    ws = K.alloc_attn_workspace(b.cache, 32, 32, 24, 1, 20000, window, smaller=True)
    lens = ints(lens)
    needs = []
    for n in range(1, 33):
        args = (b.cache, b.q[:n], lens[:n], b.table[:n], 20000, b.scale, window)
        needs.append(K.attn_workspace_size(b.cache, n, n, 24, 1, 20000, window))
        assert needs[-1] <= ws.numel()
        assert torch.equal(K.decode_local(*args, workspace=ws), K.decode_local(*args))
    assert needs != sorted(needs)  # a size is its own shape's
    for rows in (2, 9, 100):  # and few or many rows of fewer sequences
        big = K.alloc_attn_workspace(b.cache, 800, 32, 24, 100, 20000, window, smaller=True)
        for n in (1, 2, 3, 8):
            q = b.q[:1].expand(n * rows, 24, 256)
            args = (b.cache, q, ints(range(0, n * rows + 1, rows)), lens[:n], b.table[:n], rows, 20000, b.scale, window)
            assert torch.equal(K.attn_seqs(*args, workspace=big), K.attn_seqs(*args))
