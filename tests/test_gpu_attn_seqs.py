"""Rows of several sequences over the paged cache, with windows and sinks (decode_local,
attn_seqs), against plain 64-bit arithmetic on the values that the cache holds.

Tolerances count roundings.  In the cache's space an output value is sum_j w_j v_j with
weights w_j = p_j / z.  A weight is rounded to fp16 (or two bf16 halves), at most twice,
each off by at most 2^-12 of it (uniform: 2^-12 / sqrt(3) in the mean square); its score is
off where an operand was rounded before the product: queries and keys each by at most
2^-12 of every term in the kernel for many rows (2^-22 and not at all in the one for few);
values by 2^-12 there.  The roundings are independent, so the error's mean square is the sum
of theirs, and the tests allow eight times its root (the plain form's own error in 64
bits is nothing beside it), then the output's half step.  bf16 rows' operands are bf16 (a
half step of 2^-9) in the kernel for many rows.  An error of a weight is one for all of its
row's values (of a group of them), so it multiplies the value rotated back; those of the
values themselves mix orthonormally as they are rotated back: their mean squares average.
"""
import itertools
import math

import pytest
import torch

from bit_quantized_kv_store_gb300 import synth
from tests.test_gpu_parity import K  # noqa: F401

pytestmark = pytest.mark.gpu

DEV = "cuda"
LEVELS = (0.12841796875, 0.387939453125, 0.65673828125, 0.9423828125, 1.255859375, 1.6181640625, 2.068359375,
          2.732421875)
FMTS = {"q4_had32": 0, "bf16": 1, "q4_0": 3, "tq4": 4}


def rnd(shape, *key, dtype=torch.float32, scale=1.0):
    return (synth.normal(shape, DEV, "attn_seqs", *key) * scale).to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Batch:
    """A filled cache of `lens` tokens a sequence in shuffled pages, and queries for its last `rows`."""

    def __init__(self, K, fmt, Hk, D, ps, lens, rows, group, seed=0, dtype=torch.bfloat16, spread=0.3, v_scale=1.0, pad=1,
                 spare_pages=3):
        self.K, self.fmt, self.Hk, self.D, self.ps, self.lens, self.rows, self.group = K, fmt, Hk, D, ps, lens, rows, group
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // ps) for n in lens]
        self.wide = max(need + [1]) + pad
        total = sum(need) + spare_pages
        order = torch.randperm(total, generator=g).to(torch.int32)
        signs = torch.randint(-2 ** 31, 2 ** 31, (D // 32,), generator=g).to(torch.int32).to(DEV)
        self.cache = K.Cache(FMTS[fmt], Hk, D, ps, total, signs=signs if fmt == "tq4" else None)
        self.table = torch.full((len(lens), self.wide), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.table = self.table.to(DEV)
        for b, n in enumerate(lens):
            if n:
                pos = torch.arange(n, device=DEV)
                slots = (self.table[b].long()[pos // ps] * ps + pos % ps).to(torch.int32)
                mag = torch.exp(spread * rnd((n, Hk, 1), seed, b, "mag"))
                k = (rnd((n, Hk, D), seed, b, "k") * mag).to(torch.bfloat16)
                v = (rnd((n, Hk, D), seed, b, "v") * mag * v_scale).to(torch.bfloat16)
                K.store(self.cache, k, v, slots)
        self.n = sum(rows)
        self.cu = [0, *itertools.accumulate(rows)]
        self.q = rnd((self.n, Hk * group, D), seed, "q", dtype=dtype, scale=2.0)
        self.scale = D ** -0.5

    def kv(self, b, keys):
        """Values at positions `keys` of sequence b in the cache's space, 64 bits [heads, keys, D]."""
        slots = self.table[b].long()[keys // self.ps] * self.ps + keys % self.ps
        k, v = self.K.load(self.cache, slots.to(torch.int32), dtype=torch.float32, rotate_back=0)
        return k.double().transpose(0, 1), v.double().transpose(0, 1)

    def turn(self, x, inverse=False):
        """Rows into the cache's space, 64 bits, and back."""
        x = x.double()
        n = {"q4_had32": 32, "tq4": self.D}.get(self.fmt)
        if not n:
            return x
        i = torch.arange(n, device=DEV)
        bits = i[:, None] & i[None, :]
        odd = sum((bits >> s) & 1 for s in range(9)) & 1
        h = (1.0 - 2.0 * odd.double()) / math.sqrt(n)
        if self.fmt == "tq4":
            d = torch.arange(self.D, device=DEV)
            sg = 1.0 - 2.0 * ((self.cache.signs.long()[d // 32] >> (d % 32)) & 1).double()
            return (x @ h) * sg if inverse else (x * sg) @ h
        return (x.reshape(-1, 32) @ h).reshape(x.shape)

    def mix(self, var):
        """Mean squares of values rotated back."""
        n = {"q4_had32": 32, "tq4": self.D}.get(self.fmt)
        if not n:
            return var
        return var.reshape(*var.shape[:-1], -1, n).mean(-1, keepdim=True).expand(*var.shape[:-1], self.D // n, n).reshape(var.shape)

    def want(self, window=0, sinks=0):
        """(outputs, mean squares of their errors) [rows, heads, D] in 64 bits."""
        out = torch.zeros(self.n, self.Hk * self.group, self.D, dtype=torch.float64, device=DEV)
        var = torch.zeros_like(out)
        for b, (T, n) in enumerate(zip(self.lens, self.rows)):
            if T == 0 or n == 0:
                continue
            key = torch.arange(T, device=DEV)
            if window:
                key = key[(key < sinks) | (key > T - n - window)]
            k, v = self.kv(b, key)
            back = self.turn(v, inverse=True)
            p = torch.arange(T - n, T, device=DEV)[:, None]
            seen = key <= p
            if window:
                seen = seen & ((key > p - window) | (key < sinks))
            q = self.turn(self.q[self.cu[b]:self.cu[b + 1]])
            for h in range(self.Hk * self.group):
                kh, vh, qh, vo = k[h // self.group], v[h // self.group], q[:, h], back[h // self.group]
                s = torch.where(seen, qh @ kh.T * self.scale, -math.inf)
                top = s.amax(-1, keepdim=True)
                w = torch.where(seen, torch.exp(s - torch.where(top > -math.inf, top, 0.0)), 0.0)
                w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
                o = w @ vo
                out[self.cu[b]:self.cu[b + 1], h] = o
                half = 2.0 ** -9 if self.fmt == "bf16" else 2.0 ** -12
                u2 = half ** 2 / 3
                s2 = (qh ** 2) @ (kh ** 2).T * 2  # of a score: q and k rounded
                if self.fmt == "tq4":
                    # level x scale: a rounding is one for all elements of a row with that level, +-
                    pg = self.table[b].long()[key // self.ps]
                    mag = kh.abs() / self.cache.k_scale[pg, h // self.group, key % self.ps].double()[:, None]
                    s2 = s2 / 2 + sum((qh @ torch.where((mag - m).abs() < 1e-2, kh, 0.0).T) ** 2 for m in LEVELS)
                s2 = s2 * self.scale ** 2 * u2
                s2 = torch.where(seen, s2, 0.0)
                # a relative error of a score's p_j moves the output by w_j (v_j - o), one of p' alone by w_j v_j
                m = (w ** 2 * s2) @ vo ** 2 - 2 * o * ((w ** 2 * s2) @ vo) + o ** 2 * (w ** 2 * s2).sum(-1, keepdim=True)
                own = self.mix(w ** 2 @ vh ** 2)
                if self.fmt == "tq4":  # (as for keys)
                    mag = vh.abs() / self.cache.v_scale[pg, h // self.group, key % self.ps].double()[:, None]
                    own = w ** 2 @ sum(self.turn(torch.where((mag - m_).abs() < 1e-2, vh, 0.0), inverse=True) ** 2 for m_ in LEVELS)
                var[self.cu[b]:self.cu[b + 1], h] = m.clamp(min=0) + (w ** 2 @ vo ** 2) * 2 * u2 + own * u2
        return out, var

    def check(self, got, window=0, sinks=0, rows=None):
        want, var = self.want(window, sinks)
        half = torch.finfo(got.dtype).eps / 2
        # (2^-18 of the largest value: sums of thousands of fp32 terms)
        tol = 8 * var.sqrt() + half * want.abs() + 2.0 ** -18 * want.abs().amax() + 1e-30
        bad = ~((got.double() - want).abs() <= tol)
        if rows is not None:
            bad = bad[rows]
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}, " \
                              f"error {float(((got.double() - want).abs() / tol).nan_to_num(9e9).max()):.3g} of the tolerance"

    def attn(self, window=0, sinks=0, **kw):
        return self.K.attn_seqs(self.cache, self.q, ints(self.cu), ints(self.lens), self.table, max(self.rows + [0]),
                                max(self.lens + [0]), self.scale, window=window, sinks=sinks, **kw)

    def local(self, window, sinks=0, **kw):
        return self.K.decode_local(self.cache, self.q, ints(self.lens), self.table, max(self.lens), self.scale, window,
                                   sinks=sinks, **kw)


# ------------------------------------------------------------------ single tokens

LOCAL = [(0, 0), (1, 0), (1, 1), (16, 0), (17, 5), (64, 16), (100, 33), (1000, 4), (100000, 7)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", LOCAL)
def test_decode_local(K, fmt, D, window, sinks):
    lens = [1, 0, 2, 15, 16, 17, 33, 129, 700, 1501]
    b = Batch(K, fmt, 2, D, 16, lens, [1] * len(lens), 3, seed=D + window)
    b.check(b.local(window, sinks, dtype=torch.bfloat16), window, sinks)
    b.check(b.local(window, sinks), window, sinks)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hk,group", [(1, 1), (1, 8), (4, 6), (8, 2), (1, 12), (2, 64)])
def test_decode_local_heads(K, fmt, Hk, group):
    b = Batch(K, fmt, Hk, 128, 48, [301, 77], [1, 1], group, seed=group, dtype=torch.float32)
    b.check(b.local(50, 4), 50, 4)
    b.check(b.local(0), 0, 0)


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_local_long(K, fmt):
    """One sequence over many CTAs: clusters and ranges."""
    b = Batch(K, fmt, 1, 256, 64, [40001], [1], 5, seed=1)
    for window, sinks in ((0, 0), (4096, 4), (30011, 100), (1024, 1000)):
        b.check(b.local(window, sinks), window, sinks)


def test_pages_not_seen_are_not_looked_at(K):
    lens, W, S = [900, 333, 40], 100, 20
    b = Batch(K, "q4_had32", 2, 256, 16, lens, [1, 1, 1], 4, seed=5)
    want = b.local(W, S)
    table = b.table.cpu()
    for i, n in enumerate(lens):
        for p in range(table.shape[1]):
            seen = any(j < n and (j < S or j > n - 1 - W) for j in range(16 * p, 16 * p + 16))
            if not seen:
                table[i, p] = (-1, 10 ** 9, -2 ** 31)[p % 3]
    status = ints([0])
    got = K.decode_local(b.cache, b.q, ints(lens), table.to(DEV), 900, b.scale, W, sinks=S, status=status)
    assert torch.equal(got, want) and int(status) == 0


# ------------------------------------------------------------------ ragged chunks

CHUNKS = [  # lens, rows
    ([1], [1]),
    ([5], [5]),
    ([40, 17, 300, 1], [3, 17, 40, 0]),
    ([200, 64, 0, 130, 77], [200, 64, 0, 1, 70]),
    ([3, 50], [9, 2]),  # rows at negative positions
    ([40, 0, 300], [100, 70, 90]),
    ([1500], [333]),
    ([700, 900], [129, 260]),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(CHUNKS)))
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 5), (200, 70)])
def test_attn_seqs(K, fmt, D, case, window, sinks):
    lens, rows = CHUNKS[case]
    b = Batch(K, fmt, 2, D, 32, lens, rows, 3, seed=case)
    b.check(b.attn(window, sinks, dtype=torch.bfloat16), window, sinks)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hk,group", [(1, 1), (1, 8), (4, 6), (1, 7), (2, 16), (1, 64)])
@pytest.mark.parametrize("n", [4, 150])
def test_attn_seqs_heads(K, fmt, Hk, group, n):
    b = Batch(K, fmt, Hk, 256, 16, [n + 500, n], [n, n], group, seed=group, dtype=torch.float32)
    b.check(b.attn(), 0, 0)
    b.check(b.attn(60, 3), 60, 3)


def test_strides_and_rows_left_alone(K):
    b = Batch(K, "q4_had32", 2, 256, 16, [300, 90], [200, 20], 3, seed=9)
    want = b.attn()
    wide = torch.zeros(260, 10, 256, dtype=torch.bfloat16, device=DEV)
    wide[20:240, 2:8] = b.q
    out = torch.full((6, 260, 264), 7.0, device=DEV).transpose(0, 1)[..., :256]
    got = K.attn_seqs(b.cache, wide[:, 2:8], ints([20, 220, 240]), ints(b.lens), b.table, 200, 300, b.scale, out=out)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(out[20:240], want) and bool((out[:20] == 7).all()) and bool((out[240:] == 7).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [2, 100])
def test_bad_pages(K, fmt, rows):
    """Rows that see a key of a bad page are NaN, the others as they are without it."""
    b = Batch(K, fmt, 2, 256, 16, [600], [rows], 3, seed=11)
    for window, sinks, page in ((0, 0, 36), (0, 0, 37), (30, 0, 36), (30, 5, 0), (30, 5, 20)):
        want = b.attn(window, sinks)
        table = b.table.clone()
        table[0, page] = (-1, b.cache.num_pages)[page % 2]
        status = ints([0])
        got = K.attn_seqs(b.cache, b.q, ints(b.cu), ints(b.lens), table, rows, 600, b.scale, window=window, sinks=sinks,
                          status=status)
        keys = range(16 * page, 16 * page + 16)
        hit = [any(j <= p and (not window or j > p - window or j < sinks) for j in keys) for p in range(600 - rows, 600)]
        for i, h in enumerate(hit):
            if h:
                assert bool(got[i].isnan().all()), (window, page, i)
            else:
                assert torch.equal(got[i], want[i]), (window, page, i)
        assert (int(status) == K.DEV_BAD_PAGE) == any(hit)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [3, 100])
@pytest.mark.parametrize("what", ["k", "v"])
def test_values_that_are_not_numbers(K, fmt, rows, what):
    """A NaN key or value reaches the rows that see it, and nobody else."""
    for window, sinks, key in ((0, 0, 598), (0, 0, 550), (33, 0, 560), (33, 5, 3), (33, 5, 100)):
        b = Batch(K, fmt, 2, 256, 16, [600], [rows], 3, seed=13)
        want = b.attn(window, sinks)
        at = int(b.table[0, key // 16]), 1, key % 16
        if fmt == "bf16":
            (b.cache.k if what == "k" else b.cache.v)[at][100] = math.nan
        else:  # the scale of elements 96 .. 127, or of the row
            plane = b.cache.k_scale if what == "k" else b.cache.v_scale
            plane[at if fmt == "tq4" else (*at, 3)] = math.nan
        got = b.attn(window, sinks)
        for i, p in enumerate(range(600 - rows, 600)):
            seen = key <= p and (not window or key > p - window or key < sinks)
            assert torch.equal(got[i, :3], want[i, :3])
            if not seen:
                assert torch.equal(got[i, 3:], want[i, 3:]), (window, key, i)
            elif what == "k":
                assert bool(got[i, 3:].isnan().all())
            else:
                assert bool(got[i, 3:, 100].isnan().all())
                if fmt == "bf16":
                    assert not bool(got[i, 3:, :100].isnan().any() or got[i, 3:, 101:].isnan().any())
                elif fmt != "tq4":
                    assert not bool(got[i, 3:, :96].isnan().any() or got[i, 3:, 128:].isnan().any())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("v_scale", [1e-4, 300.0])
def test_scales_of_values(K, fmt, v_scale):
    b = Batch(K, fmt, 2, 256, 16, [600, 70], [3, 70], 3, seed=17, spread=1.5, v_scale=v_scale)
    b.check(b.attn())
    b = Batch(K, fmt, 2, 256, 16, [600, 70], [1, 1], 3, seed=17, spread=1.5, v_scale=v_scale)
    b.check(b.local(100, 4), 100, 4)


def test_rows_without_value_scales(K):
    """Zero values among others: their weights count."""
    b = Batch(K, "q4_had32", 1, 256, 16, [300], [1], 2, seed=19)
    b.cache.v_scale[b.table[0, 3:9].long()] = 0
    b.check(b.local(0))
    b.cache.v_scale.zero_()
    assert bool((b.local(0) == 0).all())


def test_bad_lengths(K):
    b = Batch(K, "q4_had32", 2, 256, 16, [100, 60, 80], [10, 1, 5], 3, seed=21)
    want = b.attn()
    for bad in (-1, 101, 2 ** 31 - 1):
        status = ints([0])
        got = K.attn_seqs(b.cache, b.q, ints(b.cu), ints([100, bad, 80]), b.table, 10, 100, b.scale, status=status)
        assert bool(got[10:11].isnan().all()) and torch.equal(got[:10], want[:10]) and torch.equal(got[11:], want[11:])
        assert int(status) == K.DEV_BAD_LENGTH
    # rows that are too many or outside: left as they were
    for cu, left in (([0, 10, 9, 14], slice(9, 16)), ([-1, 10, 11, 16], slice(0, 10)), ([0, 10, 11, 17], slice(11, 16)),
                     ([0, 11, 12, 16], slice(0, 11))):
        out = torch.full((16, 6, 256), 3.0, device=DEV)
        status = ints([0])
        K.attn_seqs(b.cache, b.q, ints(cu), ints(b.lens), b.table, 10, 100, b.scale, out=out, status=status)
        assert int(status) == K.DEV_BAD_LENGTH
        assert bool((out[left][-1] == 3).all()) or cu[2] == 9


def test_streams_graphs_and_workspaces(K):
    b = Batch(K, "q4_had32", 1, 256, 16, [9000, 500], [1, 1], 4, seed=23)
    want, wchunk = b.local(0), b.attn(300, 4)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = b.local(0)
    got2 = b.local(0, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, want)
    ws = K.alloc_attn_workspace(b.cache, 2, 2, 4, 1, 9000)
    ws.fill_(255)  # its contents do not matter
    lens, cu = ints(b.lens), ints(b.cu)
    out, out2 = torch.empty_like(want), torch.empty_like(wchunk)
    ws2 = K.alloc_attn_workspace(b.cache, 2, 2, 4, 1, 9000, 300, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.decode_local(b.cache, b.q, lens, b.table, 9000, b.scale, 0, out=out, workspace=ws)
        K.attn_seqs(b.cache, b.q, cu, lens, b.table, 1, 9000, b.scale, window=300, sinks=4, out=out2, workspace=ws2)
    for _ in range(3):
        out.zero_()
        out2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out2, wchunk)


def test_far_pages(K):
    """Rows past 2^31 bytes of a plane."""
    pages = 2 ** 24 // 16 + 64
    b = Batch(K, "q4_had32", 1, 256, 16, [700], [40], 3, seed=25, spare_pages=pages)
    far = b.table.clone()
    used = far[0, :44].long()
    new = torch.arange(pages - 44, pages, device=DEV)
    for t in (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale):
        t[new] = t[used].clone()
    def both():
        few = K.decode_local(b.cache, b.q[:1], ints([700]), b.table, 700, b.scale, 0)
        return b.attn(), b.attn(100, 3), few

    want = both()
    b.table[0, :44] = new.to(torch.int32)
    assert all(torch.equal(x, y) for x, y in zip(both(), want))


def test_with_the_calls_around(K):
    """A layer's step: the new tokens stored, then a chunk and a token attended over window and sinks."""
    Hk, Hq, D, ps, W, S = 2, 6, 256, 16, 64, 4
    cache = K.Cache(K.FMT_Q4_HAD32, Hk, D, ps, 40)
    table = torch.randperm(40, generator=torch.Generator().manual_seed(3)).to(torch.int32).reshape(2, 20).to(DEV)
    rope = K.Rope([1e4 ** (-i / 32) for i in range(32)])
    lens = [150, 33]
    qs, done = [], [0, 0]
    for rows in ([150, 33], [1, 1]):
        pos = torch.cat([torch.arange(d, d + r) for d, r in zip(done, rows)]).to(torch.int32).to(DEV)
        seq = torch.cat([torch.full((r,), i) for i, r in enumerate(rows)]).to(DEV)
        slots = (table[seq].long().gather(1, (pos.long() // ps)[:, None])[:, 0] * ps + pos % ps).to(torch.int32)
        x = rnd((sum(rows), Hq + 2 * Hk, D), "step", sum(rows), dtype=torch.bfloat16)
        q = K.norm_rope_store(cache, x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], slots, pos, rope=rope, rotate=False)
        done = [d + r for d, r in zip(done, rows)]
        qs.append((q, list(rows), list(done)))
        if rows[0] > 1:
            got = K.attn_seqs(cache, q, ints([0, 150, 183]), ints(done), table, 150, 150, D ** -0.5, window=W, sinks=S)
        else:
            got = K.decode_local(cache, q, ints(done), table, 160, D ** -0.5, W, sinks=S)
        b = Batch.__new__(Batch)
        b.K, b.fmt, b.Hk, b.D, b.ps, b.lens, b.rows, b.group = K, "q4_had32", Hk, D, ps, done, rows, 3
        b.cache, b.table, b.q, b.n, b.cu, b.scale = cache, table, q, sum(rows), [0, *itertools.accumulate(rows)], D ** -0.5
        b.check(got, W, S)
    assert lens[0] + 1 == done[0]


def test_workspace_is_asked_for(K):
    b = Batch(K, "q4_had32", 1, 256, 16, [40000], [1], 4, seed=27)
    size = K.attn_workspace_size(b.cache, 1, 1, 4, 1, 40000)
    assert size > 0
    for bad in (torch.empty(size - 1, dtype=torch.uint8, device=DEV), torch.empty(0, dtype=torch.uint8, device=DEV)):
        with pytest.raises(K.KvqError):
            b.local(0, workspace=bad)
    with pytest.raises(K.KvqError):  # off its 32 bytes
        b.local(0, workspace=torch.empty(size + 64, dtype=torch.uint8, device=DEV)[16:])
    ws = torch.full((size + 64,), 7, dtype=torch.uint8, device=DEV)
    assert torch.equal(b.local(0, workspace=ws[32:-32]), b.local(0))
    assert bool((ws[:32] == 7).all()) and bool((ws[-32:] == 7).all())


def test_tensors_that_are_refused(K):
    b = Batch(K, "q4_had32", 2, 128, 16, [50, 20], [2, 1], 2, seed=29)
    good = dict(cache=b.cache, q=b.q, cu_rows=ints(b.cu), seq_lens=ints(b.lens), block_tables=b.table, max_rows=2,
                max_seq_len=50, sm_scale=0.1)
    K.attn_seqs(**good)
    for name, bad in (("q", b.q.double()), ("q", b.q[..., :64]), ("q", b.q.cpu()), ("q", b.q[:, :3]), ("q", b.q[..., ::2]),
                      ("cu_rows", ints(b.cu)[:2]), ("cu_rows", ints(b.cu).long()), ("seq_lens", ints([50])),
                      ("block_tables", b.table[:1]), ("block_tables", b.table[:, ::2]), ("max_seq_len", -1), ("window", -1),
                      ("sinks", -2), ("max_rows", -1), ("out", torch.empty(3, 4, 64, device=DEV)), ("out", b.q),
                      ("out", torch.empty(3, 4, 128, dtype=torch.float16, device=DEV)), ("dtype", torch.float16),
                      ("sm_scale", math.nan), ("max_seq_len", 10 ** 6), ("status", torch.zeros(1, device=DEV)),
                      ("workspace", torch.zeros(1))):
        with pytest.raises((ValueError, TypeError, K.KvqError)):
            K.attn_seqs(**{**good, name: bad})
    fp8 = K.Cache(K.FMT_FP8_ROW, 1, 512, 16, 4, rope_dim=64)
    with pytest.raises(K.KvqError):
        K.decode_local(fp8, torch.zeros(1, 16, 512, device=DEV), ints([1]), ints([[0]]), 16, 1.0, 0)


def test_same_bits_whatever_the_batch(K):
    """A window's row does not depend on the sequences beside it, nor on other calls under way."""
    b = Batch(K, "tq4", 2, 128, 16, [3000, 3000, 900], [1, 1, 1], 4, seed=31)
    want = b.local(500, 4)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for s in streams:
            outs.append(b.local(500, 4, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    c = Batch(K, "q4_had32", 1, 256, 16, [700, 400], [150, 90], 6, seed=33)
    chunk = c.attn(200, 4)
    outs = [c.attn(200, 4, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, chunk) for o in outs)


def test_many_rows(K):
    """A whole prompt at once, longer than a grid dimension's 65535 blocks of 8 columns."""
    b = Batch(K, "q4_0", 8, 64, 64, [22000], [22000], 3, seed=35)
    b.check(b.attn(40, 5), 40, 5)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [1, 3, 150])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 0), (50, 5), (300, 37)])
def test_slots_that_nobody_sees(K, fmt, rows, window, sinks):
    """Whatever lies behind a sequence's end, or between sinks and window, reaches nobody."""
    b = Batch(K, fmt, 2, 256, 64, [777, 300], [rows, rows], 3, seed=37)
    want = b.attn(window, sinks)
    hidden = torch.ones(b.cache.num_pages, 64, dtype=torch.bool, device=DEV)
    for i, T in enumerate(b.lens):
        key = torch.arange(T, device=DEV)
        if window:
            key = key[(key < sinks) | (key > T - rows - window)]
        hidden[b.table[i].long()[key // 64], key % 64] = False
    for p in (b.cache.k, b.cache.v) if fmt == "bf16" else (b.cache.k_scale, b.cache.v_scale):
        p.transpose(1, 2)[hidden] = math.nan
    assert torch.equal(b.attn(window, sinks), want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 2, 4, 8, 9, 10, 11, 16, 17])
def test_rows_at_which_the_work_is_split_otherwise(K, fmt, D, rows):
    """Numbers of columns on both sides of the kernels' ranges (32, 36, 40, 64 and 68 of 4
    heads), one long sequence (clusters and their fold) and several of unequal lengths."""
    for lens in ([4099], [3001, rows, 700]):
        b = Batch(K, fmt, 2, D, 16, lens, [rows] * len(lens), 4, seed=rows, dtype=torch.float32)
        b.check(b.attn(), 0, 0)
        b.check(b.attn(900, 7), 900, 7)


@pytest.mark.parametrize("fmt", FMTS)
def test_a_window_of_one_row_over_many_clusters(K, fmt):
    b = Batch(K, fmt, 1, 128, 64, [20000], [1], 8, seed=3, dtype=torch.float32)
    b.check(b.attn(), 0, 0)
    b.check(b.local(15000, 33), 15000, 33)
