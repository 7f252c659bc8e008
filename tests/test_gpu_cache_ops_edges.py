"""The calls around the cache at values and layouts that the other tests leave out:
keys, queries and rows that are not numbers, a bad page inside a prompt chunk,
strides that no element uses, positions that axes share, outputs that do not fit."""
import math

import pytest
import torch

from tests.test_gpu_cache_ops import DEV, diff_problem, fill_random, make_cache, rnd, rope_of
from tests.test_gpu_parity import K  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ keys and queries that are not numbers

@pytest.mark.parametrize("fmt", ["Q4_HAD32", "Q4_0", "TQ4", "BF16"])
@pytest.mark.parametrize("T", [1, 2, 513, 512 * 33 + 1, 512 * 130 + 1])
def test_a_key_that_is_not_a_number(K, fmt, T):
    """The last key of one KV head is NaN, for most lengths alone in its partition: the
    heads that attend it are NaN in the merge and in both arrangements of its
    difference, the others as they are without it.  (Q4_0: a NaN among numbers is
    stored as code 0 under their scale, so that the row stays finite.)"""
    cache, q, lens, bt, T, ws = diff_problem(K, getattr(K, "FMT_" + fmt), [T])
    lam = torch.rand(12, device=DEV)
    at = T - 1
    slot = (bt[0, at // 16] * 16 + at % 16).to(torch.int32)[None]
    k, v = rnd((1, 4, 256), "nan key"), rnd((1, 4, 256), "nan value")
    results = []
    for bad in (False, True):
        if bad:
            k[0, 1, 7] = math.nan
        K.store(cache, k, v, slot)
        heads = K.decode(cache, q, lens, bt, T, 1 / 16, ws).clone()
        results.append((heads, K.decode_diff(cache, q, lens, bt, T, 1 / 16, ws, lam)))
    (h0, d0), (h1, d1) = results
    gone = torch.isfinite if fmt == "Q4_0" else torch.isnan
    assert gone(h1[0, 6:12]).all() and gone(d1[0, 3:6]).all()
    for a, b, hit in ((h0, h1, slice(6, 12)), (d0, d1, slice(3, 6))):
        keep = torch.ones(a.shape[1], dtype=torch.bool, device=DEV)
        keep[hit] = False
        assert torch.isfinite(a).all() and torch.equal(a[0, keep], b[0, keep])


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "Q4_0", "TQ4", "BF16"])
@pytest.mark.parametrize("T", [1, 700, 40000])
def test_a_query_that_is_not_a_number(K, fmt, T):
    cache, q, lens, bt, T, ws = diff_problem(K, getattr(K, "FMT_" + fmt), [T])
    lam = torch.rand(12, device=DEV)
    q[0, 5, 9] = math.nan
    heads = K.decode(cache, q, lens, bt, T, 1 / 16, ws)
    assert torch.isnan(heads[0, 5]).all() and torch.isfinite(heads[0, :5]).all() and torch.isfinite(heads[0, 6:]).all()
    for norm in (None, K.Norm(torch.ones(256, device=DEV))):
        y = K.decode_diff(cache, q, lens, bt, T, 1 / 16, ws, lam, norm=norm)
        assert torch.isnan(y[0, 2]).all() and torch.isfinite(y[0, :2]).all() and torch.isfinite(y[0, 3:]).all()


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "Q4_0", "TQ4", "BF16"])
@pytest.mark.parametrize("T", [1, 15, 700, 513, 40003])
def test_slots_behind_the_end_that_are_not_numbers(K, fmt, T):
    """The last page's slots behind the sequence hold NaN rows: the outputs are those
    over finite ones."""
    f = getattr(K, "FMT_" + fmt)
    cache, q, lens, bt, T, ws = diff_problem(K, f, [T])
    lam = torch.rand(12, device=DEV)
    want = K.decode(cache, q, lens, bt, T, 1 / 16, ws), K.decode_diff(cache, q, lens, bt, T, 1 / 16, ws, lam)
    page = bt[0, (T - 1) // 16].long()
    for name in ("k", "v") if f == K.FMT_BF16 else ("k_scale", "v_scale"):
        getattr(cache, name)[page, :, T % 16 or 16:] = math.nan
    got = K.decode(cache, q, lens, bt, T, 1 / 16, ws), K.decode_diff(cache, q, lens, bt, T, 1 / 16, ws, lam)
    assert torch.isfinite(want[0]).all() and all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ a bad page inside a prompt chunk

@pytest.mark.parametrize("fmt", ["Q4_HAD32", "Q4_0"])
@pytest.mark.parametrize("T0,n,bad", [(0, 200, 2), (0, 200, 5), (1000, 100, 64), (40, 1, 1)])
def test_rows_before_a_bad_page(K, fmt, T0, n, bad):
    """Rows that attend the page are NaN, the rows before it what they are with a good
    one, also those that share a query block with NaN rows."""
    f = getattr(K, "FMT_" + fmt)
    pages = (T0 + n + 15) // 16
    cache = make_cache(K, f, 4, 256, pages)
    fill_random(cache, K, n)
    junk = make_cache(K, f, 4, 256, pages)      # fills the shared memory with rows of NaN first
    for name in ("k", "v"):
        getattr(junk, name + "_scale").fill_(math.nan)
    bt = torch.arange(pages, dtype=torch.int32, device=DEV)
    broken = bt.clone()
    broken[bad] = pages
    q = rnd((n, 24, 256), "bp rows", n, scale=0.1)
    lam = torch.rand(12, device=DEV)
    first = max(0, min(n, 16 * bad - T0))        # the first row that attends the page
    for call in (lambda c, t, s: K.prefill_attn(c, q, T0, t, 1 / 16, status=s),
                 lambda c, t, s: K.prefill_diff(c, q, T0, t, 1 / 16, lam, status=s),
                 lambda c, t, s: K.prefill_diff(c, q, T0, t, 1 / 16, lam, norm=K.Norm(torch.ones(256, device=DEV)), status=s)):
        want = call(cache, bt, None)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        call(junk, bt, None)
        got = call(cache, broken, status)
        assert K.read_status(status) == K.DEV_BAD_PAGE
        assert torch.isfinite(want).all() and torch.equal(got[:first], want[:first])
        assert torch.isnan(got[first:]).all()


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "Q4_0"])
@pytest.mark.parametrize("T0,n,at", [(0, 200, 0), (0, 200, 70), (0, 200, 199), (1000, 100, 1031), (1000, 100, 3), (4000, 700, 4400)])
def test_rows_before_a_key_that_is_not_a_number(K, fmt, T0, n, at):
    """A chunk's rows that mask a NaN key or value are what they are without it; those
    that attend a NaN value lose its group of 32, those that attend a NaN key everything."""
    cache = make_cache(K, getattr(K, "FMT_" + fmt), 4, 256, (T0 + n + 15) // 16)
    fill_random(cache, K, n)
    bt = torch.arange(cache.num_pages, dtype=torch.int32, device=DEV)
    q = rnd((n, 24, 256), "nan rows", n, scale=0.1)
    lam = torch.rand(12, device=DEV)
    first = max(0, at - T0)
    calls = (lambda: K.prefill_attn(cache, q, T0, bt, 1 / 16), lambda: K.prefill_diff(cache, q, T0, bt, 1 / 16, lam))
    want = [f() for f in calls]
    for plane, groups, lost in (("v_scale", [3], slice(96, 128)), ("v_scale", [0, 7], None), ("k_scale", [5], slice(0, 256))):
        scales = getattr(cache, plane)
        keep = scales.clone()
        for G in groups:
            scales[at // 16, 2, at % 16, G] = math.nan
        for f, w in zip(calls, want):
            got, heads = f(), w.shape[1] // 4           # heads of a KV head
            hit = torch.zeros_like(got, dtype=torch.bool)
            mine = hit[first:, 2 * heads:3 * heads]
            if lost is None:
                mine[..., :32] = mine[..., 224:] = True
            else:
                mine[..., lost] = True
            # (of 2.4 million random scales a few are above 8188: -8 of them is infinite in the kernel's fp16)
            assert torch.isnan(got[hit]).all() and torch.allclose(got[~hit], w[~hit], rtol=0, atol=0, equal_nan=True)
        scales.copy_(keep)


# ------------------------------------------------------------------ rows that are not numbers, on the way in and back

BAD = {"nan": math.nan, "inf": math.inf, "-inf": -math.inf, "huge": 3e38}


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "Q4_0", "TQ4", "BF16", "FP8_ROW"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", sorted(BAD))
def test_store_of_values_that_are_not_numbers(K, fmt, dtype, kind):
    """norm_rope_store's bytes are kvq_store's for rows with NaN, infinities and values
    whose sums overflow, with and without norm and rotation; rows without them are untouched by
    their neighbours; read back, NaN stays in its group (row, part)."""
    f = getattr(K, "FMT_" + fmt)
    fp8 = f == K.FMT_FP8_ROW
    n, Hk, D, W = 9, 1 if fp8 else 3, 512 if fp8 else 256, 576 if fp8 else 256
    k, v, q = rnd((n, Hk, W), "bv k"), rnd((n, Hk, W), "bv v"), rnd((n, 6, W), "bv q")
    clean = k.clone(), v.clone()
    for x in (k, v, q):
        x[2, 0, 5] = BAD[kind]
        x[4, -1, 40], x[4, -1, 41] = BAD[kind], -BAD[kind]
        x[6, 0, 520 if fp8 else 255] = BAD[kind]
    k, v, q = (x.to(dtype) for x in (k, v, q))
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    rope = rope_of(K, 64, 0, 1)[0]
    pos = torch.arange(n, dtype=torch.int32, device=DEV) * 7
    for norm, rp in ((None, None), (K.Norm(rnd((D,), "bv w"), 1e-6), rope)):
        a, b = make_cache(K, f, Hk, D, 2), make_cache(K, f, Hk, D, 2)
        got = K.norm_rope_store(a, q, k, None if fp8 else v, slots, pos if rp else None, rope=rp,
                                q_norm=None if fp8 else norm, k_norm=norm)
        if fp8:
            k32, q32 = torch.empty(n, Hk, W, device=DEV), q.float().clone()
            K.norm_rope(k[..., :512], norm=norm, out=k32[..., :512])
            K.norm_rope(k[..., 512:], pos if rp else None, rope=rp, out=k32[..., 512:])
            K.norm_rope(q[..., 512:], pos if rp else None, rope=rp, out=q32[..., 512:])
            K.store(b, k32, None, slots)
            want = q32
        else:
            k32 = K.norm_rope(k, pos if rp else None, rope=rp, norm=norm, dtype=torch.float32)
            want = K.norm_rope(q, pos if rp else None, rope=rp, norm=norm, dtype=torch.float32)
            K.store(b, k32, v.float().contiguous(), slots)
            want = K.rotate_query(want) if f == K.FMT_Q4_HAD32 else K.tq4_rotate(b, want) if f == K.FMT_TQ4 else want
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
        for name in ("k", "v", "k_scale", "v_scale"):
            ta, tb = getattr(a, name), getattr(b, name)
            if ta is None:
                continue
            if ta.dtype != torch.uint8:
                assert torch.equal(torch.isnan(ta), torch.isnan(tb)), name
                ta, tb = ta.float().nan_to_num(nan=0.0), tb.float().nan_to_num(nan=0.0)
            assert torch.equal(ta, tb), name
        good = [0, 1, 3, 5, 7, 8]
        back = K.load(a, slots, dtype=torch.float32)
        c = make_cache(K, f, Hk, D, 2)
        ck, cv = (x.to(dtype) for x in clean)
        K.norm_rope_store(c, None, ck, None if fp8 else cv, slots, pos if rp else None, rope=rp, k_norm=norm)
        for x, y in zip(back, K.load(c, slots, dtype=torch.float32)):
            if x is not None:
                assert torch.equal(x[good], y[good]) and torch.isfinite(x[good]).all()
    if kind == "nan" and not fp8:      # (values: stored as they are; fp8 holds NaN as zero)
        hit = torch.zeros(n, Hk, D, dtype=torch.bool, device=DEV)
        group = {"Q4_HAD32": 32, "TQ4": 256, "BF16": 1}.get(fmt)
        for t, h, e in ((2, 0, 5), (4, Hk - 1, 40), (4, Hk - 1, 41), (6, 0, 255)):
            if group:
                hit[t, h, e // group * group:(e // group + 1) * group] = True
        if group:
            assert torch.equal(torch.isnan(back[1]), hit)


def test_heads_that_are_not_numbers(K):
    """diff_heads: NaN and infinity stay in their head (without a norm, in their element)."""
    x = rnd((5, 8, 256), "dh nan")
    lam = torch.rand(4, device=DEV)
    bad = x.clone()
    bad[1, 2, 7], bad[2, 5, 8], bad[3, 0, 9], bad[3, 1, 9] = math.nan, math.inf, math.inf, math.inf
    for norm in (None, K.Norm(torch.ones(256, device=DEV), 1e-5)):
        want, got = K.diff_heads(x, lam, norm=norm), K.diff_heads(bad, lam, norm=norm)
        hit = torch.zeros(5, 4, dtype=torch.bool, device=DEV)
        hit[1, 1] = hit[2, 2] = hit[3, 0] = True
        assert torch.equal(got[~hit], want[~hit])
        if norm is None:
            where = torch.zeros(5, 4, 256, dtype=torch.bool, device=DEV)
            where[1, 1, 7] = where[2, 2, 8] = where[3, 0, 9] = True
            assert torch.equal(~torch.isfinite(got), where) and torch.equal(got[~where], want[~where])
        else:
            assert torch.isnan(got[1, 1]).all() and torch.isnan(got[3, 0]).all()


# ------------------------------------------------------------------ strides that no element uses

def test_strides_of_single_elements_do_not_count(K):
    """One token, or one head, with a stride that nothing is reached by: the rows of the
    plain layout, in place as well."""
    x = rnd((1, 4, 256), "single")
    norm = K.Norm(rnd((256,), "single w"))
    want = K.norm_rope(x, norm=norm)
    for tok in (0, 1, 1024, 1025, 2 ** 33):
        y = x.clone()
        odd = torch.as_strided(y, (1, 4, 256), (tok, 256, 1))
        assert torch.equal(K.norm_rope(odd, norm=norm), want)
        K.norm_rope(odd, norm=norm, out=y)
        assert torch.equal(y, want)
    one = rnd((7, 1, 256), "single head")
    want = K.norm_rope(one, norm=norm)
    for head in (0, 1, 257, 2 ** 33):
        y = one.clone()
        odd = torch.as_strided(y, (7, 1, 256), (256, head, 1))
        assert torch.equal(K.norm_rope(odd, norm=norm), want)
        K.norm_rope(y, norm=norm, out=odd)
        assert torch.equal(y, want)
    cache = make_cache(K, K.FMT_Q4_HAD32, 1, 256, 2)
    fill_random(cache, K, 1)
    slots = torch.tensor([5], dtype=torch.int32, device=DEV)
    k, v = K.load(cache, slots)
    out = torch.zeros(1, 1, 256, dtype=torch.bfloat16, device=DEV)
    odd = torch.as_strided(out, (1, 1, 256), (2 ** 34, 3, 1))
    K.load(cache, slots, k=odd)
    assert torch.equal(out, k)
    again = make_cache(K, K.FMT_Q4_HAD32, 1, 256, 2)
    plain = make_cache(K, K.FMT_Q4_HAD32, 1, 256, 2)
    K.norm_rope_store(again, None, torch.as_strided(x, (1, 1, 256), (2 ** 34, 2 ** 35, 1)), x[:, :1], slots)
    K.norm_rope_store(plain, None, x[:, :1], x[:, :1], slots)
    assert torch.equal(again.k, plain.k) and torch.equal(again.v, plain.v)


def test_positions_that_all_axes_share(K):
    """Text positions broadcast over three axes: those of three equal rows."""
    n = 37
    rope = rope_of(K, 64, 0, 3)[0]
    x = rnd((n, 4, 128), "shared positions")
    pos = torch.arange(100, 100 + n, dtype=torch.int32, device=DEV)
    want = K.norm_rope(x, pos.repeat(3, 1), rope=rope)
    assert torch.equal(K.norm_rope(x, pos.expand(3, n), rope=rope), want)
    assert torch.equal(K.norm_rope(x[:1], pos[:1].expand(3, 1), rope=rope), want[:1])


def test_an_output_that_does_not_fit(K):
    """As an allocation of torch's own: the caller can tell it from other errors."""
    x = torch.zeros(1, 1, 512, device=DEV).expand(2 ** 30, 1, 512)       # 2 TB of output
    with pytest.raises(torch.OutOfMemoryError):
        K.norm_rope(x)
    c = make_cache(K, K.FMT_Q4_HAD32, 4, 256, 2)
    bt, cu = torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(torch.OutOfMemoryError):
        K.load_seqs(c, bt, cu, 2 ** 31 - 1)                              # 4 TB
    assert torch.equal(K.norm_rope(x[:3]), x[:3])


# ------------------------------------------------------------------ a norm's weight

def test_a_norm_follows_its_weight(K):
    """A parameter whose storage, type or place changes after the Norm was made: calls
    take it as it is, or refuse it."""
    x = rnd((3, 2, 256), "follow")
    new = [rnd((256,), "follow w", i) for i in range(3)]
    param = torch.nn.Parameter(new[0].clone(), requires_grad=False)
    norm = K.Norm(param, 1e-6, 1.0)
    c = make_cache(K, K.FMT_Q4_HAD32, 2, 256, 2)
    slots = torch.arange(3, dtype=torch.int32, device=DEV)

    def check(w):
        for got, want in ((K.norm_rope(x, norm=norm), K.norm_rope(x, norm=K.Norm(w, 1e-6, 1.0))),
                          (K.diff_heads(x, torch.ones(1, device=DEV), norm=norm),
                           K.diff_heads(x, torch.ones(1, device=DEV), norm=K.Norm(w, 1e-6, 1.0))),
                          (K.norm_rope_store(c, x, x, x, slots, q_norm=norm),
                           K.norm_rope_store(c, x, x, x, slots, q_norm=K.Norm(w, 1e-6, 1.0)))):
            assert torch.equal(got, want)

    check(new[0])
    param.data = new[1].clone()
    check(new[1])
    param.data = new[2].bfloat16()
    check(new[2].bfloat16())
    norm.weight = new[0]
    check(new[0])
    norm.weight = param
    for bad in (torch.ones(128, device=DEV), torch.ones(512, device=DEV)[::2], torch.ones(256)):
        param.data = bad
        with pytest.raises(ValueError):
            K.norm_rope(x, norm=norm)
    param.data = torch.ones(256, device=DEV, dtype=torch.float16)
    with pytest.raises(TypeError):
        K.norm_rope(x, norm=norm)


def test_a_cache_on_another_device_is_refused(K):
    """Every call compares the cache's device with its tensors' (here the handle names a
    device that the planes are not on)."""
    c = make_cache(K, K.FMT_Q4_HAD32, 2, 256, 4)
    x, q = rnd((3, 2, 256), "dev"), rnd((1, 4, 256), "dev q")
    slots = torch.arange(3, dtype=torch.int32, device=DEV)
    bt, cu = torch.arange(4, dtype=torch.int32, device=DEV)[None], torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    ws, lens, lam = K.alloc_workspace(c, 1, 4, 64), torch.tensor([3], dtype=torch.int32, device=DEV), torch.ones(2, device=DEV)
    calls = (lambda: K.norm_rope_store(c, x, x, x, slots), lambda: K.load(c, slots), lambda: K.load_seqs(c, bt, cu, 3),
             lambda: K.merge_diff(c, ws, 1, 4, lens, 64, lam), lambda: K.prefill_diff(c, q, 2, bt, 1 / 16, lam))
    K.decode_diff(c, q, lens, bt, 64, 1 / 16, ws, lam)
    for call in calls:
        call()
    c.handle = (c.handle[0], 1)
    for call in calls:
        with pytest.raises(ValueError, match="cache is on cuda:1"):
            call()
    c.refresh()
    for call in calls:
        call()
