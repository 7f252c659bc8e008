"""The calls around the cache on the GPU -- norms and rotary positions, alone and
with the store, rows read back, differential heads -- against plain 64-bit
arithmetic, at the sizes, strides, masks and metadata where they can go wrong.

Tolerances count roundings: u = 2^-24 (a half step of fp32) and 2^-8 (of bf16),
relative to the value, each derived where it is used.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from bit_quantized_kv_store_gb300 import synth
from tests.test_gpu_parity import K, bits_u16, make_cache_pair, to_np_in  # noqa: F401

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
LEVELS = (0.12841796875, 0.387939453125, 0.65673828125, 0.9423828125, 1.255859375, 1.6181640625, 2.068359375,
          2.732421875)


def rnd(shape, *key, dtype=torch.float32, scale=1.0):
    return (synth.normal(shape, DEV, "cache_ops", *key) * scale).to(dtype)


def guarded(shape, dtype, fill=777.0):
    """A tensor inside a larger one filled with a sentinel on both sides."""
    n = math.prod(shape)
    buf = torch.full((n + 128,), fill, dtype=dtype, device=DEV)
    return buf, buf[64:64 + n].view(shape)


# ------------------------------------------------------------------ plain forms in 64 bits

def rope64(x, pos, inv_freq, axis, interleaved):
    """(rotated, magnitude of each result's terms): x [n, heads, W] in 64 bits."""
    R = 2 * len(inv_freq)
    f = torch.tensor(inv_freq, dtype=torch.float64, device=x.device)
    ang = pos.double()[torch.tensor(axis, device=x.device)].T * f
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    if interleaved:
        ia, ib = slice(0, R, 2), slice(1, R, 2)
    else:
        ia, ib = slice(0, R // 2), slice(R // 2, R)
    a, b = x[..., ia], x[..., ib]
    y, mag = x.clone(), x.abs()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    m = a.abs() + b.abs()
    mag[..., ia] = m
    mag[..., ib] = m
    return y, mag


def norm64(x, w, eps, offset=0.0):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (w.double() + offset)


def had64(x):
    h = torch.from_numpy(O_hadamard(32)).to(x.device)
    return ((x.reshape(-1, 32) @ h) / math.sqrt(32)).reshape(x.shape)


def O_hadamard(n):
    i = np.arange(n)
    return np.array([[(-1.0) ** bin(a & b).count("1") for b in i] for a in i])


def tq64(x, signs, inverse=False):
    D = x.shape[-1]
    bits = [(int(signs[i // 32]) >> (i % 32)) & 1 for i in range(D)]
    s = torch.tensor([-1.0 if b else 1.0 for b in bits], dtype=torch.float64, device=x.device)
    h = torch.from_numpy(O_hadamard(D)).to(x.device)
    return (x @ h) / math.sqrt(D) * s if inverse else ((x * s) @ h) / math.sqrt(D)


def values64(cache, plane, K):
    """Every row of a plane in the cache's space, in 64 bits."""
    codes = getattr(cache, plane)
    if cache.fmt == K.FMT_BF16:
        return codes.double()
    sc = getattr(cache, plane + "_scale").double()
    if cache.fmt == K.FMT_FP8_ROW:
        return codes.view(torch.float8_e4m3fn).double() * sc[..., None]
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    if cache.fmt == K.FMT_TQ4:
        lev = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)
        return torch.cat((lev, -lev))[c] * sc[..., None]
    return (c - 8).double() * sc.repeat_interleave(32, -1)


def rotated_back64(cache, x, K):
    if cache.fmt == K.FMT_Q4_HAD32:
        return had64(x)
    if cache.fmt == K.FMT_TQ4:
        return tq64(x, cache.signs.tolist(), inverse=True)
    return x


def make_cache(K, fmt, Hk, D, pages, seed=0, ps=16):
    signs = synth.sign_mask(D, "cache_ops", seed) if fmt == K.FMT_TQ4 else None
    return K.Cache(fmt, Hk, D, ps, pages, rope_dim=64 if fmt == K.FMT_FP8_ROW else 0, signs=signs)


def fill_random(cache, K, seed):
    """Random planes: every code, scales of several magnitudes (zero among them)."""
    g = synth.generator(DEV, "fill", seed)
    for name in ("k", "v"):
        t = getattr(cache, name)
        if cache.fmt == K.FMT_BF16:
            t.copy_(torch.randn(t.shape, generator=g, device=DEV).to(torch.bfloat16))
            continue
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
        if cache.fmt == K.FMT_FP8_ROW:
            t[(t & 0x7F) == 0x7F] = 0   # the encoder never writes NaN
        sc = getattr(cache, name + "_scale")
        v = torch.exp(torch.randn(sc.shape, generator=g, device=DEV) * 2)
        v[torch.rand(sc.shape, generator=g, device=DEV) < 0.02] = 0
        sc.copy_(v.to(sc.dtype))


def rope_of(K, rot, interleaved, axes, theta=1e4):
    n = rot // 2
    inv = [theta ** (-2 * i / rot) for i in range(n)]
    ax = [i * axes // n for i in range(n)]
    return K.Rope(inv, axes=ax, interleaved=interleaved), inv, ax


def positions(axes, n, seed):
    g = synth.generator(DEV, "positions", axes, n, seed)
    pos = torch.randint(-1000, 262144, (axes, n), generator=g, device=DEV)
    special = [0, 2 ** 31 - 1, -(2 ** 31), 262143, 1]
    pos.view(-1)[:len(special)] = torch.tensor(special, device=DEV)[:pos.numel()]
    return pos.to(torch.int32)


# ------------------------------------------------------------------ norm and rotary positions

# fp32 roundings in norm_rope, relative to |a| + |b| of the normed pair: the sum of
# squares (at most 10 levels of a tree plus the square itself, halved by the root:
# 6), mean and eps (1), rsqrt (2 ulp = 4), weight + offset (1), the two products
# (2), the rotation's product and fused add (2); cos and sin: the angle's rounding
# to a float (2^-27 of half a turn: 0.4 u) and its cut to 2^-32 of a turn (0.03 u),
# and sincospi's 2 ulp (4 u).  20 and a half; with the table's 2^-63 turns times 2^31
# (a quarter of 2^-30 rad: 4 u, only at positions near 2^31) under 26.
NORM_ROPE_U = 26


@pytest.mark.parametrize("width,rot,interleaved", [(64, 64, 0), (64, 32, 0), (64, 16, 0), (64, 6, 1), (128, 48, 0), (256, 240, 0), (128, 128, 1), (128, 96, 0),
                                                   (256, 64, 0), (256, 256, 0), (256, 96, 0), (256, 250, 1), (64, 2, 1), (512, 16, 0),
                                                   (512, 256, 0), (512, 64, 1)])
@pytest.mark.parametrize("n,heads,axes", [(1, 1, 1), (1, 24, 3), (7, 3, 4), (300, 5, 2), (3001, 9, 3)])
@pytest.mark.parametrize("xt,yt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.float32)])
def test_norm_rope_against_64_bits(K, width, rot, interleaved, n, heads, axes, xt, yt):
    axes = min(axes, rot // 2)
    x = rnd((n, heads, width), width, n, heads, dtype=xt, scale=3.0)
    w = rnd((width,), "w", width, dtype=xt)
    pos = positions(axes, n, width)
    rope, inv, ax = rope_of(K, rot, interleaved, axes)
    pos_arg = pos[0] if axes == 1 else pos
    for norm, off in ((None, 0.0), (K.Norm(w, 1e-6), 0.0), (K.Norm(w, 1e-3, 1.0), 1.0)):
        for rp in (rope, None):
            y = x.double()
            if norm is not None:
                y = norm64(y, w, norm.eps, off)
            mag = y.abs()
            if rp is not None:
                y, mag = rope64(y, pos, inv, ax, interleaved)
            got = K.norm_rope(x, pos_arg if rp is not None else None, rope=rp, norm=norm, dtype=yt)
            assert got.shape == x.shape and got.dtype == yt
            # doubles: the plain form's angle (2^-53 of it), and the table's turns (1 / (2 pi) and its product, 2^-52)
            far = pos.double().abs().max(0).values[:, None, None] * (2.0 ** -51) if rp is not None else 0.0
            tol = (NORM_ROPE_U * U + far) * mag + (HALF_BF16 * (y.abs() + NORM_ROPE_U * U * mag) if yt == torch.bfloat16
                                                    else 0.0)
            err = (got.double() - y).abs()
            assert (err <= tol).all(), f"{(err / tol.clamp(min=1e-300)).max().item()} of the tolerance"
            if rp is None and norm is None and xt == yt:
                assert torch.equal(got, x)


@pytest.mark.parametrize("width", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_rope_strides_and_in_place(K, width, dtype):
    """Slices of a fused projection, heads beside a gate, transposed heads, bases
    and strides off 16 bytes, and in-place calls: the bits of the contiguous call."""
    n, heads = 9, 4
    base = rnd((n, heads, width), "strides", width, dtype=dtype)
    w = rnd((width,), "strides w", width, dtype=dtype)
    norm = K.Norm(w, 1e-6)
    rope, _, _ = rope_of(K, 64, 0, 1)
    pos = positions(1, n, 3)[0]
    want = K.norm_rope(base, pos, rope=rope, norm=norm)
    fused = torch.zeros(n, 3 * heads, width, dtype=dtype, device=DEV)
    fused[:, heads:2 * heads] = base
    gated = torch.zeros(n, heads, 2, width, dtype=dtype, device=DEV)
    gated[:, :, 1] = base
    turned = base.transpose(0, 1).contiguous().transpose(0, 1)
    odd_buf = torch.zeros(n * (heads * width + 3) + 1, dtype=dtype, device=DEV)
    odd = torch.as_strided(odd_buf, (n, heads, width), (heads * width + 3, width, 1), 1)
    odd.copy_(base)
    for x in (fused[:, heads:2 * heads], gated[:, :, 1], turned, odd):
        before = x.clone()
        assert torch.equal(K.norm_rope(x, pos, rope=rope, norm=norm), want)
        assert torch.equal(x, before)
        # written into the same kind of slice, what lies beside it stays
        assert K.norm_rope(x, pos, rope=rope, norm=norm, out=x) is x
        assert torch.equal(x, want)
    assert fused[:, :heads].abs().max() == 0 and fused[:, 2 * heads:].abs().max() == 0
    assert gated[:, :, 0].abs().max() == 0
    buf, out = guarded((n, heads, width), dtype)
    K.norm_rope(base, pos, rope=rope, norm=norm, out=out)
    assert torch.equal(out, want) and (buf[:64] == 777).all() and (buf[-64:] == 777).all()
    # one token of no stride at all: a broadcast input
    one = base[:1].expand(n, heads, width)
    assert torch.equal(K.norm_rope(one, norm=norm), K.norm_rope(one.contiguous(), norm=norm))


@pytest.mark.parametrize("width,heads,rot", [(64, 1, 64), (64, 1, 32), (64, 3, 64), (64, 4, 32), (64, 4, 64),
                                             (128, 1, 128), (128, 1, 96), (128, 2, 32), (128, 2, 64), (128, 2, 128),
                                             (256, 1, 32), (256, 1, 64), (256, 1, 96), (256, 1, 192), (256, 1, 256)])
@pytest.mark.parametrize("interleaved,axes", [(0, 1), (1, 3)])
@pytest.mark.parametrize("xt,yt", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                   (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
def test_norm_rope_few_heads_of_many_tokens(K, width, heads, rot, interleaved, axes, xt, yt):
    """One to four heads of more tokens than the warps that are resident: bit for bit the
    rows that calls of a few tokens give, and nothing beside them."""
    n = 5003
    rope, _, _ = rope_of(K, rot, interleaved, axes)
    pos = positions(axes, n, 7) if axes > 1 else positions(1, n, 7)[0]
    x = rnd((n, heads + 1, width), "few", width, heads, dtype=xt)[:, :heads]
    norm = K.Norm(rnd((width,), "few w", width), offset=1.0) if axes == 1 else None
    buf, out = guarded((n, heads, width), yt)
    K.norm_rope(x, pos, rope=rope, norm=norm, out=out)
    want = [K.norm_rope(x[i:i + 701], pos[..., i:i + 701].contiguous(), rope=rope, norm=norm, dtype=yt)
            for i in range(0, n, 701)]
    assert torch.equal(out, torch.cat(want))
    assert (buf[:64] == 777).all() and (buf[-64:] == 777).all()


@pytest.mark.parametrize("width,heads,rot,interleaved", [(64, 1, 2, 1), (64, 2, 6, 1), (64, 4, 16, 0), (128, 1, 16, 0),
                                                         (128, 2, 126, 1), (256, 1, 250, 1), (256, 1, 240, 0)])
def test_norm_rope_few_heads_other_rotary_widths(K, width, heads, rot, interleaved):
    """Rotary widths that end inside a lane, in place, strided, the last batch part
    empty: bit for bit the rows of calls of a few tokens."""
    n = 9002
    axes = min(3, rot // 2)
    rope, _, _ = rope_of(K, rot, interleaved, axes)
    pos = positions(axes, n, 9) if axes > 1 else positions(1, n, 9)[0]
    base = rnd((n, 3, heads, width), "few odd", width, heads, dtype=torch.bfloat16)
    x = base[:, 1]
    want = torch.cat([K.norm_rope(x[i:i + 501], pos[..., i:i + 501].contiguous(), rope=rope) for i in range(0, n, 501)])
    beside = base.clone()
    K.norm_rope(x, pos, rope=rope, out=x)
    assert torch.equal(x, want)
    assert torch.equal(base[:, 0], beside[:, 0]) and torch.equal(base[:, 2], beside[:, 2])


def test_norm_rope_values_that_are_not_numbers(K):
    """Infinities and NaN stay in their rows (and pairs); what lies past rot_dim stays as it is."""
    x = rnd((4, 2, 256), "nan")
    x[1, 0, 3], x[2, 1, 5], x[3, 0, 200] = math.nan, math.inf, math.inf
    rope, _, _ = rope_of(K, 64, 0, 1)
    pos = torch.arange(1, 5, dtype=torch.int32, device=DEV)
    y = K.norm_rope(x, pos, rope=rope)
    assert torch.isnan(y[1, 0, [3, 35]]).all() and torch.isfinite(y[1, 0]).sum() == 254
    assert (~torch.isfinite(y[2, 1, [5, 37]])).all() and torch.isfinite(y[2, 1]).sum() == 254
    assert torch.equal(y[..., 64:], x[..., 64:])
    z = K.norm_rope(x, norm=K.Norm(torch.ones(256, device=DEV)))
    assert torch.isnan(z[1, 0]).all() and torch.isfinite(z[1, 1]).all() and torch.isfinite(z[0]).all()
    zero = K.norm_rope(torch.zeros(2, 3, 256, device=DEV), norm=K.Norm(torch.ones(256, device=DEV)))
    assert torch.equal(zero, torch.zeros_like(zero))


def test_norm_rope_axis_out_of_range_is_flagged(K):
    rope = K.Rope([1.0] * 32, axes=[0] * 31 + [2])
    rope.desc.num_axes = 2                            # the last pair names a third axis
    rope.handle = (rope.handle[0], 2, rope.handle[2])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = rnd((3, 2, 64), "axis")
    pos = torch.ones(2, 3, dtype=torch.int32, device=DEV)
    y = K.norm_rope(x, pos, rope=rope, status=status)
    assert K.read_status(status) == K.DEV_BAD_INDEX
    bad = torch.isnan(y)
    assert bad[..., [31, 63]].all() and bad.sum() == 2 * 3 * 2


# ------------------------------------------------------------------ with the store

def formats(K, D):
    f = [K.FMT_BF16]
    if D <= 256:
        f += [K.FMT_Q4_HAD32, K.FMT_Q4_0, K.FMT_TQ4]
    return f


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("n,Hq,Hk", [(1, 24, 4), (5, 3, 3), (32, 8, 1), (301, 12, 2), (2501, 15, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_rope_store_equals_its_parts(K, D, n, Hq, Hk, dtype):
    """The same bytes in every plane and the same query bits as norm_rope into fp32,
    store and the rotation, with tokens that are skipped and slots out of range."""
    for fmt in formats(K, D):
        for with_norm, rot, inter, axes in ((True, 64, 0, 3), (False, min(D, 256), 1, 1), (True, 0, 0, 1)):
            qkv = rnd((n, Hq + 2 * Hk, D), D, n, Hq, dtype=dtype, scale=2.0)
            qkv[..., :3] *= 15
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
            if n == 301:
                k[7] = 0          # a zero row: scale 0
                v[7] = 0
            wq, wk = rnd((D,), "wq", D, dtype=dtype), rnd((D,), "wk", D, dtype=dtype)
            qn, kn = (K.Norm(wq, 1e-6), K.Norm(wk, 1e-5, 1.0)) if with_norm else (None, None)
            rope = rope_of(K, rot, inter, axes)[0] if rot else None
            pos = positions(axes, n, D) if rot else None
            pages = n // 16 + 3
            perm = synth.page_permutation(pages, "nrs", n).to(DEV)
            at = torch.arange(n, device=DEV)
            slots = (perm[at // 16] * 16 + at % 16).to(torch.int32)
            if n > 4:
                slots[2], slots[4] = -1, pages * 16 + 5
            a, b = make_cache(K, fmt, Hk, D, pages), make_cache(K, fmt, Hk, D, pages)
            sa, sb = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2))
            got = K.norm_rope_store(a, q, k, v, slots, pos, rope=rope, q_norm=qn, k_norm=kn, status=sa)
            q32 = K.norm_rope(q, pos, rope=rope, norm=qn, dtype=torch.float32)
            k32 = K.norm_rope(k, pos, rope=rope, norm=kn, dtype=torch.float32)
            K.store(b, k32, v.float().contiguous(), slots, status=sb)
            want = q32
            if fmt == K.FMT_Q4_HAD32:
                want = K.rotate_query(q32)
            elif fmt == K.FMT_TQ4:
                want = K.tq4_rotate(b, q32)
            assert torch.equal(got, want)
            for name in ("k", "v", "k_scale", "v_scale"):
                ta, tb = getattr(a, name), getattr(b, name)
                if ta is not None:
                    assert torch.equal(ta.view(torch.uint8), tb.view(torch.uint8)), (fmt, name)
            assert K.read_status(sa) == K.read_status(sb) == (K.DEV_BAD_SLOT if n > 4 else 0)
            # unrotated queries in bf16, and keys and values alone
            c = make_cache(K, fmt, Hk, D, pages)
            qb = torch.empty((n, Hq, D), dtype=torch.bfloat16, device=DEV)
            K.norm_rope_store(c, q, k, v, slots, pos, rope=rope, q_norm=qn, k_norm=kn, q_out=qb, rotate=False)
            assert torch.equal(qb, q32.to(torch.bfloat16))
            d = make_cache(K, fmt, Hk, D, pages)
            assert K.norm_rope_store(d, None, k, v, slots, pos, rope=rope, k_norm=kn) is None
            for other in (c, d):
                assert torch.equal(other.k.view(torch.uint8), a.k.view(torch.uint8))
                assert torch.equal(other.v.view(torch.uint8), a.v.view(torch.uint8))


@pytest.mark.parametrize("n", [3, 2000])
def test_norm_rope_store_mixed_types_and_strides(K, n):
    """Queries, keys and values of different types, strides off 16 bytes and queries
    rotated in place: the bits of contiguous fp32 inputs of the same values."""
    D, Hq, Hk = 128, 6, 2
    q, k, v = rnd((n, Hq, D), "mx q"), rnd((n, Hk, D), "mx k"), rnd((n, Hk, D), "mx v")
    q, k, v = (t.bfloat16().float() for t in (q, k, v))
    pos = positions(2, n, 5)
    rope = rope_of(K, 32, 0, 2)[0]
    qn, kn = K.Norm(rnd((D,), "mx wq"), 1e-6), K.Norm(rnd((D,), "mx wk", dtype=torch.bfloat16), 1e-6)
    slots = torch.arange(n, dtype=torch.int32, device=DEV)

    def run(q, k, v, **kw):
        c = make_cache(K, K.FMT_Q4_HAD32, Hk, D, n // 16 + 1)
        return c, K.norm_rope_store(c, q, k, v, slots, pos, rope=rope, q_norm=qn, k_norm=kn, **kw)

    want, wq = run(q, k, v)
    odd = torch.zeros(n, Hk, D + 1, device=DEV)
    odd[..., 1:] = k
    inplace = q.clone()
    for args, kw in (((q.bfloat16(), k, v.bfloat16()), {}), ((q, odd[..., 1:], v.bfloat16()), {}),
                     ((inplace, k.bfloat16(), v), dict(q_out=inplace)),
                     ((q.bfloat16(), k.bfloat16(), v.bfloat16()), {}),
                     ((q.transpose(0, 1).contiguous().transpose(0, 1), k, v), {})):
        c, got = run(*args, **kw)
        assert torch.equal(got, wq)
        for name in ("k", "v", "k_scale", "v_scale"):
            assert torch.equal(getattr(c, name).view(torch.uint8), getattr(want, name).view(torch.uint8))


@pytest.mark.parametrize("n,Hq", [(1, 128), (1, 3), (40, 16), (700, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_rope_store_latent_rows(K, n, Hq, dtype):
    """Fp8 latent rows: the bytes of norm_rope on either part and the store, and the
    query bits of norm_rope on the rope part beside the latent part as it is."""
    pages = n // 16 + 2
    at = torch.arange(n, device=DEV)
    perm = synth.page_permutation(pages, "latent", n).to(DEV)
    slots = (perm[at // 16] * 16 + at % 16).to(torch.int32)
    if n > 20:
        slots[3], slots[9] = -1, pages * 16
    row = (synth.latent_rows(n, 576, DEV, "latent", n) * 2).to(dtype)
    row[n // 2, 512:] = 0
    wide = torch.zeros(n, 1, 640, dtype=dtype, device=DEV)       # beside other columns of one projection
    wide[:, 0, 32:608] = row
    k = wide[..., 32:608]
    q = rnd((n, Hq, 576), "latent q", n, Hq, dtype=dtype)
    norm = K.Norm(rnd((512,), "latent w", dtype=dtype), 1e-6)
    for inter, axes, with_rope, with_norm in ((1, 1, 1, 1), (0, 2, 1, 1), (1, 1, 0, 1), (0, 1, 1, 0)):
        rope = rope_of(K, 64, inter, axes)[0] if with_rope else None
        pos = positions(axes, n, 7) if with_rope else None
        kn = norm if with_norm else None
        a, b = make_cache(K, K.FMT_FP8_ROW, 1, 512, pages), make_cache(K, K.FMT_FP8_ROW, 1, 512, pages)
        sa, sb = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2))
        got = K.norm_rope_store(a, q, k, None, slots, pos, rope=rope, k_norm=kn, status=sa)
        parts = torch.empty(n, 1, 576, device=DEV)
        K.norm_rope(k[..., :512], norm=kn, out=parts[..., :512])
        K.norm_rope(k[..., 512:], pos, rope=rope, out=parts[..., 512:])
        K.store(b, parts, None, slots, status=sb)
        for name in ("k", "v", "k_scale", "v_scale"):
            assert torch.equal(getattr(a, name).view(torch.uint8), getattr(b, name).view(torch.uint8)), name
        want = q.float().clone()
        K.norm_rope(q[..., 512:], pos, rope=rope, out=want[..., 512:])
        assert torch.equal(got, want)
        assert K.read_status(sa) == K.read_status(sb) == (K.DEV_BAD_SLOT if n > 20 else 0)
        c = make_cache(K, K.FMT_FP8_ROW, 1, 512, pages)
        mine = q.clone()                                          # rotated in place, in its own type
        K.norm_rope_store(c, mine, k.contiguous(), None, slots, pos, rope=rope, k_norm=kn, q_out=mine, rotate=False)
        assert torch.equal(mine, want.to(dtype))
        d = make_cache(K, K.FMT_FP8_ROW, 1, 512, pages)
        assert K.norm_rope_store(d, None, k, None, slots, pos, rope=rope, k_norm=kn) is None
        for other in (c, d):
            assert torch.equal(other.k, a.k) and torch.equal(other.v, a.v)


def test_norm_rope_store_queries_of_padding_tokens(K):
    """A token without a slot still has its queries; n = 0 writes nothing."""
    a = make_cache(K, K.FMT_Q4_HAD32, 2, 256, 2)
    q, k = rnd((4, 4, 256), "pad q"), rnd((4, 2, 256), "pad k")
    slots = torch.full((4,), -1, dtype=torch.int32, device=DEV)
    assert torch.equal(K.norm_rope_store(a, q, k, k, slots), K.rotate_query(q))
    assert a.k.abs().max() == 0 and a.v.abs().max() == 0
    K.norm_rope_store(a, q[:0], k[:0], k[:0], slots[:0])


# ------------------------------------------------------------------ rows read back

# A value is fl(sum * fl(scale * c)) with the sum exact, c the rounded 1 / sqrt(n)
# (1 u), its product (1 u) and the last product (1 u).
LOAD_U = 3


def check_values(got, want):
    tol = LOAD_U * 1.01 * U * want.abs()
    if got.dtype == torch.bfloat16:
        tol = tol + HALF_BF16 * (want.abs() + tol)
    # below the smallest normal number the steps are absolute
    err = (got.double() - want).abs()
    assert (err <= tol + 2.0 ** -133).all(), f"{(err / (tol + 1e-300)).max().item()} of the tolerance"


@pytest.mark.parametrize("fmt,D,Hk", [(f, D, Hk) for f, D in (
    ("Q4_HAD32", 32), ("Q4_HAD32", 64), ("Q4_HAD32", 128), ("Q4_HAD32", 256), ("Q4_0", 32), ("Q4_0", 256), ("TQ4", 64),
    ("TQ4", 128), ("TQ4", 256), ("BF16", 96), ("BF16", 256)) for Hk in (1, 3, 8)] + [("FP8_ROW", 512, 1), ("FP8_ROW", 32, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_load_against_64_bits(K, fmt, D, Hk, dtype):
    f = getattr(K, "FMT_" + fmt)
    fp8 = f == K.FMT_FP8_ROW
    cache = make_cache(K, f, Hk, D, 9)
    fill_random(cache, K, D * 10 + Hk)
    n = 133
    g = synth.generator("cpu", "load", fmt, D, Hk)
    slots = torch.randint(0, 9 * 16, (n,), generator=g).to(torch.int32)
    slots[5], slots[6], slots[100] = slots[4], -1, 9 * 16
    slots = slots.to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    width = D + cache.rope if fp8 else D
    for rb in ((0, 1) if fmt in ("Q4_HAD32", "TQ4") else (0,)):
        outs = [guarded((n, Hk, width), dtype) for _ in range(1 if fp8 else 2)]
        K.load(cache, slots, k=outs[0][1], v=None if fp8 else outs[1][1], rotate_back=rb, status=status)
        assert K.read_status(status) == K.DEV_BAD_SLOT
        row = slots.long().clamp(0, 9 * 16 - 1)
        want = []
        for plane in ("k", "v"):
            x = values64(cache, plane, K)[row // 16, :, row % 16]
            want.append(rotated_back64(cache, x, K) if rb else x)
        if fp8:
            want = [torch.cat(want, -1)]
        for (buf, got), w in zip(outs, want):
            ok = torch.ones(n, dtype=torch.bool, device=DEV)
            ok[[6, 100]] = False
            check_values(got[ok], w[ok])
            assert (got[6] == 777).all() and torch.isnan(got[100]).all()
            assert (buf[:64] == 777).all() and (buf[-64:] == 777).all()
    if not fp8:   # one plane alone; strided and unaligned outputs
        k, none = K.load(cache, slots[:4], k=torch.empty(4, Hk, D, dtype=dtype, device=DEV))
        assert none is None
        both, v = K.load(cache, slots[:4], dtype=dtype)
        assert torch.equal(k, both)
        wide = torch.full((4, 2 * Hk, D + 1), 5.0, dtype=dtype, device=DEV)
        K.load(cache, slots[:4], k=wide[:, :Hk, 1:], v=wide[:, Hk:, 1:])
        assert torch.equal(wide[:, :Hk, 1:], both) and torch.equal(wide[:, Hk:, 1:], v) and (wide[..., 0] == 5).all()


@pytest.mark.parametrize("fmt,D", [("Q4_HAD32", 32), ("Q4_HAD32", 64), ("Q4_HAD32", 128), ("Q4_HAD32", 256),
                                   ("TQ4", 64), ("TQ4", 128), ("TQ4", 256), ("Q4_0", 32), ("Q4_0", 256)])
@pytest.mark.parametrize("Hk", [1, 2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_load_few_heads(K, fmt, D, Hk, dtype):
    """One and two heads in more rows than one round of the warps, among them positions
    that keep what they hold, positions without a row, and views with gaps: against the
    same rows loaded a few at a time, bit for bit."""
    n, pages = 40037, 2600
    cache = make_cache(K, getattr(K, "FMT_" + fmt), Hk, D, pages)
    fill_random(cache, K, D + Hk)
    g = torch.Generator(device=DEV).manual_seed(D + Hk)
    slots = torch.randperm(pages * 16, generator=g, device=DEV)[:n].to(torch.int32)
    skip, bad = [0, 3, 32, 17000, n - 1], [1, 33, 20001, n - 2]
    broken = slots.clone()
    broken[skip], broken[bad] = -1, pages * 16
    bufs = [torch.full((n, 2 * Hk, D), 777.0, dtype=dtype, device=DEV) for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.load(cache, broken, k=bufs[0][:, :Hk], v=bufs[1][:, Hk:], status=status)
    assert K.read_status(status) == K.DEV_BAD_SLOT
    parts = [K.load(cache, slots[i:i + 997], dtype=dtype) for i in range(0, n, 997)]
    want = [torch.cat([p[j] for p in parts]) for j in range(2)]
    for w in want:
        w[skip], w[bad] = 777.0, float("nan")
    assert torch.equal(bufs[0][:, :Hk].nan_to_num(nan=-5.0), want[0].nan_to_num(nan=-5.0))
    assert torch.equal(bufs[1][:, Hk:].nan_to_num(nan=-5.0), want[1].nan_to_num(nan=-5.0))
    assert (bufs[0][:, Hk:] == 777).all() and (bufs[1][:, :Hk] == 777).all()


@pytest.mark.parametrize("fmt,D,Hk", [("Q4_HAD32", 32, 3), ("Q4_HAD32", 64, 5), ("Q4_HAD32", 128, 2),
                                      ("Q4_HAD32", 256, 4), ("Q4_HAD32", 256, 9), ("TQ4", 64, 1), ("TQ4", 128, 6),
                                      ("TQ4", 256, 4), ("Q4_0", 256, 8), ("BF16", 128, 3), ("FP8_ROW", 512, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_load_many_rows(K, fmt, D, Hk, dtype):
    """Enough rows that every warp takes several: by slot and by table, against the
    same rows loaded a few at a time."""
    f = getattr(K, "FMT_" + fmt)
    n, pages = 23003, 1500
    cache = make_cache(K, f, Hk, D, pages)
    fill_random(cache, K, D + Hk)
    perm = synth.page_permutation(pages, "many", fmt).to(torch.int32).to(DEV)
    lens = [0, 9001, 5, 13997, 0]
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    bt = torch.stack([perm[i * 100:i * 100 + 900] for i in range(5)])
    starts = torch.tensor([0, 7, 3, 0, 1], dtype=torch.int32, device=DEV)
    at = torch.cat([torch.arange(m, device=DEV) + int(starts[i]) for i, m in enumerate(lens)])
    seq = torch.repeat_interleave(torch.arange(5, device=DEV), torch.tensor(lens, device=DEV))
    slots = (bt.long()[seq, at // 16] * 16 + at % 16).to(torch.int32)
    k, v = K.load_seqs(cache, bt, cu, n, starts=starts, dtype=dtype)
    k2, v2 = K.load(cache, slots, dtype=dtype)
    parts = [K.load(cache, slots[i:i + 4001], dtype=dtype) for i in range(0, n, 4001)]
    small = [K.load(cache, slots[i:i + 3], dtype=dtype) for i in (0, 11000, n - 3)]
    assert torch.equal(k, k2) and torch.equal(k, torch.cat([p[0] for p in parts]))
    for i, p in zip((0, 11000, n - 3), small):
        assert torch.equal(k[i:i + 3], p[0])
    if v is not None:
        assert torch.equal(v, v2) and torch.equal(v, torch.cat([p[1] for p in parts]))
        # into strided outputs, and one plane alone
        wide = torch.full((n, Hk, 2, D), 5.0, dtype=dtype, device=DEV)
        K.load(cache, slots, k=wide[:, :, 0])
        assert torch.equal(wide[:, :, 0], k) and (wide[:, :, 1] == 5).all()
        K.load(cache, slots, v=wide[:, :, 1])
        assert torch.equal(wide[:, :, 0], k) and torch.equal(wide[:, :, 1], v)


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "TQ4", "BF16", "FP8_ROW", "Q4_0"])
def test_load_seqs_ragged(K, fmt):
    """Packed runs of several sequences, empty ones among them, equal the load of
    their slots; rows past the last run stay; bad pages and positions come out NaN."""
    f = getattr(K, "FMT_" + fmt)
    fp8 = f == K.FMT_FP8_ROW
    Hk, D, pages = (1, 512, 40) if fp8 else (2, 256, 40)
    cache = make_cache(K, f, Hk, D, pages)
    fill_random(cache, K, 5)
    lens = [0, 17, 0, 0, 1, 40, 16, 0]
    starts = [3, 5, 0, 90, 31, 0, 16, 2]
    B, mp = len(lens), 6
    perm = synth.page_permutation(pages, "seqs").to(torch.int32)
    bt = torch.stack([perm[i * 4:i * 4 + mp] for i in range(B)])
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    n = int(cu[-1])
    slots = []
    for b in range(B):
        for i in range(lens[b]):
            pos = starts[b] + i
            slots.append(int(bt[b, pos // 16]) * 16 + pos % 16)
    slots = torch.tensor(slots, dtype=torch.int32, device=DEV)
    want, want_v = K.load(cache, slots)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (cache, bt.to(DEV), cu.to(DEV))
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    k, v = K.load_seqs(*args, n, starts=st, status=status)
    assert torch.equal(k, want) and (fp8 or torch.equal(v, want_v)) and K.read_status(status) == 0
    # five rows past the last run, and a first run that starts at row 2
    out = torch.full((n + 5, Hk, want.shape[-1]), 3.0, dtype=torch.bfloat16, device=DEV)
    K.load_seqs(args[0], args[1], args[2], n + 5, starts=st, k=out)
    assert torch.equal(out[:n], want) and (out[n:] == 3).all()
    out.fill_(3)
    K.load_seqs(args[0], args[1], args[2] + 2, n + 5, starts=st, k=out)
    assert torch.equal(out[2:n + 2], want) and (out[:2] == 3).all() and (out[n + 2:] == 3).all()
    # without starts: from position 0
    k0, _ = K.load_seqs(*args, n)
    s0 = torch.tensor([int(bt[b, i // 16]) * 16 + i % 16 for b in range(B) for i in range(lens[b])], dtype=torch.int32,
                      device=DEV)
    assert torch.equal(k0, K.load(cache, s0)[0])
    # a page outside the pool, and positions before the first and behind the last
    bad = bt.clone()
    bad[1, 0] = pages
    bad[5, 2] = -3
    k1, _ = K.load_seqs(cache, bad.to(DEV), args[2], n, starts=st, status=status)
    assert K.read_status(status) == K.DEV_BAD_PAGE
    nan = torch.isnan(k1.float()).flatten(1).all(1).cpu()
    hit = torch.zeros(n, dtype=torch.bool)
    hit[:11] = True                                      # sequence 1: positions 5 .. 15
    hit[17 + 1 + 32:17 + 1 + 40] = True                  # sequence 5: positions 32 .. 39
    assert torch.equal(nan, hit)
    assert torch.equal(k1[~hit.to(DEV)], want[~hit.to(DEV)])
    status.zero_()
    far = st.clone()
    far[1], far[4] = -2, mp * 16
    k2, _ = K.load_seqs(*args, n, starts=far, status=status)
    assert K.read_status(status) == K.DEV_BAD_LENGTH
    assert torch.isnan(k2[:2].float()).all() and torch.isfinite(k2[2:17].float()).all()
    assert torch.isnan(k2[17].float()).all()
    assert torch.equal(k2[18:], want[18:])
    # no sequences, no rows
    e, _ = K.load_seqs(cache, bt[:0].to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV), 3,
                       k=torch.full((3, Hk, want.shape[-1]), 2.0, dtype=torch.bfloat16, device=DEV))
    assert (e == 2).all()
    K.load_seqs(*args, 0)


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "TQ4", "BF16"])
@pytest.mark.parametrize("ps", [48, 256])
def test_other_page_sizes(K, fmt, ps):
    """Pages of 48 and 256 slots: stored and loaded as in a cache of 16-slot pages."""
    f, n, Hk, D = getattr(K, "FMT_" + fmt), 700, 3, 128
    pages = n // ps + 3
    a, b = make_cache(K, f, Hk, D, pages, ps=ps), make_cache(K, f, Hk, D, n // 16 + 1)
    q, k, v = rnd((n, 6, D), "ps q"), rnd((n, Hk, D), "ps k"), rnd((n, Hk, D), "ps v")
    perm = synth.page_permutation(pages, "ps", ps).to(DEV)
    at = torch.arange(n, device=DEV)
    slots = (perm[at // ps] * ps + at % ps).to(torch.int32)
    qa = K.norm_rope_store(a, q, k, v, slots)
    qb = K.norm_rope_store(b, q, k, v, at.to(torch.int32))
    assert torch.equal(qa, qb)
    want = K.load(b, at.to(torch.int32))
    cu = torch.tensor([0, 300, n], dtype=torch.int32, device=DEV)
    st = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    bt = perm.to(torch.int32).expand(2, -1).contiguous()
    for got in (K.load(a, slots), K.load_seqs(a, bt, cu, n, starts=st)):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_load_seqs_of_many_sequences(K):
    """A thousand sequences, most of them of no or one position."""
    cache = make_cache(K, K.FMT_Q4_HAD32, 2, 64, 60)
    fill_random(cache, K, 9)
    lens = synth.ragged_lengths(1000, 0, 3, "many seqs")
    lens[::7] = 0
    lens[500] = 200
    bt = torch.stack([synth.page_permutation(60, "ms", i)[:13] for i in range(1000)]).to(torch.int32).to(DEV)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(lens, 0)]).to(torch.int32).to(DEV)
    n = int(cu[-1])
    seq = torch.repeat_interleave(torch.arange(1000), lens).to(DEV)
    at = torch.arange(n, device=DEV) - cu.long()[seq]
    slots = (bt.long()[seq, at // 16] * 16 + at % 16).to(torch.int32)
    got, want = K.load_seqs(cache, bt, cu, n), K.load(cache, slots)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_more_than_2_31_elements(K):
    """Activations and outputs of more than 2^31 elements: their last rows are those
    of a call on them alone."""
    n, H, W = 351003, 24, 256
    x = torch.zeros(n, H, W, dtype=torch.bfloat16, device=DEV)
    x[-5:] = rnd((5, H, W), "2^31", dtype=torch.bfloat16)
    norm = K.Norm(rnd((W,), "2^31 w"), 1e-6)
    rope, _, _ = rope_of(K, 64, 0, 1)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    y = K.norm_rope(x, pos, rope=rope, norm=norm)
    assert torch.equal(y[-5:], K.norm_rope(x[-5:], pos[-5:], rope=rope, norm=norm))
    assert y[:-5].abs().max() == 0
    del x
    z = torch.zeros(n, H, W, device=DEV)
    z[-5:] = y[-5:].float()
    lam = torch.rand(n, H // 2, device=DEV)
    d = K.diff_heads(z, lam, norm=norm, dtype=torch.bfloat16)
    assert torch.equal(d[-5:], K.diff_heads(z[-5:], lam[-5:], norm=norm, dtype=torch.bfloat16))
    assert d[:-5].abs().max() == 0
    del y, z, d
    cache = make_cache(K, K.FMT_Q4_HAD32, 8, 256, 2)
    fill_random(cache, K, 4)
    m = 1050007
    slots = (torch.arange(m, device=DEV) % 32).to(torch.int32)
    k, v = K.load(cache, slots)
    small = K.load(cache, slots[:32])
    last = slots[-7:].long()
    assert torch.equal(k[-7:], small[0][last]) and torch.equal(v[-7:], small[1][last])
    torch.cuda.empty_cache()


def test_rows_past_two_gigabytes(K):
    """A pool whose planes pass 2^31 bytes: rows at its end store and load."""
    pages = (1 << 31) // (16 * 128) + 70
    cache = make_cache(K, K.FMT_Q4_HAD32, 1, 256, pages)
    k, v = rnd((33, 1, 256), "far k"), rnd((33, 1, 256), "far v")
    slots = torch.arange(pages * 16 - 33, pages * 16, dtype=torch.int32, device=DEV)
    q = K.norm_rope_store(cache, None, k, v, slots)
    assert q is None
    small = make_cache(K, K.FMT_Q4_HAD32, 1, 256, 3)
    K.store(small, k, v, torch.arange(33, dtype=torch.int32, device=DEV))
    a, b = K.load(cache, slots), K.load(small, torch.arange(33, dtype=torch.int32, device=DEV))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    bt = torch.arange(pages - 3, pages, dtype=torch.int32, device=DEV)[None]
    cu = torch.tensor([0, 33], dtype=torch.int32, device=DEV)
    st = torch.tensor([15], dtype=torch.int32, device=DEV)
    c = K.load_seqs(cache, bt, cu, 33, starts=st)
    assert torch.equal(c[0], b[0]) and torch.equal(c[1], b[1])


# ------------------------------------------------------------------ differential heads

def diff64(o, lam, norm, offset, scale, K):
    """The difference, norm and scale of merged heads o [rows, Hq, W] in 64 bits."""
    y = o[:, 0::2] - lam.double()[..., None] * o[:, 1::2]
    if norm is not None:
        y = norm64(y, norm.weight, norm.eps, offset)
    return y * scale


@pytest.mark.parametrize("width,Hq", [(64, 2), (128, 6), (256, 24), (512, 4)])
@pytest.mark.parametrize("rows", [1, 77])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_diff_heads_against_64_bits(K, width, Hq, rows, dtype):
    x = rnd((rows, Hq, width), "dh", rows, width)
    w = rnd((width,), "dh w", width)
    lams = (torch.sigmoid(rnd((rows, Hq // 2), "lam", rows)), torch.rand(Hq // 2, device=DEV),
            torch.sigmoid(rnd((rows, Hq), "lam wide", rows))[:, :Hq // 2])
    for lam in lams:
        for norm, off in ((None, 0.0), (K.Norm(w, 1e-5), 0.0), (K.Norm(w.bfloat16(), 1e-5, 1.0), 1.0)):
            want = diff64(x.double(), lam, norm, off, 0.7, K)
            got = K.diff_heads(x, lam, norm=norm, out_scale=0.7, dtype=dtype)
            # y: one rounding of a - l b; norm: the sum of squares 6, mean and eps 1, rsqrt 4, weight 1, products 2;
            # scale (its own rounding and the product): 2.  Relative to |a| + l |b| over the rms where normed.
            mag = x.double()[:, 0::2].abs() + lam.double()[..., None] * x.double()[:, 1::2].abs()
            if norm is not None:
                y = diff64(x.double(), lam, None, 0.0, 1.0, K)
                r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + norm.eps)
                # the error of y moves the mean, too: by at most its rms relative to y's
                shift = r * torch.sqrt((mag * mag).mean(-1, keepdim=True))
                mag = (mag * r + y.abs() * r * shift) * (norm.weight.double() + off).abs()
            tol = 17 * U * mag * 0.7
            if dtype == torch.bfloat16:
                tol = tol + HALF_BF16 * (want.abs() + tol)
            err = (got.double() - want).abs()
            assert (err <= tol).all(), (err / tol.clamp(min=1e-300)).max().item()
    buf, out = guarded((rows, Hq // 2, width), dtype)
    K.diff_heads(x, lams[0], out=out)
    assert (buf[:64] == 777).all() and (buf[-64:] == 777).all()
    shifted = torch.empty(rows * Hq * width + 1, device=DEV)[1:].view(rows, Hq, width)   # off 16 bytes
    shifted.copy_(x)
    assert torch.equal(K.diff_heads(shifted, lams[0]), K.diff_heads(x, lams[0]))


def diff_problem(K, fmt, lens, Hk=4, group=6, seed=0, extra=0):
    """A filled cache, queries, tables and the workspace of a decode over `lens`."""
    T = max(max(lens), 1) + extra
    B, mp = len(lens), -(-T // 16)
    need = [-(-max(t, 1) // 16) for t in lens]
    cache = make_cache(K, fmt, Hk, 256, sum(need) + 1, seed)
    fill_random(cache, K, seed)
    for name in ("k", "v"):
        if fmt != K.FMT_BF16:   # scales near one another: scores of a few units
            sc = getattr(cache, name + "_scale")
            sc.copy_((0.3 + 0.05 * torch.rand(sc.shape, device=DEV)) * (2.0 if fmt == K.FMT_TQ4 else 1.0))
    perm = synth.page_permutation(sum(need) + 1, "diff", seed).to(torch.int32)
    bt = torch.zeros(B, mp, dtype=torch.int32)
    at = 0
    for b in range(B):
        bt[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    q = rnd((B, Hk * group, 256), "diff q", seed)
    ws = K.alloc_workspace(cache, B, Hk * group, T)
    return cache, q, torch.tensor(lens, dtype=torch.int32, device=DEV), bt.to(DEV), T, ws


def check_merge_diff(K, cache, q, lens, bt, T, ws, lam, dtype=torch.float32, sel=None):
    """decode_diff against the difference of decode()'s heads in 64 bits: the same
    partials, so only the difference, the rotation back and the norm round apart."""
    B, Hq = q.shape[:2]
    heads = K.decode(cache, q, lens, bt, T, 1 / 16, ws, sel=sel)
    o = heads.double()
    w = rnd((256,), "md w")
    # rotation back: 5 (TQ4: 8) stages and a product on either side, of values up to
    # sqrt(32) (16) times the largest; and the difference
    st, top = (9, 16) if cache.fmt == K.FMT_TQ4 else (7, math.sqrt(32)) if cache.fmt == K.FMT_Q4_HAD32 else (1, 1)
    big = o.abs().amax(-1, keepdim=True)
    spread = 2 * st * U * top * (big[:, 0::2] + lam.double()[..., None] * big[:, 1::2]) if lam.dim() == 2 else \
        2 * st * U * top * (big[:, 0::2] + lam.double()[None, :, None] * big[:, 1::2])
    for norm, scale in ((None, 1.0), (K.Norm(w, 1e-5), 0.8)):
        got = K.decode_diff(cache, q, lens, bt, T, 1 / 16, ws, lam, norm=norm, out_scale=scale, dtype=dtype, sel=sel)
        assert got.shape == (B, Hq // 2, 256) and got.dtype == dtype
        want = diff64(o, lam, norm, 0.0, scale, K)
        tol = spread * scale
        if norm is not None:
            y = diff64(o, lam, None, 0.0, 1.0, K)
            r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + norm.eps)
            # an error e of every y: e r, and through the rms at most |y| r (e r); the norm's own 14 roundings
            tol = ((spread * r) * (1 + y.abs() * r) + 14 * U * y.abs() * r) * w.double().abs() * scale
        tol = tol + 2 * U * want.abs()
        if dtype == torch.bfloat16:
            tol = tol + HALF_BF16 * (want.abs() + tol)
        err = (got.double() - want).abs()
        ok = torch.isfinite(want)
        assert torch.equal(torch.isfinite(got), ok)
        assert (err[ok] <= (tol + torch.zeros_like(err))[ok] + 1e-30).all(), \
            (err[ok] / (tol + torch.zeros_like(err))[ok].clamp(min=1e-300)).max().item()
    return heads


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "Q4_0", "TQ4", "BF16"])
@pytest.mark.parametrize("lens", [[1], [513], [0, 1, 2, 511, 512, 513, 1025, 0], [4097, 30], [70000], [140000]])
def test_decode_diff_is_the_difference_of_the_heads(K, fmt, lens):
    f = getattr(K, "FMT_" + fmt)
    p = diff_problem(K, f, lens)
    lam = torch.sigmoid(rnd((len(lens), 12), "lam", len(lens)))
    check_merge_diff(K, *p, lam)
    check_merge_diff(K, *p, lam[0].contiguous(), dtype=torch.bfloat16)
    for b, t in enumerate(lens):
        if t == 0:
            out = K.decode_diff(p[0], p[1], p[2], p[3], p[4], 1 / 16, p[5], lam, norm=K.Norm(torch.ones(256, device=DEV)))
            assert (out[b] == 0).all()


@pytest.mark.parametrize("Hk,group", [(1, 2), (2, 8), (8, 4)])
def test_decode_diff_head_layouts_and_batches(K, Hk, group):
    """Groups of two to eight, a batch of more than four waves of merge CTAs, lengths
    out of range (NaN rows, the others unaffected), one lambda row for all."""
    lens = [int(x) for x in synth.ragged_lengths(100, 1, 700, "dd", Hk)]
    p = diff_problem(K, K.FMT_Q4_HAD32, lens, Hk=Hk, group=group, seed=Hk)
    lam = torch.rand(100, Hk * group, device=DEV)[:, :Hk * group // 2]     # rows wider than the heads
    check_merge_diff(K, *p, lam)
    cache, q, sl, bt, T, ws = p
    good = K.decode_diff(cache, q, sl, bt, T, 1 / 16, ws, lam)
    for norm in (None, K.Norm(torch.ones(256, device=DEV))):
        want = K.decode_diff(cache, q, sl, bt, T, 1 / 16, ws, lam, norm=norm)
        bad = sl.clone()
        bad[3], bad[50] = T + 1, -1
        out = K.decode_diff(cache, q, bad, bt, T, 1 / 16, ws, lam, norm=norm)
        assert torch.isnan(out[[3, 50]]).all()
        keep = [i for i in range(100) if i not in (3, 50)]
        assert torch.equal(out[keep], want[keep])
    # alone or in the batch: the same bits (in the batch one CTA takes a head; alone with a long table, eight)
    one = K.decode_diff(cache, q[7:8].contiguous(), sl[7:8].contiguous(), bt[7:8].contiguous(), T, 1 / 16,
                        K.alloc_workspace(cache, 1, Hk * group, T), lam[7:8])
    assert torch.equal(one[0], good[7])


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "TQ4"])
@pytest.mark.parametrize("longest", [60000, 140000, 600000])
def test_both_arrangements_of_the_merge_agree(K, fmt, longest):
    """One CTA for a head (many heads, or few partitions) and eight (a long
    sequence's few heads) give the same bits, with and without the norm."""
    lens = [longest, 3, 513, longest - 700] + [900] * 9
    cache, q, sl, bt, T, ws = diff_problem(K, getattr(K, "FMT_" + fmt), lens)
    lam = torch.rand(len(lens), 12, device=DEV)
    for norm in (None, K.Norm(torch.rand(256, device=DEV), 1e-5)):
        many = K.decode_diff(cache, q, sl, bt, T, 1 / 16, ws, lam, norm=norm)
        for b in (0, 1, 2, 3):
            few = K.decode_diff(cache, q[b:b + 1].contiguous(), sl[b:b + 1].contiguous(), bt[b:b + 1].contiguous(), T,
                                1 / 16, K.alloc_workspace(cache, 1, 24, T), lam[b:b + 1], norm=norm)
            assert torch.equal(few[0], many[b])


def test_merge_diff_of_a_window_and_a_gather(K):
    cache, q, sl, bt, T, ws = diff_problem(K, K.FMT_Q4_HAD32, [2000])
    lam = torch.rand(12, device=DEV)
    sel = synth.distinct_sorted(700, 2000, "sel").to(torch.int32)[None].to(DEV)
    wsel = K.alloc_workspace(cache, 1, 24, T, n_sel=700)
    check_merge_diff(K, cache, q, sl, bt, T, wsel, lam, sel=sel)
    rows = torch.tensor([1990, 1991, 1992], dtype=torch.int32, device=DEV)
    qw = rnd((3, 24, 256), "window")
    w3 = K.alloc_workspace(cache, 3, 24, T)
    K.decode_window(cache, K.rotate_query(qw), rows, bt, T, 1 / 16, w3)
    got = K.merge_diff(cache, w3, 3, 24, rows, T, lam)
    want = K.decode_diff(cache, qw, rows, bt.expand(3, -1).contiguous(), T, 1 / 16, K.alloc_workspace(cache, 3, 24, T), lam)
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "TQ4"])
def test_decode_diff_against_the_oracle(K, fmt):
    """Both maps from the oracle's fp64 attention over the same cache; each map is
    within the decode's 2e-3 of its largest output."""
    T, Hk, Hq, ps = 1500, 2, 8, 16
    g, o = make_cache_pair(K, getattr(K, "FMT_" + fmt), Hk, 256, ps, 94)
    k, v = (synth.heavy_tailed((T, Hk, 256), "cpu", "diff oracle", t) for t in "kv")
    slots = np.arange(T, dtype=np.int32)
    K.store(g, k.to(DEV), v.to(DEV), torch.from_numpy(slots).to(DEV))
    O.store(o, to_np_in(k), to_np_in(v), slots)
    q = synth.normal((1, Hq, 256), "cpu", "diff oracle q")
    bt = np.arange(94, dtype=np.int32)[None]
    lam = torch.tensor([0.2, 0.5, 0.8, 1.3])
    ref = np.asarray(O.decode(o, q.numpy(), [T], bt, 1 / 16), np.float64).reshape(Hq, 256)
    want = ref[0::2] - lam.double().numpy()[:, None] * ref[1::2]
    got = K.decode_diff(g, q.to(DEV), torch.tensor([T], dtype=torch.int32, device=DEV), torch.from_numpy(bt).to(DEV), T,
                        1 / 16, K.alloc_workspace(g, 1, Hq, T), lam.to(DEV))[0].cpu().numpy()
    big = np.abs(ref).max()
    assert (np.abs(got - want) <= 2e-3 * big * (1 + lam.numpy()[:, None])).all()


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "Q4_0"])
@pytest.mark.parametrize("T0,n,Hk,group", [(0, 1, 4, 6), (0, 70, 1, 2), (100, 37, 4, 6), (1500, 16, 2, 8), (2000, 130, 1, 4),
                                           (63, 300, 8, 6), (4000, 1000, 4, 6)])
def test_prefill_diff_against_64_bits(K, fmt, T0, n, Hk, group):
    """Chunks of one row to many, cut into one to 32 ranges of keys, against 64-bit
    attention over the same rows; each map within the prefill's 2e-3 of its largest output."""
    Hq = Hk * group
    pages = (T0 + n + 15) // 16 + 2
    cache = make_cache(K, getattr(K, "FMT_" + fmt), Hk, 256, pages)
    k, v = rnd((T0 + n, Hk, 256), "pd k", n), rnd((T0 + n, Hk, 256), "pd v", n)
    perm = synth.page_permutation(pages, "pd", n).to(torch.int32).to(DEV)
    at = torch.arange(T0 + n, device=DEV)
    slots = (perm.long()[at // 16] * 16 + at % 16).to(torch.int32)
    K.store(cache, k, v, slots)
    q = rnd((n, Hq, 256), "pd q", n, dtype=torch.bfloat16, scale=2.0)
    lam = torch.rand(n, Hq // 2, device=DEV)
    w = rnd((256,), "pd w")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    rk, rv = (x.double() for x in K.load(cache, slots, dtype=torch.float32))
    rows = sorted({0, n - 1, n // 2, n // 3, min(n - 1, 21), min(n - 1, 64)})
    ref = []
    for i in rows:
        p = torch.softmax(torch.einsum("hd,thd->ht", q[i].double(), rk[:T0 + i + 1].repeat_interleave(group, 1)) / 16, -1)
        ref.append(torch.einsum("ht,thd->hd", p, rv[:T0 + i + 1].repeat_interleave(group, 1)))
    ref = torch.stack(ref)
    for norm, scale in ((None, 1.0), (K.Norm(w, 1e-5), 0.8)):
        got = K.prefill_diff(cache, q, T0, perm, 1 / 16, lam, norm=norm, out_scale=scale, status=status)
        assert got.shape == (n, Hq // 2, 256) and torch.isfinite(got).all()
        y = diff64(ref, lam[rows], None, 0.0, 1.0, K)
        want = diff64(ref, lam[rows], norm, 0.0, scale, K)
        e = 2e-3 * ref.abs().amax((1, 2), keepdim=True) * (1 + lam[rows].double()[..., None])
        tol = e * scale
        if norm is not None:
            r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + norm.eps)
            tol = tol * w.double().abs() * r * (1 + y.abs() * r)
        assert ((got[rows].double() - want).abs() <= tol).all()
        # a workspace of the caller's, bf16, one lambda row for all
        ws = torch.empty(K.lib().kvq_prefill_diff_workspace_size(cache.ref, n, Hq, T0), dtype=torch.uint8, device=DEV)
        one = K.prefill_diff(cache, q, T0, perm, 1 / 16, lam[0].contiguous(), norm=norm, out_scale=scale, workspace=ws)
        bf = K.prefill_diff(cache, q, T0, perm, 1 / 16, lam[:1].expand(n, -1).contiguous(), norm=norm, out_scale=scale,
                            dtype=torch.bfloat16)
        assert torch.equal(one.bfloat16(), bf)
    assert K.read_status(status) == 0
    if n > 1:
        with pytest.raises(K.KvqError):
            K.prefill_diff(cache, q, T0, perm, 1 / 16, lam, workspace=ws[:-1].clone())


def test_prefill_diff_bad_page(K):
    """Rows that attend a page outside the pool come out NaN, rows before it do not."""
    cache = make_cache(K, K.FMT_Q4_HAD32, 4, 256, 200)
    fill_random(cache, K, 3)
    n, T0 = 30, 3000
    bt = torch.arange(200, dtype=torch.int32, device=DEV)
    bt[40] = 4000
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = rnd((n, 24, 256), "bp q", scale=0.1)
    out = K.prefill_diff(cache, q, T0, bt, 1 / 16, torch.rand(12, device=DEV), status=status)
    assert torch.isnan(out).all() and K.read_status(status) == K.DEV_BAD_PAGE


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "Q4_0"])
@pytest.mark.parametrize("n,Hq", [(1, 8), (45, 24), (200, 12)])
def test_prefill_attn_places_of_its_tensors(K, fmt, n, Hq):
    """Outputs and queries off a 32-byte boundary: the same bits, nothing beside them; an
    output off its 16 bytes is refused."""
    T0 = 100
    cache = make_cache(K, getattr(K, "FMT_" + fmt), 4, 256, 40)
    fill_random(cache, K, n)
    bt = torch.arange(40, dtype=torch.int32, device=DEV)
    q = rnd((n, Hq, 256), "place q", n, scale=0.3)
    want = K.prefill_attn(cache, q, T0, bt, 1 / 16)
    for shift in (4, 8, 12):
        buf = torch.full((n * Hq * 256 + 64,), 777.0, device=DEV)
        out = buf[shift:shift + q.numel()].view(n, Hq, 256)
        moved = torch.empty(q.numel() + 64, device=DEV)[shift // 4:shift // 4 + q.numel()].view(n, Hq, 256)
        moved.copy_(q)
        K.prefill_attn(cache, moved, T0, bt, 1 / 16, out=out)
        assert torch.equal(out, want)
        assert (buf[:shift] == 777).all() and (buf[shift + q.numel():] == 777).all()
    off = torch.empty(q.numel() + 64, device=DEV)[1:1 + q.numel()].view(n, Hq, 256)
    with pytest.raises(K.KvqError):
        K.prefill_attn(cache, q, T0, bt, 1 / 16, out=off)


# ------------------------------------------------------------------ a run of them together

def serve_step(K, s):
    """One layer's decode step as a model makes it: projections to the cache, differential attention over it."""
    q = K.norm_rope_store(s["cache"], s["q"], s["k"], s["v"], s["slots"], s["pos"], rope=s["rope"], q_norm=s["qn"],
                          k_norm=s["kn"], q_out=s["q_out"], stream=s.get("stream"))
    K.decode_attn(s["cache"], q, s["lens"], s["bt"], s["T"], 1 / 16, s["ws"], stream=s.get("stream"))
    return K.merge_diff(s["cache"], s["ws"], s["q"].shape[0], 24, s["lens"], s["T"], s["lam"], norm=s["on"], out_scale=0.8,
                        out=s["out"], stream=s.get("stream"))


def serve_state(K, fmt, B=3, seed=0):
    lens = [700, 33, 1500][:B]
    cache, _, sl, bt, T, ws = diff_problem(K, fmt, lens, seed=seed)
    qkv = rnd((B, 32, 256), "serve", seed, dtype=torch.bfloat16)
    last = sl.long() - 1
    slots = (bt.long()[torch.arange(B, device=DEV), last // 16] * 16 + last % 16).to(torch.int32)
    rope, inv, ax = rope_of(K, 64, 0, 3)
    return dict(cache=cache, q=qkv[:, :24], k=qkv[:, 24:28], v=qkv[:, 28:], slots=slots, pos=positions(3, B, seed),
                rope=rope, inv=inv, ax=ax, qn=K.Norm(rnd((256,), "sq"), 1e-6), kn=K.Norm(rnd((256,), "sk"), 1e-6),
                on=K.Norm(rnd((256,), "so"), 1e-5), lens=sl, bt=bt, T=T, ws=ws, lam=torch.rand(B, 12, device=DEV),
                q_out=torch.empty(B, 24, 256, device=DEV), out=torch.empty(B, 12, 256, device=DEV))


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "TQ4", "BF16"])
def test_decode_step_of_a_model_end_to_end(K, fmt):
    """norm + rope + store, read back, and differential attention over it, against
    64-bit attention over the rows read back."""
    s = serve_state(K, getattr(K, "FMT_" + fmt))
    out = serve_step(K, s).clone()
    cache, B = s["cache"], 3
    k64, _ = rope64(norm64(s["k"].double(), s["kn"].weight, 1e-6), s["pos"], s["inv"], s["ax"], 0)
    new_k, new_v = K.load(cache, s["slots"], dtype=torch.float32)
    # the stored rows: within a step of the code (amax / 8 of the rotated group, sqrt(32) of them at most add up
    # in a value; the codebook's widest cell is 0.67 of the row's rms, its outermost values clip)
    for got, ref in ((new_k, k64), (new_v, s["v"].double())):
        rel = (got.double() - ref).norm() / ref.norm()
        assert rel < (0.004 if fmt == "BF16" else 0.2)
    q64, _ = rope64(norm64(s["q"].double(), s["qn"].weight, 1e-6), s["pos"], s["inv"], s["ax"], 0)
    cu = torch.tensor([0] + list(np.cumsum(s["lens"].tolist())), dtype=torch.int32, device=DEV)
    rk, rv = K.load_seqs(cache, s["bt"], cu, int(cu[-1]), dtype=torch.float32)
    for b in range(B):
        k = rk[cu[b]:cu[b + 1]].double().repeat_interleave(6, 1)
        v = rv[cu[b]:cu[b + 1]].double().repeat_interleave(6, 1)
        p = torch.softmax(torch.einsum("hd,thd->ht", q64[b], k) / 16, -1)
        o = torch.einsum("ht,thd->hd", p, v)[None]
        y = diff64(o, s["lam"][b:b + 1], None, 0.0, 1.0, K)
        r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-5)
        want = diff64(o, s["lam"][b:b + 1], s["on"], 0.0, 0.8, K)
        # each map is within the decode's 2e-3 of its largest value
        e = 2e-3 * o.abs().max() * (1 + s["lam"][b].double().max())
        tol = 0.8 * s["on"].weight.double().abs() * e * r * (1 + y.abs() * r)
        assert ((out[b].double() - want[0]).abs() <= tol[0]).all()


@pytest.mark.parametrize("fmt", ["Q4_HAD32", "TQ4"])
def test_two_captured_steps_with_their_own_workspaces(K, fmt):
    """The step captured twice on a side stream, replayed with new inputs in place:
    the bits of eager calls."""
    f = getattr(K, "FMT_" + fmt)
    a, b = serve_state(K, f, seed=1), serve_state(K, f, seed=2)
    graphs = []
    side = torch.cuda.Stream()
    for s in (a, b):
        s["stream"] = side
        serve_step(K, s)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            serve_step(K, s)
        graphs.append(g)
    for s, seed in ((a, 11), (b, 12)):
        for name in ("q", "k", "v"):
            s[name].copy_(rnd(s[name].shape, "new", name, seed))
        s["lam"].copy_(torch.rand_like(s["lam"]))
        s["out"].zero_()
    torch.cuda.synchronize()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for s in (a, b):
        got = s["out"].clone()
        s.pop("stream")
        assert torch.equal(serve_step(K, s), got)


def test_binding_refusals_on_the_gpu(K):
    c = make_cache(K, K.FMT_Q4_HAD32, 2, 256, 2)
    x = rnd((4, 2, 256), "r")
    rope = K.Rope([1.0, 0.1], axes=[0, 1])
    i32 = torch.zeros(4, dtype=torch.int32, device=DEV)
    lam = torch.zeros(1, device=DEV)
    for call in (lambda: K.norm_rope(x[..., ::2]), lambda: K.norm_rope(x[0]),
                 lambda: K.norm_rope(x, rope=rope), lambda: K.norm_rope(x, i32, rope=rope),
                 lambda: K.norm_rope(x, norm=K.Norm(torch.ones(128, device=DEV))),
                 lambda: K.norm_rope(x, out=x[:3]),
                 lambda: K.norm_rope_store(c, x, x, x, i32[:3]),
                 lambda: K.norm_rope_store(c, x, x[:, :1], x, i32),
                 lambda: K.norm_rope_store(c, None, x, x, i32, q_out=x),
                 lambda: K.load(c, i32, k=x[:3]),
                 lambda: K.load(c, torch.zeros(8, dtype=torch.int32, device=DEV)[::2]),
                 lambda: K.load_seqs(c, i32, i32[:2], 4),
                 lambda: K.diff_heads(x, lam[:, None].expand(4, 1)[:3]),
                 lambda: K.diff_heads(x, lam, out=torch.empty(4, 2, 256, device=DEV))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: K.norm_rope(x.half()), lambda: K.norm_rope(x, i32.long(), rope=K.Rope([1.0] * 8)),
                 lambda: K.load(c, i32.long()), lambda: K.diff_heads(x, lam.double()),
                 lambda: K.diff_heads(x.bfloat16(), lam)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: K.norm_rope(x[..., :96]), lambda: K.load(c, i32, rotate_back=2),
                 lambda: K.norm_rope_store(c, x, x, x, i32, q_out=x.bfloat16())):
        with pytest.raises(K.KvqError):
            call()
