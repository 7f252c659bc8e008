"""Cases of the operators around the quantized cache: the head norms and rotary
positions on the way into it, the rows read back out of it, and differential
attention over it.

Each case is one call (or the calls that belong together) of a program that
serves a model from a paged cache; `run` computes it either in plain tensor
operations (own = False) or through the library (own = True).
"""
import math

import torch

own = False

PAGE = 16
# Lloyd-Max magnitudes of N(0, 1) for 16 levels, as the TQ4 rows hold them
TQ4_LEVELS = (0.12841796875, 0.387939453125, 0.65673828125, 0.9423828125, 1.255859375, 1.6181640625, 2.068359375,
              2.732421875)
FORMATS = {"q4_had32": 0, "bf16": 1, "fp8_row": 2, "q4_0": 3, "tq4": 4}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the rope part of an absorbed latent query, one new token: rotation only, written beside the latent part
        dict(name="rope_latent_query_1", op="norm_rope", tokens=1, heads=128, width=64, rot=64, interleaved=True, axes=1,
             norm=False, x="f32", y="f32", pad=512),
        # the queries of an image-and-text chunk for the prefill kernel: norm and three-axis partial rotation
        dict(name="norm_rope_q_4099_axes3", op="norm_rope", tokens=4099, heads=24, width=256, rot=64, interleaved=False,
             axes=3, norm=True, x="bf16", y="bf16", pad=0),
        # one decode token of one sequence: queries into the cache's space, its K and V rows stored
        dict(name="store_token_1", op="norm_rope_store", fmt="q4_had32", tokens=1, q_heads=24, kv_heads=4, width=256,
             rot=64, interleaved=False, axes=1, norm=True, x="bf16"),
        # a decode batch of 32 sequences, codebook rows
        dict(name="store_batch_32_tq4", op="norm_rope_store", fmt="tq4", tokens=32, q_heads=24, kv_heads=4, width=256,
             rot=256, interleaved=False, axes=1, norm=True, x="bf16"),
        # a prompt chunk of 4096 tokens, three position axes
        dict(name="store_chunk_4096_axes3", op="norm_rope_store", fmt="q4_had32", tokens=4096, q_heads=24, kv_heads=4,
             width=256, rot=64, interleaved=False, axes=3, norm=True, x="bf16"),
        # an odd chunk of fp32 activations with 128-wide heads and interleaved pairs
        dict(name="store_chunk_1001_d128_f32", op="norm_rope_store", fmt="q4_had32", tokens=1001, q_heads=32, kv_heads=8,
             width=128, rot=128, interleaved=True, axes=1, norm=True, x="f32"),
        # 2048 selected latent rows for a dense kernel
        dict(name="load_selected_fp8_2048", op="load", fmt="fp8_row", tokens=2048, seqs=1, kv_heads=1, width=512,
             by="slots", y="bf16"),
        # eight ragged sequences' prefixes of codebook rows in fp32
        dict(name="load_ragged_8_tq4_f32", op="load", fmt="tq4", tokens=20011, seqs=8, kv_heads=4, width=256,
             by="tables", y="f32"),
        # a whole 262144-token sequence read back (export, or a dense kernel over it)
        dict(name="load_262144", op="load", fmt="q4_had32", tokens=262144, seqs=1, kv_heads=4, width=256, by="tables",
             y="bf16"),
        # one decode query of one 32K sequence
        dict(name="diff_decode_32769", op="decode_diff", fmt="q4_had32", seqs=1, longest=32769, q_heads=24, kv_heads=4,
             norm=True),
        # a ragged decode batch of 32 sequences over codebook rows
        dict(name="diff_decode_batch_32_tq4", op="decode_diff", fmt="tq4", seqs=32, longest=8000, q_heads=24, kv_heads=4,
             norm=False),
        # a prompt chunk at depth 4096
        dict(name="diff_prefill_1024_at_4096", op="prefill_diff", fmt="q4_had32", tokens=1024, start=4096, q_heads=24,
             kv_heads=4, norm=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _rot(rng, width):
    return rng.choice([r for r in (32, 64, 96, 128, 192, 256, 512) if r <= min(width, 256) and r % (width // 16) == 0])


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_store", "load", "decode_diff", "prefill_diff"])
    if op == "norm_rope":
        width = rng.choice([64, 128, 256, 512])
        heads = rng.choice([1, 3, 4, 8, 16, 24, 32, 64, 128])
        tokens = _log(rng, 1, min(16384, 2 ** 25 // (heads * width)))
        return dict(op=op, tokens=tokens, heads=heads, width=width, rot=_rot(rng, width),
                    interleaved=rng.random() < 0.4, axes=rng.choice([1, 1, 3]), norm=rng.random() < 0.7,
                    x=rng.choice(["bf16", "bf16", "f32"]), y=rng.choice(["bf16", "f32"]),
                    pad=rng.choice([0, 0, width, 512]))
    if op == "norm_rope_store":
        fmt = rng.choice(["q4_had32", "q4_had32", "tq4", "bf16", "q4_0"])
        width = rng.choice([64, 128, 256, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        return dict(op=op, fmt=fmt, tokens=_log(rng, 1, 150 if fmt == "q4_0" else 4096),
                    q_heads=kv_heads * rng.choice([1, 3, 4, 6, 8]), kv_heads=kv_heads, width=width,
                    rot=_rot(rng, width), interleaved=rng.random() < 0.4, axes=rng.choice([1, 1, 3]),
                    norm=rng.random() < 0.8, x=rng.choice(["bf16", "bf16", "f32"]))
    if op == "load":
        fmt = rng.choice(["q4_had32", "tq4", "bf16", "q4_0", "fp8_row"])
        fp8 = fmt == "fp8_row"
        seqs = rng.choice([1, 1, 2, 5, 8, 16, 33])
        return dict(op=op, fmt=fmt, tokens=_log(rng, max(1, seqs), 65536), seqs=seqs,
                    kv_heads=1 if fp8 else rng.choice([1, 2, 4, 8]), width=512 if fp8 else rng.choice([64, 128, 256]),
                    by=rng.choice(["slots", "tables"]), y=rng.choice(["bf16", "bf16", "f32"]))
    if op == "decode_diff":
        seqs = rng.choice([1, 1, 2, 7, 16, 32, 64])
        kv_heads = rng.choice([1, 2, 4, 8])
        return dict(op=op, fmt=rng.choice(["q4_had32", "q4_had32", "q4_0", "tq4", "bf16"]), seqs=seqs,
                    longest=_log(rng, 100, min(65537, 2 ** 20 // (seqs * kv_heads))),
                    q_heads=kv_heads * rng.choice([2, 4, 6, 8]), kv_heads=kv_heads, norm=rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 4])
    return dict(op=op, fmt=rng.choice(["q4_had32", "q4_0"]), tokens=_log(rng, 16, 1024), start=_log(rng, 1, 4096),
                q_heads=kv_heads * rng.choice([2, 4, 6]), kv_heads=kv_heads, norm=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int64)


def _rope_inputs(g, case):
    """Frequencies of the pairs, their axes, and positions [axes, tokens]: a run of text positions, on three axes
    with image patches' (time, height, width) offsets from them."""
    n, pairs = case["tokens"], case["rot"] // 2
    inv_freq = 1e6 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    axis = (torch.arange(pairs) * case["axes"] // pairs).to(torch.int64)
    first = _ints(g, 0, 262144 - n, 1)
    pos = (first + torch.arange(n, device="cuda")).expand(case["axes"], n)
    if case["axes"] > 1:
        pos = pos + _ints(g, 0, 64, case["axes"], n)
    return dict(inv_freq=inv_freq.cuda(), axis=axis.cuda(), pos=pos.to(torch.int32).contiguous())


def _own_rope(kvq, s, case):
    return kvq.Rope(s["inv_freq"].tolist(), axes=s["axis"].tolist(), interleaved=case["interleaved"])


def _norm_weight(g, width, dtype):
    return (1 + 0.2 * _randn(g, width)).to(dtype)


def _pages(g, count):
    return torch.randperm(count, generator=g, device="cuda").to(torch.int32)


def _planes(g, case, pages):
    """The planes of a filled pool: normal-like codes and one magnitude per scale."""
    fmt, D, rows = case["fmt"], case["width"], (pages, case["kv_heads"], PAGE)
    if fmt == "bf16":
        return {p: _randn(g, *rows, D).to(torch.bfloat16) for p in ("k", "v")}
    if fmt == "fp8_row":
        out = {}
        for p, w in (("k", D), ("v", 64)):
            x = _randn(g, *rows, w)
            out[p] = (x * (448 / x.abs().amax(-1, keepdim=True))).to(torch.float8_e4m3fn).view(torch.uint8)
            out[p + "_scale"] = torch.exp(_randn(g, *rows)) * (4.0 / 448)
        return out
    out = {}
    for p in ("k", "v"):
        if fmt == "tq4":
            code = _ints(g, 0, 256, *rows, D // 2).to(torch.uint8)
            scale = torch.exp(0.3 * _randn(g, *rows))
        else:
            c = (_randn(g, *rows, D // 2, 2) * 3.4).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
            code = c[..., 0] | (c[..., 1] << 4)
            del c
            scale = torch.exp(0.3 * _randn(g, *rows, D // 32)) * 0.3
        out[p], out[p + "_scale"] = code, scale.to(torch.float16)
    return out


def _signs(g, case):
    """Random signs of a row as the words of a bit mask (int32 [width / 32])."""
    return _ints(g, -2 ** 31, 2 ** 31, case["width"] // 32).to(torch.int32)


def _own_cache(kvq, s, case, pages):
    fmt = FORMATS[case["fmt"]]
    cache = kvq.Cache(fmt, case["kv_heads"], case["width"], PAGE, pages, rope_dim=64 if case["fmt"] == "fp8_row" else 0,
                      signs=s["signs"] if case["fmt"] == "tq4" else None)
    if "planes" in s:
        for name, t in s["planes"].items():
            setattr(cache, name, t)
        cache.refresh()
    return cache


def _lengths(g, seqs, longest):
    """Ragged lengths up to `longest`, which the first sequence has."""
    n = (_rand(g, seqs) * 0.9 + 0.1) * longest
    n[0] = longest
    return n.round().to(torch.int32).clamp_(min=1)


def _lambda(g, rows, heads):
    return torch.sigmoid(_randn(g, rows, heads) - 0.5)


def prepare(case, seed):
    g = _gen(seed)
    case = dict(case) | ({"width": 256} if case["op"] in ("decode_diff", "prefill_diff") else {})
    s = {"case": case}
    if own:
        from bit_quantized_kv_store_gb300 import kvq
        s["kvq"] = kvq
    op = case["op"]
    if op in ("norm_rope", "norm_rope_store"):
        s |= _rope_inputs(g, case)
    if op == "norm_rope":
        n, H, W, pad = case["tokens"], case["heads"], case["width"], case["pad"]
        # rows beside `pad` other values each (a gate, or a latent part)
        s["x"] = (_randn(g, n, H, pad + W) * 2).to(DTYPES[case["x"]])[..., pad:]
        s["weight"] = _norm_weight(g, W, DTYPES[case["x"]]) if case["norm"] else None
        if own:
            s["rope"] = _own_rope(s["kvq"], s, case)
            s["norm"] = s["kvq"].Norm(s["weight"], 1e-6) if case["norm"] else None
    elif op == "norm_rope_store":
        n, Hq, Hk, D = case["tokens"], case["q_heads"], case["kv_heads"], case["width"]
        dt = DTYPES[case["x"]]
        qkv = _randn(g, n, Hq + 2 * Hk, D)  # one fused projection
        qkv = qkv * torch.where(_rand(g, Hq + 2 * Hk, D) < 0.05, 3.0, 1.0)  # some channels are larger
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        s["q_weight"] = _norm_weight(g, D, dt) if case["norm"] else None
        s["k_weight"] = _norm_weight(g, D, dt) if case["norm"] else None
        pages = 2 * (-(-n // PAGE)) + 1
        at = torch.arange(n, device="cuda")
        s["slots"] = (_pages(g, pages)[at // PAGE] * PAGE + (at % PAGE)).to(torch.int32)
        s["signs"] = _signs(g, case) if case["fmt"] == "tq4" else None
        s["pages"] = pages
        if own:
            s["cache"] = _own_cache(s["kvq"], s, case, pages)
            s["rope"] = _own_rope(s["kvq"], s, case)
            s["q_norm"] = s["kvq"].Norm(s["q_weight"], 1e-6) if case["norm"] else None
            s["k_norm"] = s["kvq"].Norm(s["k_weight"], 1e-6) if case["norm"] else None
    else:
        if op == "load":
            B, n = case["seqs"], case["tokens"]
            cuts = torch.sort(torch.randperm(n - 1, generator=g, device="cuda")[:B - 1] + 1).values if B > 1 else None
            cu = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
            cu[B] = n
            if B > 1:
                cu[1:B] = cuts
            s["cu"] = cu.to(torch.int32)
            s["starts"] = _ints(g, 0, 100, B).to(torch.int32)
            longest = n + 100
            lens = (cu[1:] - cu[:-1] + 100).to(torch.int32)
        elif op == "decode_diff":
            B, longest = case["seqs"], case["longest"]
            lens = _lengths(g, B, longest)
        else:
            B, longest = 1, case["start"] + case["tokens"]
            lens = torch.tensor([longest], dtype=torch.int32, device="cuda")
        s["lens"], s["longest"] = lens, longest
        # every sequence has the pages it needs, from anywhere in the pool; the rest of its table is page 0
        need = (lens.long() + PAGE - 1) // PAGE
        wide = -(-longest // PAGE) if B == 1 else int(need.max())
        first = torch.cumsum(need, 0) - need
        total = int(need.sum())
        s["pages"] = total + 3
        order = _pages(g, total + 3)
        col = torch.arange(wide, device="cuda")
        idx = (first[:, None] + col).clamp_(max=total)
        s["tables"] = torch.where(col < need[:, None], order[idx], 0).to(torch.int32).contiguous()
        s["planes"] = _planes(g, case, s["pages"])
        s["signs"] = _signs(g, case) if case["fmt"] == "tq4" else None
        if op == "load":
            if case["by"] == "slots":  # rows from anywhere, each once
                s["slots"] = torch.randperm(s["pages"] * PAGE, generator=g, device="cuda")[:n].to(torch.int32)
        else:
            rows = B if op == "decode_diff" else case["tokens"]
            s["q"] = (_randn(g, rows, case["q_heads"], 256) * 2).to(torch.bfloat16)
            s["lam"] = _lambda(g, rows, case["q_heads"] // 2)
            s["weight"] = _norm_weight(g, 256, torch.float32) if case["norm"] else None
        if own:
            s["cache"] = _own_cache(s["kvq"], s, case, s["pages"])
            if op == "decode_diff":
                s["ws"] = s["kvq"].alloc_workspace(s["cache"], B, case["q_heads"], longest)
            if op != "load":
                s["norm"] = s["kvq"].Norm(s["weight"], 1e-5) if case["norm"] else None
    _plain_tables(s, case)
    return s


# ------------------------------------------------------------------ plain forms

def _hadamard(n):
    h = torch.ones(1, 1, device="cuda")
    two = torch.tensor([[1.0, 1.0], [1.0, -1.0]], device="cuda")
    while h.shape[0] < n:
        h = torch.kron(h, two)
    return h


def _sign_vector(words, D):
    bit = torch.arange(D, device=words.device)
    return 1.0 - 2.0 * ((words.long()[bit // 32] >> (bit % 32)) & 1).float()


def _plain_tables(s, case):
    """The matrices and levels that a program of plain operations keeps for a cache."""
    n = {"q4_had32": 32, "tq4": case["width"]}.get(case.get("fmt"))
    if n:
        s["had"] = _hadamard(n)
    if case.get("fmt") == "tq4":
        s["sign"] = _sign_vector(s["signs"], n)
        lev = torch.tensor(TQ4_LEVELS, device="cuda")
        s["levels"], s["mids"] = torch.cat((lev, -lev)), (lev[:-1] + lev[1:]) / 2


def _into_space(x, s, fmt):
    """Rows into the cache's space (fp32)."""
    if fmt == "q4_had32":
        return ((x.reshape(-1, 32) @ s["had"]) * (1 / math.sqrt(32))).reshape(x.shape)
    if fmt == "tq4":
        return (x * s["sign"]) @ s["had"] * (1 / math.sqrt(x.shape[-1]))
    return x


def _out_of_space(x, s, fmt):
    if fmt == "tq4":
        return x @ s["had"] * (1 / math.sqrt(x.shape[-1])) * s["sign"]
    return _into_space(x, s, fmt)


def _normed(x, weight, eps):
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()


def _roped(x, s, case):
    angle = s["pos"].double()[s["axis"]].T * s["inv_freq"]  # [tokens, pairs]; far positions need the 64 bits
    c, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    R = case["rot"]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if case["interleaved"] else (x[..., :R // 2], x[..., R // 2:R])
    ra, rb = a * c - b * sn, b * c + a * sn
    y = torch.stack((ra, rb), -1).flatten(-2) if case["interleaved"] else torch.cat((ra, rb), -1)
    return torch.cat((y, x[..., R:]), -1)


def _pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8)


def _quantize(y, s, fmt):
    """Codes (packed) and scales of rows in the cache's space."""
    if fmt == "bf16":
        return y.to(torch.bfloat16), None
    if fmt == "tq4":
        scale = torch.sqrt(y.square().mean(-1)).clamp(max=65504).to(torch.float16)
        sf = scale.float()[..., None]
        v = torch.where(sf > 0, y / sf, 0.0)
        mag = (v.abs()[..., None] > s["mids"]).sum(-1)
        return _pack((mag + 8 * (v < 0)).to(torch.int32)), scale
    grp = y.reshape(*y.shape[:-1], -1, 32)
    scale = (grp.abs().amax(-1) / 8).clamp(max=65504).to(torch.float16)
    sf = scale.float()[..., None]
    q = torch.where(sf > 0, torch.round(grp / sf), 0.0).clamp(-8, 7) + 8
    return _pack(q.reshape(y.shape).to(torch.int32)), scale


def _values(codes, scale, s, fmt):
    """Rows as the values they stand for, in the cache's space (fp32)."""
    if fmt == "bf16":
        return codes.float()
    if fmt == "fp8_row":
        return codes.view(torch.float8_e4m3fn).float() * scale[..., None]
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int32)
    if fmt == "tq4":
        return s["levels"][c] * scale.float()[..., None]
    return ((c - 8).float().reshape(*c.shape[:-1], -1, 32) * scale.float()[..., None]).reshape(c.shape)


def _plain_store(s, case):
    fmt, D, Hk, n = case["fmt"], case["width"], case["kv_heads"], case["tokens"]
    q = _into_space(_roped(_normed(s["q"].float(), s["q_weight"], 1e-6), s, case), s, fmt)
    out = []
    page, off = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    for x in (_roped(_normed(s["k"].float(), s["k_weight"], 1e-6), s, case), s["v"].float()):
        code, scale = _quantize(_into_space(x, s, fmt), s, fmt)
        plane = torch.zeros(s["pages"], Hk, PAGE, code.shape[-1], dtype=code.dtype, device="cuda")
        plane[page, :, off] = code
        if scale is not None:
            scales = torch.zeros(s["pages"], Hk, PAGE, *scale.shape[2:], dtype=scale.dtype, device="cuda")
            scales[page, :, off] = scale
            scale = scales[page, :, off]
        out.append(_out_of_space(_values(plane[page, :, off], scale, s, fmt), s, fmt).to(torch.bfloat16))
    return {"q": q, "k": out[0], "v": out[1]}


def _where(s, case):
    """Page and offset of every row that a load returns."""
    if case["by"] == "slots":
        return s["slots"].long() // PAGE, s["slots"].long() % PAGE
    t = torch.arange(case["tokens"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    p = t - s["cu"].long()[b] + s["starts"].long()[b]
    return s["tables"].long()[b, p // PAGE], p % PAGE


def _plain_load(s, case):
    page, off = _where(s, case)
    fmt, pl, dt = case["fmt"], s["planes"], DTYPES[case["y"]]
    got = []
    for p in ("k", "v"):
        scale = None if fmt == "bf16" else pl[p + "_scale"][page, :, off]
        x = _values(pl[p][page, :, off], scale, s, fmt)
        got.append(_out_of_space(x, s, fmt).to(dt))
    return {"k": torch.cat(got, -1)} if fmt == "fp8_row" else {"k": got[0], "v": got[1]}


def _seq_rows(s, case, p):
    """[sequences, heads, positions, width] of plane p, in the cache's space."""
    page = s["tables"].long()
    fmt, pl = case["fmt"], s["planes"]
    x = _values(pl[p][page], None if fmt == "bf16" else pl[p + "_scale"][page], s, fmt)
    B, n, Hk, ps, D = x.shape
    return x.transpose(1, 2).reshape(B, Hk, n * ps, D)


def _difference(o, s):
    y = o[..., 0::2, :] - s["lam"][..., None] * o[..., 1::2, :]
    return (_normed(y, s["weight"], 1e-5) * 0.8).to(torch.bfloat16)


def _plain_diff(s, case):
    fmt, Hk = case["fmt"], case["kv_heads"]
    K, V = _seq_rows(s, case, "k"), _seq_rows(s, case, "v")
    q = _into_space(s["q"].float(), s, fmt)
    rows, Hq, D = q.shape
    if case["op"] == "decode_diff":  # one query row for each sequence
        q = q.reshape(rows, Hk, Hq // Hk, D)
        keep = (torch.arange(K.shape[2], device="cuda") < s["lens"][:, None])[:, None, None]
    else:  # the rows of one sequence; row i ends at position start + i
        q = q.reshape(1, rows, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(1, Hk, Hq // Hk * rows, D)
        keep = torch.arange(K.shape[2], device="cuda") <= case["start"] + torch.arange(rows, device="cuda")[:, None]
        keep = keep.repeat(Hq // Hk, 1)[None, None]
    sc = torch.where(keep, q @ K.transpose(-1, -2) * D ** -0.5, -math.inf)
    e = torch.exp(sc - sc.amax(-1, keepdim=True))
    o = (e @ V) / e.sum(-1, keepdim=True)
    if case["op"] == "decode_diff":
        o = o.reshape(rows, Hq, D)
    else:
        o = o.reshape(Hk, Hq // Hk, rows, D).permute(2, 0, 1, 3).reshape(rows, Hq, D)
    return _difference(_out_of_space(o, s, fmt), s)


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "norm_rope":
            return _roped(_normed(s["x"].float(), s["weight"], 1e-6), s, case).to(DTYPES[case["y"]])
        if op == "norm_rope_store":
            return _plain_store(s, case)
        return _plain_load(s, case) if op == "load" else _plain_diff(s, case)
    kvq = s["kvq"]
    if op == "norm_rope":
        return kvq.norm_rope(s["x"], s["pos"], rope=s["rope"], norm=s["norm"], dtype=DTYPES[case["y"]])
    if op == "norm_rope_store":
        q = kvq.norm_rope_store(s["cache"], s["q"], s["k"], s["v"], s["slots"], s["pos"], rope=s["rope"],
                                q_norm=s["q_norm"], k_norm=s["k_norm"])
        k, v = kvq.load(s["cache"], s["slots"])
        return {"q": q, "k": k, "v": v}
    if op == "load":
        dt = DTYPES[case["y"]]
        if case["by"] == "slots":
            k, v = kvq.load(s["cache"], s["slots"], dtype=dt)
        else:
            k, v = kvq.load_seqs(s["cache"], s["tables"], s["cu"], case["tokens"], starts=s["starts"], dtype=dt)
        return {"k": k} if v is None else {"k": k, "v": v}
    if op == "decode_diff":
        return kvq.decode_diff(s["cache"], s["q"], s["lens"], s["tables"], s["longest"], 256 ** -0.5, s["ws"], s["lam"],
                               norm=s["norm"], out_scale=0.8, dtype=torch.bfloat16)
    return kvq.prefill_diff(s["cache"], s["q"], case["start"], s["tables"], 256 ** -0.5, s["lam"], norm=s["norm"],
                            out_scale=0.8, dtype=torch.bfloat16)


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(fmt, D):
    return {"q4_had32": D // 2 + D // 16, "q4_0": D // 2 + D // 16, "tq4": D // 2 + 2, "bf16": 2 * D,
            "fp8_row": 0}[fmt]


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op == "norm_rope":
        n = case["tokens"] * case["heads"] * case["width"]
        return {"bytes": n * (size[case["x"]] + size[case["y"]]), "flops": n * 8}
    if op == "norm_rope_store":
        # activations in, rotated queries out, rows written, then read back as bf16
        D, n = case["width"], case["tokens"]
        kv = 2 * n * case["kv_heads"]
        q = n * case["q_heads"] * D
        return {"bytes": q * (size[case["x"]] + 4) + kv * (D * size[case["x"]] + 2 * _row_bytes(case["fmt"], D) + 2 * D),
                "flops": (q + kv * D) * 16}
    if op == "load":
        n, D = case["tokens"], case["width"]
        if case["fmt"] == "fp8_row":
            return {"bytes": n * (D + 64 + 8 + (D + 64) * size[case["y"]]), "flops": n * (D + 64)}
        rows = 2 * n * case["kv_heads"]
        return {"bytes": rows * (_row_bytes(case["fmt"], D) + D * size[case["y"]]), "flops": rows * D * 6}
    if op == "decode_diff":
        # lengths are spread over 0.1 .. 1 of the longest, which one sequence has
        keys = int(case["longest"] * (1 + 0.55 * (case["seqs"] - 1)))
        rows = case["seqs"] * case["q_heads"] * 256
        return {"bytes": keys * 2 * case["kv_heads"] * _row_bytes(case["fmt"], 256) + rows * 2 + rows,
                "flops": 4 * keys * case["q_heads"] * 256}
    n, T = case["tokens"], case["start"] + case["tokens"]
    pairs = n * case["start"] + n * (n + 1) // 2
    return {"bytes": T * 2 * case["kv_heads"] * _row_bytes(case["fmt"], 256) + n * case["q_heads"] * 256 * 3,
            "flops": 4 * pairs * case["q_heads"] * 256}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _wht64(x):
    """Orthonormal Walsh-Hadamard transform of the last dimension (64 bits), by its definition's matrix."""
    n = x.shape[-1]
    i = torch.arange(n, device=x.device)
    both = i[:, None] & i[None, :]
    odd = sum((both >> b) & 1 for b in range(n.bit_length())) & 1
    return torch.matmul(x, (1.0 - 2.0 * odd.double()) / n ** 0.5)


def _turn64(x, s, case, forward):
    """The cache's rotation of rows in 64 bits, and back."""
    if case["fmt"] == "q4_had32":
        return torch.cat([_wht64(g) for g in x.split(32, -1)], -1)
    if case["fmt"] == "tq4":
        words = [int(w) for w in s["signs"]]
        sign = torch.tensor([-1.0 if (words[i // 32] >> (i % 32)) & 1 else 1.0 for i in range(x.shape[-1])],
                            dtype=torch.float64, device=x.device)
        return _wht64(x * sign) if forward else _wht64(x) * sign
    return x


def _enter64(x, s, case, weight):
    """Norm and rotary positions by complex multiplication, in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x * weight.double() / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)
    R, x = case["rot"], x.clone()
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                       s["pos"].double().index_select(0, s["axis"]).t().contiguous() * s["inv_freq"])[:, None, :]
    half = slice(0, R, 2), slice(1, R, 2)
    if not case["interleaved"]:
        half = slice(0, R // 2), slice(R // 2, R)
    z = torch.complex(x[..., half[0]].contiguous(), x[..., half[1]].contiguous()) * turn
    x[..., half[0]], x[..., half[1]] = z.real, z.imag
    return x


def _stored64(y, case):
    """Rows in the cache's space -> the values they are stored as."""
    if case["fmt"] == "bf16":
        return y
    if case["fmt"] == "tq4":
        sc = ((y * y).sum(-1, keepdim=True) / y.shape[-1]).sqrt().half().double()
        lev = torch.tensor(TQ4_LEVELS, dtype=torch.float64, device="cuda")
        near = torch.bucketize((y / sc).abs(), (lev[1:] + lev[:-1]) * 0.5)
        return torch.copysign(lev[near], y) * sc
    got = []
    for g in y.split(32, -1):
        sc = (g.abs().max(-1, keepdim=True).values * 0.125).half().double()
        got.append(torch.where(sc > 0, torch.clamp(torch.round(g / sc), -8.0, 7.0), torch.zeros_like(g)) * sc)
    return torch.cat(got, -1)


def _plane64(s, case, p, page, off=None):
    """Rows of a plane as values in 64 bits: those at (page, off), or whole pages."""
    pick = (lambda t: t[page]) if off is None else (lambda t: t[page, :, off])
    raw, fmt = pick(s["planes"][p]), case["fmt"]
    if fmt == "bf16":
        return raw.double()
    sc = pick(s["planes"][p + "_scale"]).double()
    if fmt == "fp8_row":
        return raw.view(torch.float8_e4m3fn).double() * sc.unsqueeze(-1)
    x = torch.empty(*raw.shape[:-1], 2 * raw.shape[-1], dtype=torch.float64, device="cuda")
    if fmt == "tq4":
        lev = torch.tensor(TQ4_LEVELS + tuple(-v for v in TQ4_LEVELS), dtype=torch.float64, device="cuda")
        x[..., 0::2], x[..., 1::2] = lev[(raw % 16).int()], lev[(raw // 16).int()]
        return x * sc.unsqueeze(-1)
    x[..., 0::2], x[..., 1::2] = (raw % 16).double() - 8, (raw // 16).double() - 8
    return x * sc.repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    case, op = s["case"], case["op"]
    if op == "norm_rope":
        return _enter64(s["x"], s, case, s["weight"])
    if op == "norm_rope_store":
        q = _turn64(_enter64(s["q"], s, case, s["q_weight"]), s, case, True)
        k = _stored64(_turn64(_enter64(s["k"], s, case, s["k_weight"]), s, case, True), case)
        v = _stored64(_turn64(s["v"].double(), s, case, True), case)
        return {"q": q, "k": _turn64(k, s, case, False), "v": _turn64(v, s, case, False)}
    if op == "load":
        if case["by"] == "slots":
            slot = s["slots"].long()
        else:
            slot = []
            for b in range(case["seqs"]):
                p = torch.arange(int(s["cu"][b + 1]) - int(s["cu"][b]), device="cuda") + int(s["starts"][b])
                slot.append(s["tables"][b].long()[p // PAGE] * PAGE + p % PAGE)
            slot = torch.cat(slot)
        page, off = torch.div(slot, PAGE, rounding_mode="floor"), slot % PAGE
        got = [_turn64(_plane64(s, case, p, page, off), s, case, False) for p in ("k", "v")]
        return {"k": torch.cat(got, -1)} if case["fmt"] == "fp8_row" else {"k": got[0], "v": got[1]}
    Hq, Hk = case["q_heads"], case["kv_heads"]
    outs = []
    decode = op == "decode_diff"
    for b in range(s["tables"].shape[0]):
        T = int(s["lens"][b])
        page = s["tables"][b].long()[:-(-T // PAGE)]
        K, V = (_turn64(_plane64(s, case, p, page).transpose(0, 1).reshape(Hk, -1, 256)[:, :T], s, case, False)
                for p in ("k", "v"))
        q = (s["q"][b:b + 1] if decode else s["q"]).double()  # unrotated queries against rows rotated back
        heads = []
        for h in range(Hq):
            sc = q[:, h] @ K[h // (Hq // Hk)].t() / 16.0
            if not decode:
                sc = sc + torch.full_like(sc, -math.inf).triu(case["start"] + 1)
            heads.append(torch.softmax(sc, -1) @ V[h // (Hq // Hk)])
        lam = (s["lam"][b:b + 1] if decode else s["lam"]).double()
        y = torch.stack([heads[2 * i] - lam[:, i, None] * heads[2 * i + 1] for i in range(Hq // 2)], 1)
        if s["weight"] is not None:
            y = y * s["weight"].double() / torch.sqrt((y * y).sum(-1, keepdim=True) / 256 + 1e-5)
        outs.append(y * 0.8)
    return torch.cat(outs)
