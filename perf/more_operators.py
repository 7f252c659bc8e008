"""Cases of attention over the paged quantized cache in two more forms: one new token for each sequence that sees a
sliding window and the first few tokens (sinks), and ragged chunks of new tokens of several sequences in one call,
causal over everything stored or over window and sinks.

Each case is one call of a program that serves a model from a paged cache; `run` computes it either in plain tensor
operations (own = False) or through the library (own = True).
"""
import math

import torch

own = False

# Lloyd-Max magnitudes of N(0, 1) for 16 levels, as the TQ4 rows hold them
TQ4_LEVELS = (0.12841796875, 0.387939453125, 0.65673828125, 0.9423828125, 1.255859375, 1.6181640625, 2.068359375,
              2.732421875)
FORMATS = {"q4_had32": 0, "bf16": 1, "q4_0": 3, "tq4": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode token of one sequence whose layer sees 1024 tokens back
        dict(name="local_token_1_w1024", op="decode_local", fmt="q4_had32", seqs=1, longest=9001, window=1024, sinks=4,
             q_heads=24, kv_heads=4, width=256, page=16),
        # the same late in a 262144-token sequence, a wider window, the pages between long freed
        dict(name="local_token_1_w4096_at_262144", op="decode_local", fmt="q4_had32", seqs=1, longest=262144, window=4096,
             sinks=4, q_heads=24, kv_heads=4, width=256, page=16),
        # a decode batch of 32 ragged sequences, some shorter than the window
        dict(name="local_batch_32_w4096", op="decode_local", fmt="q4_had32", seqs=32, longest=20000, window=4096, sinks=4,
             q_heads=24, kv_heads=4, width=256, page=16),
        # codebook rows of 128-wide heads, an odd window
        dict(name="local_batch_64_tq4_d128", op="decode_local", fmt="tq4", seqs=64, longest=8000, window=2001, sinks=16,
             q_heads=32, kv_heads=8, width=128, page=32),
        # bf16 rows, no sinks
        dict(name="local_batch_16_bf16", op="decode_local", fmt="bf16", seqs=16, longest=6000, window=1024, sinks=0,
             q_heads=24, kv_heads=4, width=256, page=16),
        # draft rows of 16 sequences to be verified, a few for each
        dict(name="chunk_16_drafts", op="attn_seqs", fmt="q4_had32", seqs=16, rows=5, longest=8000, window=0, sinks=0,
             q_heads=24, kv_heads=4, width=256, page=16),
        # the last short chunk of a prompt
        dict(name="chunk_65_at_4000_q4_0", op="attn_seqs", fmt="q4_0", seqs=1, rows=65, longest=4065, window=0, sinks=0,
             q_heads=24, kv_heads=4, width=256, page=16),
        # prompts of eight sequences from their first token on, bf16 rows of 128-wide heads
        dict(name="chunk_8_prompts_bf16_d128", op="attn_seqs", fmt="bf16", seqs=8, rows=1501, longest=1501, window=0,
             sinks=0, q_heads=32, kv_heads=8, width=128, page=64),
        # chunks of five sequences at different depths, codebook rows
        dict(name="chunk_5_ragged_tq4", op="attn_seqs", fmt="tq4", seqs=5, rows=700, longest=9000, window=0, sinks=0,
             q_heads=24, kv_heads=4, width=256, page=16),
        # a chunk of a layer with a window
        dict(name="chunk_2048_at_30000_w4096", op="attn_seqs", fmt="q4_had32", seqs=1, rows=2048, longest=32048,
             window=4096, sinks=4, q_heads=24, kv_heads=4, width=256, page=16),
        # a whole prompt chunk at depth 16384
        dict(name="chunk_4096_at_16384", op="attn_seqs", fmt="q4_had32", seqs=1, rows=4096, longest=20480, window=0,
             sinks=0, q_heads=24, kv_heads=4, width=256, page=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    fmt = rng.choice(["q4_had32", "q4_had32", "q4_0", "tq4", "bf16"])
    width = rng.choice([64, 128, 256, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    common = dict(fmt=fmt, q_heads=kv_heads * rng.choice([1, 2, 3, 4, 6, 8]), kv_heads=kv_heads, width=width,
                  page=rng.choice([16, 16, 32, 64, 128]))
    if rng.random() < 0.5:
        seqs = _log(rng, 1, 100)
        return dict(op="decode_local", seqs=seqs, longest=_log(rng, 20, min(131072, 2 ** 20 // (seqs * kv_heads))),
                    window=_log(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 16, 33]), **common)
    seqs = rng.choice([1, 1, 2, 3, 5, 9, 16])
    rows = _log(rng, 1, 2048 // seqs)
    pairs = 4 * 10 ** 11 // (common["q_heads"] * width)  # what the largest listed case has
    longest = rows + _log(rng, 1, min(30000, pairs // (seqs * rows), 2 ** 19 // (seqs * kv_heads))) - 1
    local = rng.random() < 0.4
    return dict(op="attn_seqs", seqs=seqs, rows=rows, longest=longest, window=_log(rng, 16, 8192) if local else 0,
                sinks=rng.choice([0, 1, 4, 33]) if local else 0, **common)


def _shares(n):
    """Shares of the longest for n sequences, spread over 0.1 .. 1; the first has all of it."""
    return [1.0] + [0.1 + 0.9 * ((i * 0.6180339887498949) % 1.0) for i in range(1, n)]


def _lens(case):
    """Stored tokens of every sequence, its new ones among them."""
    return [max(1, round(case["longest"] * s)) for s in _shares(case["seqs"])]


def _rows(case):
    """New tokens of every sequence."""
    if case["op"] == "decode_local":
        return [1] * case["seqs"]
    rows = [max(1, round(case["rows"] * s)) for s in reversed(_shares(case["seqs"]))]
    return [min(r, n) for r, n in zip(rows, _lens(case))]


# ------------------------------------------------------------------ inputs

def _planes(g, case, pages):
    """The planes of a filled pool: normal-like codes and one magnitude per scale."""
    fmt, D, rows = case["fmt"], case["width"], (pages, case["kv_heads"], case["page"])

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    out = {}
    for p in ("k", "v"):
        if fmt == "bf16":
            out[p] = randn(*rows, D).to(torch.bfloat16)
            continue
        if fmt == "tq4":
            code = torch.randint(0, 256, (*rows, D // 2), generator=g, device="cuda", dtype=torch.uint8)
            scale = torch.exp(0.3 * randn(*rows))
        else:
            c = (randn(*rows, D // 2, 2) * 3.4).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
            code = c[..., 0] | (c[..., 1] << 4)
            scale = torch.exp(0.3 * randn(*rows, D // 32)) * 0.3
        out[p], out[p + "_scale"] = code, scale.to(torch.float16)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": dict(case)}
    D, page, Hq, Hk, W = case["width"], case["page"], case["q_heads"], case["kv_heads"], case["window"]
    lens, rows = _lens(case), _rows(case)
    B, n = len(lens), sum(rows)
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    s["host"] = (lens, rows, cu)  # a server knows its own lengths
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    # pages from anywhere in the pool; those that no row can see any more are given back (-1)
    wide = -(-max(lens) // page)
    col = torch.arange(wide)
    at = torch.tensor(lens)[:, None]
    keep = col * page < at
    if W:
        first = at - torch.tensor(rows)[:, None] - W + 1  # of the first new token's window
        keep &= (col * page < case["sinks"]) | (col * page + page > first)
    total = int(keep.sum())
    s["pages"] = total + 3
    order = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    tables[keep.cuda()] = order[:total]
    s["tables"] = tables
    s["planes"] = _planes(g, case, s["pages"])
    s["signs"] = None
    if case["fmt"] == "tq4":
        s["signs"] = torch.randint(-2 ** 31, 2 ** 31, (D // 32,), generator=g, device="cuda").to(torch.int32)
    # the queries of a fused projection, beside the keys and values
    s["q"] = (torch.randn((n, Hq + 2 * Hk, D), generator=g, device="cuda") * 2).to(torch.bfloat16)[:, :Hq]
    if own:
        from bit_quantized_kv_store_gb300 import kvq
        cache = kvq.Cache(FORMATS[case["fmt"]], Hk, D, page, s["pages"], signs=s["signs"])
        for name, t in s["planes"].items():
            setattr(cache, name, t)
        cache.refresh()
        s["kvq"], s["cache"] = kvq, cache
        s["ws"] = kvq.alloc_attn_workspace(cache, n, B, Hq, max(rows), max(lens), W, case["sinks"])
    else:
        _plain_tables(s)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_tables(s):
    """The matrices and levels that a program of plain operations keeps for a cache."""
    case = s["case"]
    n = {"q4_had32": 32, "tq4": case["width"]}.get(case["fmt"])
    if n:
        h = torch.ones(1, 1, device="cuda")
        two = torch.tensor([[1.0, 1.0], [1.0, -1.0]], device="cuda")
        while h.shape[0] < n:
            h = torch.kron(h, two)
        s["had"] = h * (1 / math.sqrt(n))
    if case["fmt"] == "tq4":
        bit = torch.arange(n, device="cuda")
        s["sign"] = 1.0 - 2.0 * ((s["signs"].long()[bit // 32] >> (bit % 32)) & 1).float()
        lev = torch.tensor(TQ4_LEVELS, device="cuda")
        s["levels"] = torch.cat((lev, -lev))


def _turn(x, s, forward):
    """Rows into the cache's space, and back."""
    fmt = s["case"]["fmt"]
    if fmt == "q4_had32":
        return (x.reshape(-1, 32) @ s["had"]).reshape(x.shape)
    if fmt == "tq4":
        return (x * s["sign"]) @ s["had"] if forward else (x @ s["had"]) * s["sign"]
    return x


def _stored(s, p, page, off):
    """Rows of plane p at (page, off) [..., heads, width], as values in the cache's space (fp32)."""
    fmt, raw = s["case"]["fmt"], s["planes"][p][page, :, off]
    if fmt == "bf16":
        return raw.float()
    scale = s["planes"][p + "_scale"][page, :, off].float()
    c = torch.stack((raw & 15, raw >> 4), -1).flatten(-2).to(torch.int32)
    if fmt == "tq4":
        return s["levels"][c] * scale[..., None]
    return ((c - 8).float().reshape(*c.shape[:-1], -1, 32) * scale[..., None]).reshape(c.shape)


def _plain_local(s):
    case = s["case"]
    B, Hq, Hk, D, page = case["seqs"], case["q_heads"], case["kv_heads"], case["width"], case["page"]
    T = s["lens"].long()[:, None]
    first = (T - case["window"]).clamp_(min=0)
    head = first.clamp(max=case["sinks"])  # sinks in front of the window
    count = head + T - first
    j = torch.arange(int(min(case["longest"], case["window"] + case["sinks"])), device="cuda")[None]
    seen = j < count
    pos = torch.where(j < head, j, j - head + first).clamp_(max=T - 1)
    pg, off = s["tables"].long().gather(1, pos // page), pos % page
    K, V = (_stored(s, p, pg, off).transpose(1, 2) for p in ("k", "v"))  # [B, heads, keys, width]
    q = _turn(s["q"].float(), s, True).reshape(B, Hk, Hq // Hk, D)
    sc = torch.where(seen[:, None, None], q @ K.transpose(-1, -2) * D ** -0.5, -math.inf)
    e = torch.exp(sc - sc.amax(-1, keepdim=True))
    o = (e @ V) / e.sum(-1, keepdim=True)
    return _turn(o.reshape(B, Hq, D), s, False).to(torch.bfloat16)


def _plain_chunks(s):
    case = s["case"]
    Hq, Hk, D, page, W = case["q_heads"], case["kv_heads"], case["width"], case["page"], case["window"]
    lens, rows, cu = s["host"]
    q = _turn(s["q"].float(), s, True)
    out = torch.empty(cu[-1], Hq, D, device="cuda")
    for b, (T, n) in enumerate(zip(lens, rows)):
        pos = torch.arange(T, device="cuda")
        first = T - n - W + 1 if W else 0  # of the first row's window
        if first > case["sinks"]:
            pos = torch.cat((pos[:case["sinks"]], pos[first:]))
        pg, off = s["tables"][b].long()[pos // page], pos % page
        at = torch.arange(T - n, T, device="cuda")[:, None]
        seen = pos <= at
        if W:
            seen &= (pos > at - W) | (pos < case["sinks"])
        K, V = (_stored(s, p, pg, off) for p in ("k", "v"))
        for kv in range(Hk):  # the query heads of one KV head together
            heads = slice(kv * (Hq // Hk), (kv + 1) * (Hq // Hk))
            sc = torch.where(seen, q[cu[b]:cu[b + 1], heads].transpose(0, 1) @ K[:, kv].T * D ** -0.5, -math.inf)
            e = torch.exp(sc - sc.amax(-1, keepdim=True))
            out[cu[b]:cu[b + 1], heads] = ((e @ V[:, kv]) / e.sum(-1, keepdim=True)).transpose(0, 1)
    return _turn(out, s, False).to(torch.bfloat16)


def run(s):
    case = s["case"]
    if not own:
        return _plain_local(s) if case["op"] == "decode_local" else _plain_chunks(s)
    kvq, scale = s["kvq"], case["width"] ** -0.5
    if case["op"] == "decode_local":
        return kvq.decode_local(s["cache"], s["q"], s["lens"], s["tables"], case["longest"], scale, case["window"],
                                sinks=case["sinks"], dtype=torch.bfloat16, workspace=s["ws"])
    return kvq.attn_seqs(s["cache"], s["q"], s["cu"], s["lens"], s["tables"], max(s["host"][1]), case["longest"], scale,
                         window=case["window"], sinks=case["sinks"], dtype=torch.bfloat16, workspace=s["ws"])


# ------------------------------------------------------------------ what a pass cannot do without

def _upto(p, W):
    """Tokens that positions 0 .. p - 1 see in their windows of W, added up."""
    if not W or p <= W:
        return p * (p + 1) // 2
    return W * (W + 1) // 2 + (p - W) * W


def _sinks_upto(p, W, sinks):
    """The sinks that positions 0 .. p - 1 see in front of their windows, added up: min(sinks, position - W + 1)."""
    m = max(0, p - W)
    return m * (m + 1) // 2 if m <= sinks else sinks * (sinks + 1) // 2 + (m - sinks) * sinks


def work(case):
    W, S, D = case["window"], case["sinks"], case["width"]
    row = {"q4_had32": D // 2 + D // 16, "q4_0": D // 2 + D // 16, "tq4": D // 2 + 2, "bf16": 2 * D}[case["fmt"]]
    keys = pairs = 0
    for T, n in zip(_lens(case), _rows(case)):
        pairs += _upto(T, W) - _upto(T - n, W)
        if W:
            pairs += _sinks_upto(T, W, S) - _sinks_upto(T - n, W, S)
            first = max(0, T - n - W + 1)
            keys += T - first + min(S, first)
        else:
            keys += T
    q = sum(_rows(case)) * case["q_heads"] * D
    return {"bytes": keys * 2 * case["kv_heads"] * row + q * 4, "flops": 4 * pairs * case["q_heads"] * D}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _wht64(x):
    """Orthonormal Walsh-Hadamard transform of the last dimension (64 bits), by its definition's matrix."""
    n = x.shape[-1]
    i = torch.arange(n, device=x.device)
    both = i[:, None] & i[None, :]
    odd = sum((both >> b) & 1 for b in range(n.bit_length())) & 1
    return torch.matmul(x, (1.0 - 2.0 * odd.double()) / n ** 0.5)


def _values64(s, p, page, off):
    """Rows of a plane as the original space's values, in 64 bits."""
    case = s["case"]
    raw = s["planes"][p][page, :, off]
    if case["fmt"] == "bf16":
        return raw.double()
    sc = s["planes"][p + "_scale"][page, :, off].double()
    x = torch.empty(*raw.shape[:-1], 2 * raw.shape[-1], dtype=torch.float64, device="cuda")
    if case["fmt"] == "tq4":
        lev = torch.tensor(TQ4_LEVELS + tuple(-v for v in TQ4_LEVELS), dtype=torch.float64, device="cuda")
        x[..., 0::2], x[..., 1::2] = lev[(raw % 16).int()], lev[(raw // 16).int()]
        words = [int(w) for w in s["signs"]]
        sign = torch.tensor([-1.0 if (words[i // 32] >> (i % 32)) & 1 else 1.0 for i in range(x.shape[-1])],
                            dtype=torch.float64, device="cuda")
        return _wht64(x * sc.unsqueeze(-1)) * sign
    x[..., 0::2], x[..., 1::2] = (raw % 16).double() - 8, (raw // 16).double() - 8
    x = x * sc.repeat_interleave(32, -1)
    if case["fmt"] == "q4_had32":
        x = torch.cat([_wht64(part) for part in x.split(32, -1)], -1)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    lens, rows, cu = s["host"]
    Hq, Hk, page, W = case["q_heads"], case["kv_heads"], case["page"], case["window"]
    out = torch.empty(cu[-1], Hq, case["width"], dtype=torch.float64, device="cuda")
    for b in range(len(lens)):
        T, n = lens[b], rows[b]
        key = torch.arange(T, device="cuda")
        if W:  # only the keys that some row of the sequence sees
            key = key[(key < case["sinks"]) | (key >= T - n - W + 1)]
        slot = s["tables"][b].long().index_select(0, torch.div(key, page, rounding_mode="floor"))
        K, V = (_values64(s, p, slot, key % page) for p in ("k", "v"))
        for lo in range(0, n, 512):
            hi = min(n, lo + 512)
            row = torch.arange(T - n + lo, T - n + hi, device="cuda").unsqueeze(1)
            hidden = key > row
            if W:
                hidden = hidden | ((row - key >= W) & (key >= case["sinks"]))
            for h in range(Hq):
                q = s["q"][cu[b] + lo:cu[b] + hi, h].double()
                sc = (q @ K[:, h // (Hq // Hk)].t() / case["width"] ** 0.5).masked_fill(hidden, -math.inf)
                out[cu[b] + lo:cu[b] + hi, h] = torch.softmax(sc, -1) @ V[:, h // (Hq // Hk)]
    return out
