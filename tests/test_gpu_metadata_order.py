"""Lengths and page tables that a kernel writes directly in front of a decode call count as if
the device had been waited for (the decode kernels begin while the one in front drains)."""
import pytest
import torch

from bit_quantized_kv_store_gb300 import synth
from tests.test_gpu_parity import K  # noqa: F401

pytestmark = pytest.mark.gpu

DEV = "cuda"
HQ, HK, D, PS = 24, 4, 256, 16


def write(dst, src):
    """By a kernel (a copy between tensors of one type may be the copy engine's)."""
    torch.add(src, 0, out=dst)


@pytest.mark.parametrize("fmt,call", [(f, c) for f in ("FMT_Q4_HAD32", "FMT_Q4_0") for c in ("attn", "step", "merged", "window")]
                         + [("FMT_TQ4", "attn"), ("FMT_BF16", "attn")])
@pytest.mark.parametrize("lens", [[3000], [5000, 333], [9001] * 7 + [16]])  # grids of less and of more than one wave
@pytest.mark.parametrize("last", ["lens", "table"])
def test_metadata_written_right_before(K, fmt, call, lens, last):
    B, top = len(lens), max(lens)
    pages = -(-top // PS)
    signs = torch.arange(D // 32, dtype=torch.int32, device=DEV) * 77777
    cache = K.Cache(getattr(K, fmt), HK, D, PS, pages * B, signs=signs if fmt == "FMT_TQ4" else None)
    g = torch.Generator().manual_seed(7)
    table = torch.randperm(pages * B, generator=g).to(torch.int32).reshape(B, pages).to(DEV)
    n = pages * B * PS
    kv = synth.normal((n, 2, HK, D), DEV, "order", n).to(torch.bfloat16)
    K.store(cache, kv[:, 0].contiguous(), kv[:, 1].contiguous(), torch.arange(n, dtype=torch.int32, device=DEV))
    q = synth.normal((B, HQ, D), DEV, "order", "q")
    new = synth.normal((2, B, HK, D), DEV, "order", "new").to(torch.bfloat16)
    ws = K.alloc_workspace(cache, B, HQ, top)
    ws.zero_()
    out = torch.empty(B, HQ, D, device=DEV)
    right = {"lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "table": table}
    before = {"lens": torch.tensor([max(1, x // 3) for x in lens], dtype=torch.int32, device=DEV),
              "table": table.flip(1).contiguous()}
    if call == "window":  # rows of one sequence
        right["table"], before["table"] = table[:1].contiguous(), before["table"][:1].contiguous()
    now = {k: v.clone() for k, v in before.items()}

    def run(m):
        a = (m["lens"], m["table"], top, D ** -0.5, ws)
        if call == "merged":
            return K.decode_merged(cache, q, *a, out=out)
        if call == "step":
            K.decode_step(cache, new[0], new[1], q.to(torch.bfloat16), *a)
        elif call == "window":
            K.decode_window(cache, q, *a)
        else:
            K.decode_attn(cache, q, *a)
        return K.merge(cache, ws, B, HQ, m["lens"], top, out)

    def step():
        for name in sorted(right, key=lambda k: k == last):
            write(now[name], right[name])
        run(now)
        for name in right:
            write(now[name], before[name])

    want = run(right).clone()
    for _ in range(5):
        out.zero_()
        step()
        assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
