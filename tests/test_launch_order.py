"""Kernels that may begin before the one in front of them has ended (programmatic dependent
launch) read nothing that it may have written ahead of their wait: lengths, row numbers, page
tables, slots, positions and selections are made on the device as often as not.  Read off the
sources: the order of two statements of a kernel is the same on every machine."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_kv_store_gb300", "csrc")
READS = re.compile(r"\b(seq_lens|block_tables|cu_rows|cu_lens|row_lens|starts|slots|positions|sel)\s*(?:\[|\+)|\b(seq_rows)\(")


def kernels():
    """(file, name, body without comments) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        for m in re.finditer(r"__global__\s+void\b", text):
            at = text.index("{", m.end())
            name = re.findall(r"(\w+)\s*\(", re.sub(r"__launch_bounds__\s*\((?:[^()]|\([^()]*\))*\)", "", text[m.end():at]))[0]
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            yield os.path.basename(path), name, text[at + 1:end - 1]


KERNELS = list(kernels())


def test_kernels_are_found():
    names = {name for _, name, _ in KERNELS}
    assert {"attn_few_kernel", "attn_merge_kernel", "attn_chunk_kernel", "decode_q4_round_kernel", "decode_q4_spec_kernel",
            "merge_kernel", "load_q4_kernel"} <= names


def ahead_of_the_wait(body):
    return [a or b for a, b in READS.findall(body[:body.index("pdl_wait()")])]


@pytest.mark.parametrize("file,name,body", [k for k in KERNELS if "pdl_wait()" in k[2]], ids=lambda x: x if len(x) < 40 else "")
def test_metadata_is_read_behind_the_wait(file, name, body):
    assert ahead_of_the_wait(body) == []


def test_kernels_launched_ahead_wait():
    launched = set()
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        launched |= set(re.findall(r"launch_pdl\((\w+)", open(path).read()))
    without = {name for _, name, body in KERNELS if "pdl_wait()" not in body}
    assert launched & {name for _, name, _ in KERNELS} and not launched & without
