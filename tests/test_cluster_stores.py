"""Every kernel that stores into another CTA's shared memory waits for its cluster before the first
such store: until then the other CTA may not have started, and what it gets is lost.  Read from the
sources, since a run that loses a store says nothing about the next one."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "paged_gqa_decode_kv_gb300" / "csrc"
STORE = re.compile(r"map_shared_rank\s*\(|\bsend8\s*\(|\bsend16\s*\(|st\.shared::cluster|st\.async")
WAIT = re.compile(r"barrier\.cluster\.wait|cluster_sync\s*\(|\.sync\s*\(\s*\)\s*;")


def _kernels():
    """(file, name, body) of every __global__ function, comments taken out."""
    for f in sorted(CSRC.glob("*.cu*")):
        text = re.sub(r"//[^\n]*", "", f.read_text())
        for m in re.finditer(r"__global__\s+void", text):
            start = text.index("{", m.end())
            depth, i = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            name = re.findall(r"(\w+)\s*\(", text[m.end():start])[-1]
            yield f.name, name, text[start:i]


KERNELS = [(f, n, b) for f, n, b in _kernels() if STORE.search(b)]


def test_the_kernels_are_found():
    assert {n for _, n, _ in KERNELS} >= {"grow_tables_kernel", "attention_fp4_unit_kernel"}


@pytest.mark.parametrize("file,name,body", KERNELS, ids=[n for _, n, _ in KERNELS])
def test_a_cluster_has_started_before_the_first_remote_store(file, name, body):
    first = STORE.search(body).start()
    assert WAIT.search(body[:first]), "%s: %s" % (file, name)
