"""Shared memory of another CTA may be touched once all CTAs of the cluster are known to have started: in every kernel
that does, a barrier of the cluster stands before the first access.  Read from the sources, since a kernel without it goes
wrong only when a CTA starts late."""
import re
from pathlib import Path

import pytest

SOURCES = sorted((Path(__file__).resolve().parents[1] / "speculative_decoding_dspark_gb300" / "csrc").glob("*.cu"))
# an access to, or an arrival in, another CTA's shared memory
REMOTE = re.compile(r"\b(cluster_(ld|st|atomic)\w*|expect_at|arrive_at|arrive_read|tma_load_pair|commit_pair_elect|umma_pair_elect)\s*\(")
BARRIER = re.compile(r"\b(cluster_sync|cluster_wait|pair_sync)\s*\(\s*\)")


def kernels(text):
    """The bodies of a source's kernels."""
    text = re.sub(r"//[^\n]*", "", text)
    for at in re.finditer(r"\b__global__\b", text):
        start = text.index("{", at.end())
        depth, end = 1, start + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield text[at.end():start].split("(")[-2].split()[-1] if "(" in text[at.end():start] else "?", text[start:end]


def remote_kernels():
    return [(f.name, name, body) for f in SOURCES for name, body in kernels(f.read_text()) if REMOTE.search(body)]


def test_there_are_such_kernels():
    assert {f for f, _, _ in remote_kernels()} >= {"distill.cu", "logprobs.cu", "markov_few.cu", "markov_grad.cu"}


@pytest.mark.parametrize("source,name,body", remote_kernels(), ids=[f"{f}:{n}" for f, n, _ in remote_kernels()])
def test_a_cluster_barrier_comes_before_the_first_access(source, name, body):
    barrier = BARRIER.search(body)
    assert barrier and barrier.start() < REMOTE.search(body).start()
