"""A CTA may touch a peer's shared memory only once the peer has started: in every kernel that
runs in clusters a cluster barrier stands before the first access, in the order of the
program's text."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "rank_gemv_gb300" / "csrc"
KERNELS = ["sgmv_cc.cuh", "sgmv_stream.cuh", "sgmv_tc.cu", "sgmv_verify.cu", "sgmv_sample.cu"]


def code(name):
    return re.sub(r"//[^\n]*", "", (CSRC / name).read_text())


def waits(text):
    return re.search(r"\bcluster_sync\(\)", text) or (
        re.search(r"\bcluster_arrive_relaxed\(\)", text) and re.search(r"\bcluster_wait\(\)", text))


def before_access(text, touch):
    """The text before its first access to a peer, or None."""
    places = [m.start() for t in touch for m in re.finditer(t, text)]
    return text[:min(places)] if places else None


def before_first_access(kernel):
    """A lambda with a name that touches peers is looked at where it is called, not where it
    stands, unless it waits by itself."""
    touch = [r"peer_addr\("]
    for found in list(re.finditer(r"auto (\w+) = \[&\]", kernel)):
        if not kernel.startswith("auto", found.start()):
            continue  # within another
        start = kernel.index("{", found.end())
        depth, end = 0, start
        while True:
            depth += {"{": 1, "}": -1}.get(kernel[end], 0)
            end += 1
            if depth == 0:
                break
        body = before_access(kernel[start:end], touch)
        if body is not None and not waits(body):
            touch.append(rf"\b{found[1]}\(")
        kernel = kernel[:start] + " " * (end - start) + kernel[end:]
    return before_access(kernel, touch)


@pytest.mark.parametrize("name", KERNELS)
def test_peers_have_started_before_they_are_touched(name):
    text = code(name)
    text = before_first_access(text[text.index("__global__"):])
    assert text is None or waits(text)


def test_every_kernel_that_touches_peers_is_looked_at():
    assert {p.name for p in CSRC.iterdir() if re.search(r"\bpeer_addr\((?!const)", code(p.name))} == set(KERNELS)
