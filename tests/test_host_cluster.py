"""Kernels that write into the shared memory of another CTA of their cluster, from the sources alone:
a peer's shared memory exists only once the peer has started, which nothing but a cluster barrier
shows.  A write before one is a race that no run on a GPU has to show."""
import os
import re

import pytest

from sparse_attention_fp4_pack_b200 import build

PEER_STORE = re.compile(r"st\.shared::cluster|st_cluster_\w+\(")


def kernels(source):
    """(name, body) of each __global__ function."""
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\s*\([^{;]*\)\s*\{", source):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(source[at], 0)
            at += 1
        yield m.group(1), source[m.end():at]


@pytest.mark.parametrize("name", ["paged_release_kernel", "attn_kernel"])
def test_a_peer_is_written_after_it_has_started(name):
    found = {}
    for path in build.sources():
        with open(path) as f:
            found.update({n: (os.path.basename(path), body) for n, body in kernels(f.read())})
    path, body = found[name]
    body = re.sub(r"//[^\n]*", "", body)
    store = PEER_STORE.search(body).start()
    arrive, wait = body.find("tc::cluster_arrive()"), body.find("tc::cluster_wait()")
    assert 0 <= arrive < wait < store, f"{path}: {name} writes into a peer before it is known to have started"
