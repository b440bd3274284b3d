"""What the kernels' sources have to do in order, read from the text: rules of
the programming model whose breach shows in no result most of the time."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "zero_sharded_optimizer_step_gb300", "csrc")


def kernels():
    """(file, name, body) of every __global__ function, comments left out."""
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
        for m in re.finditer(r"__global__", text):
            at = text.index("{", m.end())
            name = re.findall(r"(\w+)\s*\((?:const|int|unsigned|float|uint|int64|char|void|\w+ \*)",
                              text[m.end():at])[-1]
            depth, end = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
                if depth == 0:
                    break
            out.append((os.path.basename(path), name, text[at:end]))
    return out


ALL = kernels()
#: what reaches into another block of the cluster
PEER = r"\b(store_peer|load_peer4|peer_addr|join|arrive_first|tensor_load|commit2)\b"


def test_the_kernels_are_found():
    names = {n for _, n, _ in ALL}
    assert {"embed_cluster_kernel", "mx4_matmul_kernel", "mx4_pair_kernel", "dropout_kernel"} <= names


@pytest.mark.parametrize("kernel", [k for k in ALL if re.search(PEER, k[2])], ids=lambda k: k[1])
def test_a_cluster_barrier_comes_before_a_peers_shared_memory(kernel):
    """Another block's shared memory may be touched only once that block is
    known to run."""
    file, name, body = kernel
    first = re.search(PEER, body).start()
    barrier = re.search(r"\bcluster_(sync|wait)\(\)", body)
    assert barrier and barrier.start() < first, (file, name)


@pytest.mark.parametrize("kernel", [k for k in ALL if "pdl_wait()" in k[2]], ids=lambda k: k[1])
def test_a_kernel_waits_for_the_one_before_whatever_its_form(kernel):
    """pdl_wait() is what makes an earlier kernel's writes visible, to the grid that
    calls it: no template argument or flag may leave it out or put it off.  (A warp
    with a task of its own may have a wait of its own.)"""
    file, name, body = kernel
    assert not re.search(r"\bif\s*\([^;{}]*\)\s*pdl_wait\(\)", body), (file, name)
    for m in re.finditer(r"\bif\s*\(([^{};]*)\)\s*\{\s*pdl_wait\(\)", body):
        assert "warp" in m.group(1), (file, name)
