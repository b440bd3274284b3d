"""Another block's shared memory is touched only once that block is known to run: the
helpers through which the products and the column sums reach it, read from the sources."""
import os
import re

import pytest

from tests.test_kernel_source_order import ALL
from tests.test_tensor_waits_cpu import CSRC, function, source

#: a function of another file's that reaches a peer -> what has to stand before its call
HELPERS = {"load_peer": r"\bcluster_(sync|wait)\(\)", "settle": r"\bcluster_arrive\(\)"}


def users(helper):
    return [k for k in ALL if re.search(r"\b%s\s*[<(]" % helper, k[2])]


def test_the_helpers_are_used():
    assert {n for _, n, _ in users("load_peer")} == {"activation_grad_kernel"}
    assert {n for _, n, _ in users("settle")} == {"matmul_kernel", "matmul_mid_kernel"}


@pytest.mark.parametrize("helper,kernel", [(h, k) for h in HELPERS for k in users(h)],
                         ids=lambda v: v if isinstance(v, str) else v[1])
def test_a_cluster_barrier_comes_before_a_helper(helper, kernel):
    file, name, body = kernel
    first = re.search(r"\b%s\s*[<(]" % helper, body).start()
    barrier = re.search(HELPERS[helper], body)
    assert barrier and barrier.start() < first, (file, name)


def test_the_shares_are_sent_behind_the_barrier():
    """settle() takes the wait that belongs to the kernels' arrival, and everybody stays
    until what was sent has been received."""
    body = function(source("zero_matmul.cu"), "settle")
    wait, send = body.index("cluster_wait()"), body.index("send_shares(")
    received, meet = body.index("join<"), body.index("cluster_meet()")
    assert wait < send < received < meet
    assert body.index("fence.proxy.async") < body.index("__syncthreads()") < wait


def test_no_other_function_reaches_a_peer():
    """What is not a kernel and reaches one is in the lists of these tests."""
    known = {"load_peer", "load_peer4", "store_peer", "peer_addr", "arrive_first", "send_shares",
             "tensor_load", "join", "settle", "commit2", "commit2_first"}
    for file in sorted(os.listdir(CSRC)):
        text = source(file)
        for m in re.finditer(r"__device__ __forceinline__ [\w ]*?(\w+)\([^{;]*\)\s*\{", text):
            body = function(text[m.start():], m.group(1))
            if re.search(r"\b(peer_addr|load_peer|load_peer4|store_peer)\(|mapa\.", body):
                assert m.group(1) in known, (file, m.group(1))
