"""How the tensor-core products wait, read from the sources: what shows only where a
wait runs out, or where the hardware lets a warp's lanes drift apart."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "zero_sharded_optimizer_step_gb300", "csrc")
PRODUCTS = ["zero_matmul.cu", "zero_mx4_matmul.cu"]


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def closed(text, at, pair="()"):
    """The end of the bracket that opens at `at`."""
    depth = 0
    while True:
        depth += {pair[0]: 1, pair[1]: -1}.get(text[at], 0)
        at += 1
        if depth == 0:
            return at


def function(text, name):
    """The body of the function of that name."""
    m = re.search(r"\b%s\s*\([^;{]*\)\s*\{" % name, text)
    return text[m.end() - 1:closed(text, m.end() - 1, "{}")]


def guarded(text):
    """(condition, statement) of every `if`."""
    for m in re.finditer(r"\bif\s*(?:constexpr\s*)?\(", text):
        end = closed(text, m.end() - 1)
        at = end
        while True:                                   # a loop's head belongs to its statement
            loop = re.match(r"\s*(for|if|while)\s*\(", text[at:])
            if not loop:
                break
            at = closed(text, at + loop.end() - 1)
        brace = re.match(r"\s*\{", text[at:])
        stop = closed(text, at + brace.end() - 1, "{}") if brace else text.index(";", at)
        yield text[m.end() - 1:end], text[end:stop]


#: conditions that hold in one lane of a warp
LANE = r"threadIdx\.x == 0|\blane == 0|\bone\b"


@pytest.mark.parametrize("name", ["bar_wait", "bar_wait_both"])
def test_a_warps_lanes_get_one_answer(name):
    """Each lane's own would let some give up in the poll in which others succeed."""
    body = function(source("zero_tensor.cuh"), name)
    answers = re.findall(r"if \((.*)\) return true;", body)
    assert len(answers) == 1 and answers[0].startswith("__all_sync(0xffffffffu, "), body


@pytest.mark.parametrize("file", PRODUCTS)
def test_a_single_threads_wait_does_not_ask_its_warp(file):
    """And only that one: the others' form wants every lane."""
    text = source(file)
    alone = 0
    for condition, statement in guarded(text):
        if re.search(LANE, condition):
            assert not re.search(r"\bbar_wait(_both)?\(", statement), (condition, statement)
            alone += len(re.findall(r"\bbar_wait_alone\(", statement))
    assert alone == len(re.findall(r"\bbar_wait_alone\(", text)) > 0
    assert len(re.findall(r"\bbar_wait\(", text)) > 5


@pytest.mark.parametrize("name", ["load16", "load32"])
def test_a_warp_converges_before_it_reads_tensor_memory(name):
    """tcgen05.ld is .aligned: lanes that stored more than others before may be behind."""
    body = function(source("zero_tensor.cuh"), name)
    assert "__syncwarp();" in body[:body.index("tcgen05.ld")], body


@pytest.mark.parametrize("file", PRODUCTS)
def test_a_warp_converges_before_it_frees_tensor_memory(file):
    text = source(file)
    found = [m.start() for m in re.finditer(r"tcgen05\.dealloc", text)]
    assert found
    for at in found:
        assert re.search(r"__syncwarp\(\);\s*asm volatile\(\"$", text[:at]), text[at - 200:at]


@pytest.mark.parametrize("file", PRODUCTS)
def test_tensor_memory_is_read_through_the_helpers_alone(file):
    assert "tcgen05.ld." not in source(file)


def test_a_warp_converges_before_a_cluster_barrier():
    """barrier.cluster is .aligned too, wherever it stands."""
    found = 0
    for file in sorted(os.listdir(CSRC)):
        text = source(file)
        for m in re.finditer(r'asm volatile\("barrier\.cluster\.(arrive|wait)', text):
            before = text[:m.start()].rstrip()
            # the other half, which is .aligned itself, or the warp's own barrier
            assert re.search(r'(__syncwarp\(\)|asm volatile\("barrier\.cluster\.arrive'
                             r'[\w.]*;" ::: "memory"\));$', before), (file, before[-200:])
            found += 1
    assert found > 4
