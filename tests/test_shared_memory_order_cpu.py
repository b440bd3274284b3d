"""Shared memory that a kernel uses for two things in turn, read from the sources: a
lane that is ahead must not overwrite what another one has still to read."""
import re

from tests.test_tensor_waits_cpu import function, source


def test_values_are_turned_before_their_place_takes_the_columns_sums():
    """activation_grad_kernel turns 8-bit values in joined[warp], and adds up there."""
    body = function(source("zero_activation.cu"), "activation_grad_kernel")
    turned, sums = body.rindex("joined[warp], z"), body.index("joined[warp][rows::column")
    assert turned < sums
    assert "__syncwarp();" in body[turned:sums]


def test_turning_begins_when_the_warp_is_there():
    body = function(source("zero_rows.cuh"), "turn")
    first, second = [m.start() for m in re.finditer(r"__syncwarp\(\);", body)]
    write, read = body.index("shared[column<!BACK>(e)] ="), body.index("= shared[column<BACK>(e)]")
    assert first < write < second < read


def test_a_warp_converges_before_a_barrier_of_its_group():
    """bar.sync is .aligned, and stands behind a store by one lane."""
    body = function(source("zero_norm.cu"), "norm_grad_kernel")
    assert re.search(r"__syncwarp\(\);\s*asm volatile\(\"bar\.sync", body)
