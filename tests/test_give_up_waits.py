"""The waits on the path by which an attention kernel gives up (a bounded wait ran out): its MMAs are over
before the tensor memory is freed. A model of mbarrier phases on the CPU, with the rings, depths and tiles
in flight as the kernels' sources have them; no GPU path is made to run out."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hierarchical_sparse_attention_gb300", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def give_up(text):
    """The kernel's last `if (!ok) {` block: what a CTA that gave up does before it frees its memories."""
    at = text.rindex("if (!ok) {", 0, text.index("tcgen05.dealloc"))
    depth, end = 0, at
    for end in range(text.index("{", at), len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            break
    return text[at:end + 1]


def number(text, token):
    return int(token) if token.isdigit() else int(re.search(r"constexpr int (?:\w+ = \w+, )*%s = (\d+)" % token, text).group(1))


def returns(depth, use, over):
    """Does a parity wait for use `use` of a ring of `depth` barriers return once the uses 0 .. over - 1 are over?"""
    phases = len([u for u in range(over) if u % depth == use % depth])  # completed phases of that barrier
    return (phases - 1) % 2 == (use // depth) % 2


def test_the_model_of_a_parity_wait():
    assert not returns(1, 0, 0) and returns(1, 0, 1)
    assert not returns(1, 1, 1) and returns(1, 1, 2)
    assert returns(1, 2, 1)  # use 1 still open: the parity is use 0's, so a wait for use 2 sees it over
    assert not returns(2, 2, 1) and not returns(2, 2, 2) and returns(2, 2, 3)


@pytest.mark.parametrize("name", ["hs_fp4_mla.cu", "hs_sparse_mla.cu"])
def test_mmas_in_flight_are_waited_for(name):
    """Block n - 1's MMAs are issued once those of block n - 1 - NT are over, so up to NT blocks are in flight
    when a CTA gives up; MMAs end in the order in which they were issued."""
    text = source(name)
    in_flight = number(text, "NT")
    waits = re.findall(r"pipe_wait\(&?bs\.(\w+), (\w+), n - 1, abort\)", give_up(text))
    assert len(waits) == 2  # the S-CTA's and the O-CTA's
    for ring, depth in waits:
        depth = number(text, depth)
        for n in range(1, 40):
            for over in range(max(0, n - in_flight), n):
                assert not returns(depth, n - 1, over), f"{ring}: back with {n - over} of {n} blocks' MMAs in flight"
            assert returns(depth, n - 1, n)
