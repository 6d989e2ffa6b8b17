"""The waits on the path by which an attention kernel gives up (a bounded wait ran out): its copies and MMAs
are over before shared and tensor memory are freed. A model of mbarrier phases on the CPU, with the rings, depths and tiles
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


@pytest.mark.parametrize("name,rings", [("hs_fp4_mla.cu", ["q_raw"]), ("hs_sparse_mla.cu", ["q_raw", "raw_full"])])
def test_copies_in_flight_are_waited_for(name, rings):
    """Every ring on which copies of the copy engine complete."""
    text = source(name)
    copies = re.findall(r"complete_tx::bytes \[%0\].*?:\s*\"memory\"", text, re.S)
    assert sorted({re.search(r"smem_u32\(&bs\.(\w+)", c).group(1) for c in copies}) == sorted(rings)
    for ring in rings:
        assert re.search(r"pipe_wait\(&?bs\.%s\b" % ring, give_up(text)), ring


def test_the_gathers_last_uses_are_the_ones_waited_for():
    """Half-block k is requested once half-block k - NR has been read, so the last NR of those requested may be on
    their way, in any order."""
    text = source("hs_sparse_mla.cu")
    ring = number(text, "NR")
    assert "for (int k = m >= NR ? m - NR : 0; k < m; ++k) pipe_wait(bs.raw_full, NR, k, abort);" in give_up(text)
    for m in range(1, 30):
        for k in range(max(0, m - ring), m):
            assert not returns(ring, k, k)  # all but k itself are there
            assert returns(ring, k, k + 1)


@pytest.mark.parametrize("name", ["hs_fp4_mla.cu", "hs_sparse_mla.cu"])
def test_a_cta_that_gave_up_outlives_its_partners_stores(name):
    """A CTA that gave up takes no more P: the stores that its partner has issued complete on no wait of its own,
    so it stays, after the cluster's last barrier, for longer than any store takes."""
    text = source(name)
    end = text[text.index("tcgen05.dealloc"):]
    assert re.search(r"cluster_sync_all\(\);\s*if \(!ok && tid == 0\) stay\(\);\s*}", end)
    header = source("hs_tcgen05.cuh")
    assert int(re.search(r"kStayNs = (\d+)ull", header).group(1)) >= 1000000
