"""The waits of hs_chunk_mla's attention kernel: on the way by which a CTA gives up (a bounded wait ran out), and the parities
that its roles wait on. Models of mbarrier phases on the CPU, with the rings and buffers as the source has them; no GPU path
is made to run out."""
import re

import pytest

from test_give_up_waits import give_up, number, returns, source

NAME = "hs_chunk_mla.cu"


def const(name):
    return number(source(NAME), name)


def test_copies_in_flight_are_waited_for():
    """Every ring on which copies of the copy engine complete, over as many uses as can be in flight."""
    text = source(NAME)
    rings = set(re.findall(r"uint64_t\* bar = &bs\.(\w+)", text))
    assert rings == {"k_full", "v_full"} and len(re.findall(r"mbarrier::complete_tx::bytes \[%0\]", text)) == 3
    end = give_up(text)
    assert "for (int k = m >= 2 * NK ? m - 2 * NK : 0; k < m; ++k) pipe_wait(bs.k_full[k & 1], NK, k >> 1, abort);" in end
    assert "for (int k = m >= NV ? m - NV : 0; k < m; ++k) pipe_wait(bs.v_full, NVF, k, abort);" in end
    nk, nv = const("NK"), const("NV")
    # a slot's part k is requested once that of NK slots before has been read (NV for V): the last ones may be on their way
    for m in range(1, 40):
        for k in range(max(0, m - 2 * nk), m):
            assert not returns(nk, k >> 1, k >> 1) and returns(nk, k >> 1, (k >> 1) + 1)
        for k in range(max(0, m - nv), m):
            assert not returns(2 * nv, k, k) and returns(2 * nv, k, k + 1)


def test_mmas_in_flight_are_waited_for():
    """S: an issuer has one block in flight, whose buffer it took when the block before had been read. P . V: a half block
    on its slot."""
    end = give_up(source(NAME))
    assert "if (ctl.issued[k] > 0) pipe_wait(&bs.s_full[k], 1, ctl.issued[k] - 1, abort);" in end
    assert "if (ctl.issued[k] > 0) pipe_wait(bs.v_free, NV, 2 * (ctl.issued[k] - 1) + k, abort);" in end
    for n in range(1, 40):
        assert not returns(1, n - 1, n - 1) and returns(1, n - 1, n)


def test_a_cta_that_gave_up_outlives_its_partners_stores():
    text = source(NAME)
    end = text[text.index("tcgen05.dealloc"):]
    assert re.search(r"cluster_sync_all\(\);\s*if \(!ok && tid == 0\) stay\(\);\s*}", end)


def test_no_role_of_the_s_cta_waits_at_a_hardware_barrier():
    """A warp that gave up would be missed there. The O-CTA has one, to which its twelve warps come in every unit, whether
    their waits ended well or not."""
    text = source(NAME)
    kernel = text[text.index("chunk_mla_kernel("):text.index("outputs are not valid") if "outputs are not valid" in text else text.index("tcgen05.dealloc")]
    loop = kernel[kernel.index("for (; __all_sync"):kernel.index("__syncthreads_and")]
    assert "sync_n<" not in loop and "sync_or" not in loop and loop.count("sync_and(") == 1
    assert loop.index("sync_and(") > loop.index("const float* alpha_buf")
    assert "if (!ok && warp >= ISSUER) break;" in loop


@pytest.mark.parametrize("depth", [const("NP")])
def test_the_softmax_sees_every_phase_but_one_of_ps_buffers(depth):
    """Block g waits for P . V of block g - NP: its barrier's phase before, of block g - 2 NP, has been waited for by the
    warpgroup of block g - NP, the same as block g - 1's, which is at block g - 1 when block g's has seen m_set."""
    ns = const("NS")
    assert depth == ns + 1
    for g in range(2 * depth, 60):
        assert (g - depth) % ns == (g - 1) % ns


def test_v_s_barriers_are_one_issuers_each():
    """Uses 2 g + nh of a ring of an even number of barriers: an issuer waits on its own ones only, each phase of them."""
    nvf = 2 * const("NV")
    for nh in (0, 1):
        mine = [(2 * g + nh) % nvf for g in range(50)]
        assert {x % 2 for x in mine} == {nh}
        for g in range(50 - nvf // 2):
            assert mine[g] == mine[g + nvf // 2]
