"""Rules that the tensor-core kernels of the linear-attention prompts keep, read
from their sources: nothing a CTA asked for may arrive after it has left."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_recurrent_lq_b200", "csrc")


@pytest.mark.parametrize("name,role_end", [("lq_linear_pipe.cuh", "k / G, in pieces"), ("lq_linear_state.cuh", "// the keys, then")])
def test_the_issuing_warp_waits_for_every_commit(name, role_end):
    """A tcgen05.commit arrives on a barrier in shared memory at a later time: the
    warp that makes it waits, behind its last product, for all that it made."""
    text = open(os.path.join(CSRC, name)).read()
    made = set(re.findall(r"umma_commit\(&bars->(\w+)", text))
    assert len(made) >= 3
    # the tails of the issuing loops: what stands behind a role's last commit
    tails = ""
    for part in re.split(r"(?=umma_commit\()", text.split(role_end)[0])[1:]:
        tails += part.split("\n", 1)[1]
    waited = set(re.findall(r"(?:landed|wait)\(&bars->(\w+)", tails))
    assert made <= waited, f"{name}: nobody waits for {sorted(made - waited)}"


@pytest.mark.parametrize("name", ["lq_linear_pipe.cuh", "lq_linear_state.cuh"])
def test_the_loading_warp_waits_for_all_its_loads(name):
    """The last loads of every stage are waited for by the warp that asked for
    them, whether or not somebody else still does."""
    text = open(os.path.join(CSRC, name)).read()
    tail = text[text.rindex("tma_load_2d("):]
    loop = re.search(r"for \((?:uint32_t|int) (\w) = (\w) >=? (\w+) \? \2 - \3 : 0u?; \1 < \2; \+\+\1\)\s*wait\(&bars->full\[", tail)
    assert loop and loop.group(3) in ("ST", "kLsStages")


@pytest.mark.parametrize("name", ["lq_linear_pipe.cuh", "lq_linear_state.cuh"])
def test_a_wait_that_gives_up_does_so_for_its_whole_warp(name):
    """Behind a wait stand instructions of whole warps (tensor memory, shuffles): the
    lanes agree on its outcome, also where the phase ends as the first ones give up."""
    text = open(os.path.join(CSRC, name)).read()
    body = re.search(r"auto wait = \[&\]\(uint64_t \*b, uint32_t phase\) \{(.*?)\n    \};", text, flags=re.S).group(1)
    assert re.search(r"ok = __all_sync\(0xFFFFFFFFu, got\) && ok;", body)
    assert "ok = false" not in text
