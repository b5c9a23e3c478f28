"""What the rescoring kernels' sources have to keep about waits.  Neither a CTA
of a cluster that starts late nor a wait that gives up can be made to happen
without harm, so they are read from the source here, and not run."""
import re

import pytest

from tests.test_kernel_waits import kernels

WAITED = re.compile(r"barrier_wait\(|\bcl\.sync\(\)")


@pytest.mark.parametrize("name,kernel", [("wfst_score.cu", "score_kernel"), ("wfst_lowrank.cu", "lowrank_kernel")])
def test_a_cluster_meets_before_its_memory_is_shared(name, kernel):
    body = kernels(name)[kernel]
    assert "this_cluster" in body
    waited, remote = WAITED.search(body), re.search("map_shared_rank", body)
    assert remote and waited and waited.start() < remote.start()


@pytest.mark.parametrize("name", ["wfst_score.cu", "wfst_lowrank.cu", "wfst_prefix.cu"])
def test_no_warp_instruction_stands_behind_a_condition(name):
    """``a && f_sync(all lanes)`` leaves out the lanes that `a` leaves out, and the others wait for them."""
    import os
    from tests.test_kernel_waits import CSRC
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for statement in re.split(r"[;{}]", src):
        m = re.search(r"(&&|\|\||\?)[^,]*__\w+_sync\(", statement)
        assert not m, statement


def test_a_wait_that_gave_up_leaves_nothing_on_its_way():
    body = re.sub(r"\s+", " ", kernels("wfst_prefix.cu")["prefix_kernel"])
    # copies: only into slots that were waited for, and all of them are waited for at the end
    assert body.index("room(r, item); if (!good) break;") < body.index("copy(r, item, k, &k_map")
    assert "room(r, item + 1); if (good) copy(r, item + 1, k, &v_map" in body
    drain = body.index("if (!wait_bar(bar(sh.full[r * R + i % R]), i / R & 1)) break;")
    # products: none after a wait gave up, and a last commit that is waited for whatever `good` says
    assert len(re.findall(r"good = __all_sync\(0xffffffffu, good\); if \(!good\) (?:return|continue); tmem_after\(\);", body)) == 2
    done = body.index("commit(one, bar(sh.done[j])); good = wait_bar(bar(sh.done[j]), 0) && good;")
    assert drain < done < body.index("tcgen05.dealloc")
