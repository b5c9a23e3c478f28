"""What the second-pass kernels' sources have to keep about waits.

Shared memory of another CTA may be touched once that CTA runs, which a
cluster barrier says.  A kernel that goes without it works until the day a CTA
of the cluster starts late.  A kernel whose wait gave up starts no more copies
and products and waits for those that it started.  Neither can be made to
happen without harm, so both are read from the source here, and not run."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "wfst_beam_search_gb300", "csrc")

# a cluster barrier that is over; what reaches into another CTA's shared memory, itself or in what it calls
WAITED = re.compile(r"barrier_wait\(|\bcl\.sync\(\)|\bd\.sync\(\)")
REMOTE = re.compile(r"map_shared_rank|\bd\.(?:leave|at|cluster_sum|gather|find_bin|template find_bin|select|select_slow)\b")


def kernels(name):
    """{kernel: its body without comments} of a source file."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    found = {}
    for m in re.finditer(r"__global__[^;{]*?(\w+)\(const Args a[^{]*\{", src):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(src[i], 0)
            i += 1
        found[m.group(1)] = src[m.end():i]
    return found


@pytest.mark.parametrize("name,kernel", [("wfst_sample.cu", "sample_kernel"), ("wfst_matvec.cu", "matvec_wide")])
def test_a_cluster_meets_before_its_memory_is_shared(name, kernel):
    body = kernels(name)[kernel]
    assert "this_cluster" in body
    waited, remote = WAITED.search(body), REMOTE.search(body)
    assert remote and waited and waited.start() < remote.start()


def test_a_wait_that_gave_up_leaves_nothing_on_its_way():
    body = re.sub(r"\s+", " ", kernels("wfst_matvec.cu")["matvec_wide"])
    # what is started: only while no wait gave up, and counted
    assert len(re.findall(r"elected\(\)", body)) == 2
    starts = [m.end() for m in re.finditer(r"if \(elected\(\) && good\) \{ issued = i \+ 1;", body)]
    assert len(starts) == 2
    # what is waited for behind either loop: all that was started, whatever `good` says
    for start, bar, depth in zip(starts, ("filled", "through"), ("S", "2")):
        m = re.search(r"for \(int i = issued > %s \? issued - %s : 0; i < issued; i\+\+\) good = wait_bar\(%s\(" %
                      (depth, depth, bar), body)
        assert m and m.start() > start
        assert body.index("tcgen05.dealloc") > m.start()
