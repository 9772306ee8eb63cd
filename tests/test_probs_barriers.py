"""What orders the shared memory of a cut's steps shows in the source alone: on no
machine does a late warp have to read another's value."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dfa_parsing_delimiter_gb300", "csrc")
BARRIER = r"\b(?:row_sync<THREADS>|all_sync<THREADS>|__syncthreads|ppl::cluster_sync)\(\)"


def functions():
    """Bodies of pp_probs.cu's functions by name, without comments."""
    with open(os.path.join(CSRC, "pp_probs.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = {}
    for part in re.split(r"(?m)^\}", text):
        for name in ("cut_of_all", "cut_among", "write_cut", "cut_kernel", "plain_kernel"):
            if re.search(r"\b%s\((?:const|P&|Fast)" % name, part):
                found.setdefault(name, part)
    return found


def test_a_function_leaves_wf_with_a_barrier_after_its_last_read():
    """cut_of_all reads wf and returns to cut_kernel, which writes it: a barrier has to
    come after the last read on every way out, the ones that cut_among takes without one too."""
    body = functions()["cut_of_all"]
    reads = [m.end() for m in re.finditer(r"= -?warp_max\(-?sh\.wf\[\d\]\[lane % WARPS\]\);", body)]
    assert len(reads) == 4  # two for the range of all values, two for that of the listed ones
    for at in reads:
        rest = body[at:]
        out = re.search(r"\breturn\b", rest).start()
        barrier = re.search(BARRIER, rest)
        assert barrier and barrier.start() < out, rest[:200]


def test_cut_kernel_writes_wf_only_behind_a_barrier():
    """Between the kernel's own read of wf and its write of the same words: those are
    the other half of the array, or a barrier lies between."""
    body = functions()["cut_kernel"]
    reads = set(re.findall(r"warp_max\(sh\.wf\[(\d)\]", body))
    writes = re.findall(r"sh\.wf\[(\d)\]\[warp\] = s", body)
    assert reads == {"0"} and writes == ["1"]
