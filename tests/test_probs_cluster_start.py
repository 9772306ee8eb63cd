"""Blocks of a cluster have started before another reaches into their shared memory:
what orders the two in pp_probs.cu shows in the source alone."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dfa_parsing_delimiter_gb300", "csrc")
REMOTE = r"\b(?:put|there|remote_f|remote_u|write_cut|cut_of_all|add_up|digit_of)\("  # accesses, and what makes them


def bodies():
    with open(os.path.join(CSRC, "pp_probs.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = {}
    for part in re.split(r"(?m)^\}", text):
        head = re.search(r"\b(\w+)\((?:Shared& sh|const ProbArgs a)[^{]*\{", part)
        if head:
            found[head.group(1)] = part[head.end():]
    return found


def test_arrivals_and_waits_before_remote_accesses():
    found = bodies()
    assert {"plain_kernel", "cut_kernel", "long_kernel", "digit_of"} <= set(found)
    for name in ("plain_kernel", "cut_kernel"):
        body = found[name]
        first = re.search(REMOTE, body).start()
        assert 0 <= body.find("cluster_arrive()") < body.find("cluster_wait()") < first, name
    # in this one each remote access comes behind a barrier of the whole cluster
    sync = found["digit_of"].find("cluster_sync()")
    assert 0 <= sync < re.search(r"\bremote_u\(", found["digit_of"]).start()
    body = found["long_kernel"]
    own = re.search(r"\b(?:put|there|remote_f|remote_u)\(", body).start()
    assert 0 <= body.find("cluster_sync()") < own


def test_no_block_ends_before_others_have_read_it():
    """After the last read of another block's memory comes a barrier of the cluster;
    stores into it are made before one, and read from a block's own memory."""
    found = bodies()
    body = found["long_kernel"]
    last = [m.end() for m in re.finditer(r"\bremote_[fu]\(", body)][-1]
    assert "cluster_sync()" in body[last:]
    for name in ("plain_kernel", "cut_kernel"):
        body = found[name]
        last = [m.end() for m in re.finditer(r"\bput\(", body)][-1]
        assert re.search(r"\b(?:ppl::cluster_sync|all_sync<THREADS>)\(\)", body[last:]), name
        assert not re.search(r"\bremote_[fu]\(", body), name
