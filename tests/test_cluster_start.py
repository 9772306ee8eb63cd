"""Distributed shared memory may be accessed only once the block that owns it
has started.  What orders that cannot be seen from results (a block that is
late by a microsecond is rare), so this reads the kernels' source: in a
function with stores to another block's shared memory every thread arrives at
the cluster's barrier first, and waits at it before the first such store."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dfa_parsing_delimiter_gb300", "csrc")


def functions_with_remote_stores(name):
    """Top-level definitions (they end with a brace in the first column)."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return [d for d in re.split(r"(?m)^\}", text) if "st.shared::cluster" in d]


@pytest.mark.parametrize("name", ["pp_grammar.cu", "pp_embed.cu"])
def test_blocks_have_started_before_remote_stores(name):
    found = functions_with_remote_stores(name)
    assert found
    for body in found:
        store = body.index("st.shared::cluster")
        arrive, wait = body.find("cluster_arrive("), body.find("cluster_wait(")
        assert 0 <= arrive < wait < store
