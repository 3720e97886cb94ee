"""Rules of the kernels' barriers that hold by their source (CPU only)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "confidence_gated_kv_logit_b200", "csrc")


def test_commits_arrive_at_barriers_of_one_arrival():
    """A commit of products arrives once: a barrier that counts more would never complete by it, and a wait for it
    (the drain of an aborting block, before its tensor memory is freed) would end with products in flight."""
    with open(os.path.join(CSRC, "tree_mma.cu")) as f:
        src = f.read()
    counts = {}
    for name, n in re.findall(r"mbar_init\(&bar\.(\w+)(?:\[\w+\])?, (\w+)\)", src):
        counts[name] = n
    committed = set(re.findall(r"tc_commit\(&bar\.(\w+)", src))
    assert len(committed) >= 5
    assert {name: counts[name] for name in committed} == {name: "1" for name in committed}
