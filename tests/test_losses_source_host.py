"""What the source of the losses has to keep to where no run may show it."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "linear_recurrence_scan_affine_gb300", "csrc", "loss_rows.cuh")


def test_a_block_whose_wait_ran_out_stays_for_its_cluster():
    # Blocks of a cluster write to one another's shared memory (row statistics, the
    # answers to requests for a row). In order each has had all of it when it ends;
    # after a wait that ran out it may not: its leader lets copies arrive and waits
    # for the others before the block ends.
    src = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    stay = src[src.index("void settle("):]
    stay = stay[:stay.index("\n}")]
    assert stay.index("globaltimer_ns() < until") < stay.index("barrier.cluster.arrive") < \
        stay.index("barrier.cluster.wait")
    body = src[src.index("__device__ __forceinline__ void long_rows("):]
    leader = body[body.index("if (warp == kTeam / 32)"):]
    leader = leader[:leader.index("return;")]
    assert re.search(r"if \(\*abort\) \{[^}]*RLCS_ERR_TIMEOUT[^}]*settle\(ranks\);\s*\}\s*$",
                     leader)
