"""Bounded waits by whole warps, read in the source: the lanes that go on to instructions of a whole warp (loads from
tensor memory, full-mask barriers) decide together whether a wait was given up.  Where each decides for itself, some may
see the abort flag and others the barrier; those that left then wait for the block, the others for them, without end."""
from __future__ import annotations

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_cross_entropy_tmem_gb300", "csrc")


def test_epilogue_of_the_4_bit_logits_gives_up_by_warps():
    src = open(os.path.join(CSRC, "flce_mx_logits.cu")).read()
    epilogue, = re.findall(r"// -+ epilogue\n(.*?)\n  griddep_release\(\);", src, re.S)
    assert "tfull" in epilogue
    # a lane's own wait is only ever what its group of warps votes on
    alone = re.sub(r"group_all\(grp, stage_wait\([^;]*?\)\)", "", epilogue)
    assert "tfull" in alone and "stage_wait" not in alone and "mbar_" not in alone.replace("mbar_arrive", "")
    assert re.search(r"warp_wait\(&sm\.tfull", alone)
    # and that wait is a vote
    vote, = re.findall(r"bool warp_wait\(.*?\n}\n", src, re.S)
    returns = re.findall(r"return (.*?);", vote)
    assert returns == ["true", "__all_sync(0xffffffffu, stage_wait(bar, parity, ctl, status))"]
    assert "if (__all_sync(0xffffffffu, mbar_try_wait(addr, parity))) return true;" in vote
