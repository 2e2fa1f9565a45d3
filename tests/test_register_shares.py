"""Registers that move between the warps of the attention kernel.

setmaxnreg has to be the same instruction for the four warps of a warpgroup. The producer, the two
MMA issuers and an idle warp make up one, so their share is given up before their roles part."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "int4_quantized_paged_gb300", "csrc")


def test_each_warpgroup_moves_its_registers_in_one_place():
    text = open(os.path.join(CSRC, "prefill_ws.cuh")).read()
    roles = text[re.search(r"//\s*=+ roles", text).start():]
    moves = [m.start() for m in re.finditer(r"(give|take)_registers<RL::", roles)]
    branches = []
    for at in moves:
        head = re.findall(r"(?:if|else if) \((warp[^{]*)\) \{", roles[:at])[-1]
        tail = roles[roles[:at].rindex(head):at]
        # nothing between the branch and the move but a comment and the form's test
        body = re.sub(r"//[^\n]*", "", tail[len(head):]).replace(") {", "").split()
        assert body == "if constexpr (RL::SPLIT_REGS)".split()
        branches.append(head)
    assert branches == ["warp >= RL::PROD", "warp >= RL::SOFT", "warp < 4 * nqt"]
