"""The order of the prompt kernel's MMAs.

S of a key tile and PV of an earlier one have different accumulators, so nothing but a barrier orders
them; S overwrites the columns in which that PV reads P."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "int4_quantized_paged_gb300", "csrc")


def test_scores_wait_for_the_weights_that_they_replace():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "prompt.cu")).read())
    roles = text[text.index("warp == C::MMA_S || warp == C::MMA_PV"):]
    pv = roles.index("} else {\n          if constexpr (C::QTM) x += 2;")
    s, pv = roles[roles.index("if (scores) {"):pv], roles[pv:roles.index("umma_commit(&o_full")]
    # S: the wait, its result, then the MMAs
    parts = [r"if \(u >= SB\) go = wait\(&pv_done\[j \* SB \+ sb\], \(uint32_t\)\(\(u / SB - 1\) & 1\)\);",
             r"if \(!go\) continue;", r"umma_tmem_a\(td", r"umma_commit\(&s_full"]
    at = [re.search(x, s).start() for x in parts]
    assert at == sorted(at) and len(re.findall(r"umma(_tmem_a)?\(", s)) == 2
    # PV: each tells, behind its MMAs
    assert "pv_done" not in s[at[1]:]
    assert re.search(r"umma_commit\(&pv_done\[j \* SB \+ sb\]\);\s*if \(last\)", pv)
    assert max(m.start() for m in re.finditer(r"umma_tmem_a\(", pv)) < pv.index("umma_commit(&pv_done")
