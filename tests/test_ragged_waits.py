"""How the packed attention's warps wait, read from its source: where a whole warp goes on together (the MMA warp, the
softmax warps, the line's warp), it waits by wait_warp, which has one answer for all lanes; waits of one lane stand
where one lane is alone."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "streaming_kv_cache_duo_gb300",
                    "csrc")


def _roles():
    """Source of each role of attn_ragged_kernel, without comments."""
    with open(os.path.join(CSRC, "attn_ragged.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernel = text[text.index("attn_ragged_kernel(const"):text.index("merge_ragged_kernel(const")]
    line, rest = kernel.split("} else if (warp == kWarpZero) {")
    line = line[line.index("if (warp == kWarpLine) {"):]
    zero, rest = rest.split("} else if (warp == kWarpTma) {")
    tma, rest = rest.split("} else if (warp == kWarpMma) {")
    mma, softmax = rest.split("setmaxnreg.inc", 1)
    return dict(line=line, zero=zero, tma=tma, mma=mma, softmax=softmax)


def _body(text, start):
    """The block in braces that follows `start`."""
    at = text.index("{", text.index(start))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(start)


def _one_lane(text):
    """Blocks that one elected lane runs."""
    out, at = [], 0
    while (at := text.find("if (elect_one()) {", at)) >= 0:
        out.append(_body(text[at:], "if (elect_one())"))
        at += 1
    return out


def test_the_helpers_of_whole_warps_wait_together():
    roles = _roles()
    assert re.fullmatch(r"\{\s*return wait_warp\([^;]*\);\s*\}", _body(roles["mma"], "auto ready ="))
    meet = _body(roles["softmax"], "auto meet =")
    assert "wait_warp(bar," in meet and "wait_for(" not in meet
    for name in ("k_ready", "v_ready"):
        assert re.fullmatch(r"\{\s*return ready\([^;]*\);\s*\}", _body(roles["mma"], f"auto {name} ="))


def test_waits_of_one_lane_stand_where_it_is_alone():
    roles = _roles()
    assert "wait_for(" not in roles["line"] and "wait_for(" not in roles["softmax"] and "wait" not in roles["zero"]
    # the producer is one lane
    assert re.match(r"\s*if \(lane == 0\) \{", roles["tma"]) and "wait_warp(" not in roles["tma"]
    # the MMA warp: the last wait before its memory is given up, by the lane that committed
    alone = _one_lane(roles["mma"])
    assert sum(b.count("wait_for(") for b in alone) == roles["mma"].count("wait_for(") == 1


def test_no_whole_wait_is_in_a_branch_of_one_lane():
    roles = _roles()
    for name in ("mma", "softmax", "line"):
        for block in _one_lane(roles[name]):
            assert not re.search(r"\b(ready|k_ready|v_ready|meet|wait_warp|rows_to_use)\(", block), block
        for block in re.findall(r"if \([^;{]*lane == 0[^;{]*\) (\{[^}]*\}|[^{;]*;)", roles[name]):
            assert not re.search(r"\b(ready|meet|wait_warp)\(", block), block


def test_single_looks_are_voted_on():
    """A look at a barrier by every lane for itself: its answer is used through a vote only."""
    mma = _roles()["mma"]
    looks = re.findall(r"const bool (\w+) = [^;]*mbar_try_wait\(", mma)
    assert looks and mma.count("mbar_try_wait(") == len(looks)
    votes = " ".join(re.findall(r"__all_sync\(([^;]*)\);", mma))
    for name in looks:
        assert re.search(rf"\b{name}\b", votes)
