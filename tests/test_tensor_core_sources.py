"""How the tcgen05 kernels issue and end, read from their sources (no GPU): a commit by itself, away from
the MMAs that it covers, was the one instruction between a warp and the end of a kernel that hung."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_long_context_dsa_b200", "csrc")
MMA = r"\b(?:mma_f8<|mma_ts<|umma_e4m3\(|umma_bf16\(|mma\(std::)"


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def kernels_with_commits():
    return sorted(f for f in os.listdir(CSRC) if f != "common.cuh" and "umma_commit(" in code(f))


def test_the_files_are_found():
    assert {"attention_quant_band.cuh", "attention_quant_tc.cuh", "attention_tc.cuh", "frontend.cuh",
            "gemm_indexer.cuh"} <= set(kernels_with_commits())


@pytest.mark.parametrize("name", kernels_with_commits())
def test_every_commit_stands_behind_mmas(name):
    # in the order of the text: MMAs, then commits, with no wait, loop or other call's wait between them
    last = None
    commits = 0
    for m in re.finditer(MMA + r"|\bumma_commit\(|\bmbar_\w+\(|\bwalk_next\(|\belect_one\(", code(name)):
        t = m.group(0)
        if t == "umma_commit(":
            commits += 1
            assert last == "mma", f"{name}: commit {commits} follows {last}"
        else:
            last = "mma" if re.fullmatch(MMA, t) else t
    assert commits > 0


@pytest.mark.parametrize("name", kernels_with_commits())
def test_an_elected_lane_issues_and_waits_for_its_commits(name):
    text = code(name)
    roles = text.split("elect_one()")
    assert "umma_commit(" not in roles[0], f"{name}: commits by a lane that is not elected"
    for role in roles[1:]:
        # the role's own block, by its braces
        at, depth = role.index("{"), 0
        for end in range(at, len(role)):
            depth += {"{": 1, "}": -1}.get(role[end], 0)
            if depth == 0:
                break
        block = role[at:end]
        targets = {re.sub(r"[\[&].*", "", t.lstrip("&")) for t in re.findall(r"umma_commit\((&?[\w.]+)", block)}
        waited = {re.sub(r"[\[&].*", "", t.lstrip("&")) for t in re.findall(r"commits_done\((&?[\w.]+)", block)}
        assert targets and targets == waited, f"{name}: commits to {targets}, waits for {waited}"
        assert "umma_commit(" not in role[end:]
        # the waits stand behind the last commit
        assert block.rindex("umma_commit(") < block.index("commits_done(")
