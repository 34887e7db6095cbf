"""The bounded waits of the experts' products, by their source: lanes may see a
wait run out at different times, so where its result steers a warp the warp agrees
on it (__all_sync) before anything that takes all its lanes."""

import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_precision_gemm_gb300", "csrc",
                   "experts.cu")


def test_no_lane_leaves_its_warp_by_itself():
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    assert not re.findall(r"if \(!\s*mbar_\w+\(", text)
    # a result is voted on, or is one lane's: of a branch that only lane 0 or the issuing lane takes
    for use in re.finditer(r"(\w+) = (mbar_(?:wait|poll|spin\w*)\()", text):
        name, at = use.group(1), use.start()
        assert f"__all_sync(0xffffffffu, {name})" in text[at:at + 600], text[at:at + 120]


def test_every_wait_is_bounded():
    text = open(SRC).read()
    for use in re.finditer(r"mbar_(?:wait|poll|spin\w*)\((.*?)\);", text, re.S):
        assert "timeout_ns" in use.group(1), use.group(0)
