"""The traffic figures of the profile summaries: bytes as in dram_traffic.json, sums of
their parts, and the ratio to the algorithmic bytes that those bytes give."""
import glob
import json
import os
import re

import pytest

PROFILES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "profiles")
with open(os.path.join(PROFILES, "dram_traffic.json")) as f:
    TRAFFIC = json.load(f)


def _lines():
    for path in sorted(glob.glob(os.path.join(PROFILES, "*.md"))):
        for line in open(path):
            nums = [int(x.replace(",", "")) for x in re.findall(r"\d{1,3}(?:,\d{3})+", line)]
            ratio = re.search(r"(?<![\d.,])\d\.\d{3}(?!\d)", line)
            if nums and ratio and line.startswith("|"):
                yield os.path.basename(path), line, nums, ratio.group(0)


def test_there_are_ratios_to_check():
    assert len(list(_lines())) >= 8


@pytest.mark.parametrize("name,line,nums,ratio", list(_lines()))
def test_ratio(name, line, nums, ratio):
    if len(nums) >= 4:                               # read, write, their sum, algorithmic
        assert nums[0] + nums[1] == nums[2]
        assert ratio == f"{nums[2] / nums[3]:.3f}"
    else:
        e = next(e for e in TRAFFIC.values() if e["algorithmic_bytes"] in nums)
        assert ratio == f"{e['dram_bytes_per_launch'] / e['algorithmic_bytes']:.3f}"
        text = open(os.path.join(PROFILES, name)).read()
        for key in ("dram_bytes_read", "dram_bytes_write", "dram_bytes_per_launch"):
            assert f"{e[key]:,}" in text
