"""Reads the host code: what allocates there is caught, so that no C++ exception leaves a C entry point."""
import os
import re

from fp8_block_scaled_09_b200 import build as fp8bq_build


def test_containers_grow_only_where_a_failure_is_caught():
    with open(os.path.join(fp8bq_build.CSRC, "fp8bq.cu")) as f:
        text = re.sub(r"//.*", "", f.read())
    grows = [m.start() for m in re.finditer(r"\.(emplace|insert|push_back|resize|reserve)\w*\(|\bnew\b(?!>)", text)]
    assert grows
    for at in grows:
        before = text[:at]
        assert before.count("try {") > 0
        opened = before.rindex("try {")
        assert "}" not in text[opened + 5:at] and "catch (const std::bad_alloc &)" in text[at:at + 200]
    assert "throw " not in text and ".at(" not in text
