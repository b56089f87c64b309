"""Copies to shared memory that a thread issues and then reads itself: the compiler has to keep its reads and writes of memory on
their side of the copy, the commit and the wait. It does so where the inline assembly says that it touches memory."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_grouped_expert_gb300", "csrc")


def statements(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.findall(r"asm volatile\((.*?)\);", text, re.S)


@pytest.mark.parametrize("name,copies", [("common.cuh", 1), ("attention.cu", 2)])
def test_copies_that_the_same_thread_reads_touch_memory(name, copies):
    found = [s for s in statements(name) if "cp.async" in s]
    assert sum("[%0], [%1]" in s for s in found) == copies
    for s in found:
        assert s.rstrip().endswith('"memory"'), s


def test_waits_and_commits_touch_memory():
    found = [s for s in statements("common.cuh") if "cp.async.commit_group" in s or "cp.async.wait_group" in s]
    assert len(found) == 2
    for s in found:
        assert s.rstrip().endswith('"memory"'), s
