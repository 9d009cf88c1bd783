"""CPU: what the sources of the attention kernels say of their loads from tensor memory.  The registers of an issued
load are written asynchronously: a move by the compiler between the load and its wait would read them too early, so
both stand in one statement."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_weight_only_nvfp4_gb300", "csrc")


def _source(name):
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", src, flags=re.S))


@pytest.mark.parametrize("name", ["attend.cu", "attend.cuh", "attend_row.cu", "attend_tile.cu"])
def test_a_load_waits_in_its_own_statement(name):
    src = _source(name)
    for statement in re.findall(r"asm volatile\((.*?)\);", src, flags=re.S):
        if "tcgen05.ld." in statement:
            assert "tcgen05.wait::ld" in statement, statement
        assert "tcgen05.wait::ld" not in statement or "tcgen05.ld." in statement, statement
    # the pair of helpers that leaves a load under way is for straight-line code
    assert not re.search(r"\btmem_ld32_issue\b|\btmem_ld_wait\b", src)


def test_the_shared_helper_waits_in_its_own_statement():
    body = re.search(r"void tmem_ld32\(.*?\n}", _source("tc.cuh"), flags=re.S).group(0)
    assert "tcgen05.wait::ld" in body and body.count("asm volatile") == 1
