"""Rules that the page kernels' source keeps, and that no run would show broken
(no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "agent_shared_compressed_gb300", "csrc")


def _code(name):
    """The source without its comments."""
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", src, flags=re.S)


@pytest.mark.parametrize("name", ["kvp_pages.cuh", "kvpages_append.cu", "kvpages_attend.cu"])
def test_no_read_only_loads_of_what_may_be_written(name):
    """The page kernels are resident while the kernel before them runs, and read
    what it writes (queries, lengths, table, pages); the writing kernel may also
    turn queries in their own tensor.  None of their loads may be of the kind that
    wants memory nobody writes while the kernel is resident, or that the compiler
    may move above the kernel's wait."""
    assert not re.findall(r"\b__ldg\b|\b__ldc[agsv]\b|\.nc\b|\bld_stream_\w+|\bld_v4_policy\b|__restrict__", _code(name))


def test_refused_pool_attention_waits_for_the_kernel_before_it():
    """Attention over the pool may start while a page write runs.  If it finds
    another pool than the caller described it still ends after that write: what
    comes next in the stream waits for its end only."""
    code = _code("kvpool_attend.cu")
    at = code.index("hdr[0] != POOL_MAGIC")
    refusal = code[at:code.index("return;", at)]
    assert "griddepcontrol.wait;" in refusal
