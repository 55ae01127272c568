"""Rules that the sources of the paged cache's append, page moves and prompt
attention keep (CPU)."""
import re

import pytest

from decode_step_gb300.build import CSRC


@pytest.mark.parametrize("name", ["kv_append.cu", "kv_pages.cu", "prompt_attn.cu"])
def test_no_read_only_loads(name):
    """These kernels may start while the kernel before them still writes tables,
    contexts and rows: nothing of theirs is read through the read-only path, by
    an instruction or by the compiler's leave."""
    lines = [x for x in (CSRC / name).read_text().splitlines()
             if re.search(r"__ldg\b|ld\.global\.nc|\bconst\b[^,()]*__restrict__", x)]
    assert not lines, lines


@pytest.mark.parametrize("name", ["kv_append.cu", "kv_pages.cu", "prompt_attn.cu"])
def test_dependents_may_start_only_behind_the_wait(name):
    """A kernel that reads a table before its own wait may stand behind one of
    these in a chain whose first kernel writes the table: it must not start before
    that one has finished, so each kernel waits before it lets others start.
    (The append that reads pinned memory waits last: it stands at the head of a step.)"""
    text = (CSRC / name).read_text()
    kernels = re.split(r"__global__", text)[1:]
    assert kernels
    for k in kernels:
        allow, wait = k.find("pdl_allow_dependents();"), k.find("pdl_wait_prerequisites();")
        assert wait >= 0 and (allow < 0 or wait < allow)
