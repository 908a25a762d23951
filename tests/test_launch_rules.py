"""Kernels launched with programmatic serialization: what they may touch before
they have waited for the kernels in front of them.  Read from the sources."""
import glob
import os
import re

import pytest

import sparse_attention_top_idx_gb300 as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")
WAIT = 'asm volatile("griddepcontrol.wait;" ::: "memory");'


def waiting_kernels():
    """(file, text from the kernel's head to its wait) of every kernel that waits."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        text = re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S))
        for part in text.split("__global__")[1:]:
            if WAIT in part:
                found.append((os.path.basename(path), part[part.index("{"):part.index(WAIT)]))
    return found


def test_every_programmatic_launch_has_a_kernel_that_waits():
    files = {f.replace(".cuh", "").replace(".cu", "").replace("_kernel", "") for f, _ in waiting_kernels()}
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        if "ProgrammaticStreamSerialization" in open(path).read():
            assert os.path.basename(path).replace(".cu", "") in files, path


@pytest.mark.parametrize("name,head", waiting_kernels(), ids=[f for f, _ in waiting_kernels()])
def test_nothing_in_global_memory_is_read_before_the_wait(name, head):
    """A kernel lets the next one start before it has waited itself, so what
    a kernel reads before its wait may still be written by any kernel in front
    of it (a staged copy of the lengths, say)."""
    assert not re.search(r"__ldg|ld\.global|cp\.async|tma_(tile|load|bulk)|seq_lens|block_table|row_keys|find_item|find_row", head), name
