"""The kernels of the backward pass, of the rotary axes and of the 8-bit checkpoints start while the kernel before them still
writes: they wait for it before they touch memory, and read nothing that it may write through the non-coherent path (which
stands for rotation tables only). Read from the sources, since a stale line can hardly be provoked."""
import glob
import os
import re

import pytest

from transformer_attention_02_gb300 import build as B

FILES = sorted(f for pattern in ("bwd_*", "rope_axes*", "checkpoint*") for f in glob.glob(os.path.join(B.CSRC, pattern))
               if f.endswith((".cu", ".cuh")))


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_there_are_sources():
    assert len(FILES) >= 9


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_only_rotation_tables_are_read_that_way(path):
    code = _code(path)
    for m in re.finditer(r"__ldg\(([^;]*);|ld_global_nc\w*|ld\.global\.nc", code):
        assert m.group(1) and m.group(1).startswith("p.table"), m.group(0)
    assert "__restrict__" not in code                    # (a restricted const pointer may be read non-coherently)


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_kernels_wait_before_they_read(path):
    """Every kernel but the one that fills a table (an ordinary launch) waits before its first use of its parameters' memory."""
    code = _code(path)
    for m in re.finditer(r"__global__ void (?:__launch_bounds__\([^)]*\)\s*)?(\w+)\(", code):
        if m.group(1) == "axes_table_kernel":
            continue
        body = code[m.end():]
        before = body[body.index("{"):body.index("wait_for_inputs();")]
        assert "__global__" not in before, m.group(1)
        for read in re.findall(r"\bp\.(\w+)", before):
            assert read in ("status", "timeout_ns"), (m.group(1), read)      # (for the waits; neither is of the stream)
