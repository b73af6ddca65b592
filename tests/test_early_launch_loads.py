"""Kernels that start while the kernel before them still writes (early_launch.h) may read nothing that it writes through
the non-coherent path, which takes memory to be constant as long as the reading kernel lives: in their sources __ldg and
ld.global.nc stand for rotation tables only. Read from the sources, since a stale line can hardly be provoked."""
import glob
import os
import re

from transformer_attention_02_gb300 import build as B

PAGED = sorted(glob.glob(os.path.join(B.CSRC, "paged_*.cu")) + glob.glob(os.path.join(B.CSRC, "paged_*.cuh")))
NON_COHERENT = r"__ldg\(\s*|ld_global_nc\w*\(\s*|ld\.global\.nc"


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_paged_kernels_read_rotation_tables_alone_that_way():
    assert len(PAGED) >= 5
    reads = 0
    for path in PAGED:
        code = _code(path)
        for m in re.finditer(rf"({NON_COHERENT})(\w*)", code):
            name = m.group(2)
            made = re.findall(rf"\*\s*(?:const\s+)?{name}\s*=\s*([^;]*);", code) if name else []
            at = f"{os.path.basename(path)}: {code[m.start():m.start() + 60]}"
            assert any("p.rope" in x for x in made), at
            reads += 1
    assert reads >= 4                                    # the tables themselves


def test_the_ragged_kernel_reads_its_lengths_plainly():
    code = _code(os.path.join(B.CSRC, "attn_kernel.cuh"))
    body = code[code.index("Lens lens_of("):]
    assert not re.search(NON_COHERENT, body[:body.index("\n}")])
