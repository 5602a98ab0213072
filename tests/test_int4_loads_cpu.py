"""The order of the loads in the built stages of the INT4 kernel of many rows.

A stage begins with a wait for all but the last so many loads: right only while
every stage issues its copies of x, then of codes, then the loads of scales.  To
the compiler the last are independent of the others, and it has exchanged them;
values do not show that while other waits happen to stand nearby.  So this reads
the device assembly of the source (no GPU needed)."""
import os
import re
import shutil
import subprocess

import pytest

from quantized_moe_router_amd import build

SOURCE = os.path.join(build.PKG, "csrc", "int4_linear.hip")
COPY = re.compile(r"buffer_load_dwordx4 \S+ (s\[\d+:\d+\]).* lds")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if shutil.which(build.HIPCC) is None:
        pytest.skip("needs hipcc")
    out = tmp_path_factory.mktemp("asm") / "int4_linear.s"
    subprocess.run([build.HIPCC, *build.FLAGS, "-I", os.path.join(build.ROOT, "include"), "-I",
                    os.path.dirname(SOURCE), "-S", "--cuda-device-only", SOURCE, "-o", str(out)], check=True,
                   stderr=subprocess.DEVNULL)
    found, lines = {}, None
    for line in out.read_text().split("\n"):
        if re.match(r"_Z\w+:", line):
            m = re.search(r"int4_tile_kernelILi(\d+)ELi(\d+)E", line)
            lines = found.setdefault((int(m[1]), int(m[2])), []) if m else None
        if lines is not None:
            lines.append(line)
    return found


@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("tiles", [4, 6])   # of 32 rows, at most
def test_order_of_a_stage(kernels, group, tiles):
    lines = kernels[group, tiles]
    copies_x, scales, deep = tiles, 128 // group, tiles <= 4   # 512 threads: 32 rows of 256 bytes a copy
    in_flight = copies_x + 2 + 2 * scales if deep else 2 + scales
    codes = next(m[1] for m in map(COPY.search, lines) if m)   # the first copies are of codes
    stages, stage = [], None
    lines = [l for l in lines if l.strip() and not l.strip().startswith((";", "."))]
    for line, behind in zip(lines, lines[1:]):
        # a stage's own wait and its barrier (the compiler's waits elsewhere may have the same count)
        if f"s_waitcnt vmcnt({in_flight}) lgkmcnt(0)" in line and "s_barrier" in behind:
            stage = []
            stages.append(stage)
        elif stage is not None and len(stage) < copies_x + 2 + scales:
            m = COPY.search(line)
            if m:
                stage.append("codes" if m[1] == codes else "x")
            elif "global_load" in line:
                stage.append("scales")
    # stages of one to `tiles` row tiles, three or six of them to a turn of the loop
    assert len(stages) >= (3 if deep else 6) * tiles
    for stage in stages:
        assert stage == ["x"] * copies_x + ["codes"] * 2 + ["scales"] * scales
