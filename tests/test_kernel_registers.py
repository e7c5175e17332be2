"""The attention kernels of the library built here take no more registers than
the workgroups that their plans count on leave them (a SIMD's 512 over the
waves it is to hold), and spill nothing in their loops."""
import os
import re
import subprocess
import tempfile

import pytest

from test_isa_hazards import LIB, LLVM, _code_objects


@pytest.fixture(scope="module")
def kernels():
    """{name: (VGPRs, scratch bytes)} by the code objects' own notes."""
    if not os.path.exists(LIB):
        pytest.skip("libqgemv.so is not built")
    found = {}
    with tempfile.TemporaryDirectory() as d:
        for i, obj in enumerate(_code_objects(LIB)):
            path = os.path.join(d, "co%d.o" % i)
            with open(path, "wb") as f:
                f.write(obj)
            out = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", path], check=True, capture_output=True, text=True).stdout
            for part in out.split("- .agpr_count:")[1:]:
                get = lambda key: re.search(r"\.%s:\s+(\S+)" % key, part).group(1)  # noqa: E731
                found[get("name")] = (int(get("vgpr_count")), int(get("private_segment_fixed_size")))
    return found


def room(waves):
    return 512 // waves // 8 * 8


def test_requests(kernels):
    seen = 0
    for name, (vgprs, scratch) in kernels.items():
        m = re.search(r"14kv_attn_kernelILb(\d)ELi(\d+)ELi(\d)ELi(\d)ELi(\d)ELNS_6KvModeE(\d)E", name)
        if not m:
            continue
        e4m3, D, NR, RS, W, mode = (int(v) for v in m.groups())
        waves = 2 if NR > 1 or D > 128 or W != 4 else 4 if e4m3 and D == 64 and mode == 0 else 3
        # (12 bytes outside the loops: int8, heads of 128)
        assert vgprs <= room(waves) and scratch <= 16, (name, vgprs, scratch)
        seen += 1
    assert seen >= 60


def test_prefix_rows(kernels):
    seen = 0
    for name, (vgprs, scratch) in kernels.items():
        m = re.search(r"21kv_prefix_rows_kernelILb(\d)ELi(\d+)ELi(\d)ELi(\d)E", name)
        if not m:
            continue
        _, D, NR, W = (int(v) for v in m.groups())
        waves = 3 if D == 64 or (D == 128 and NR == 1) else 2
        assert vgprs <= room(waves) and scratch == 0, (name, vgprs, scratch)
        seen += 1
    assert seen == 10
