"""The LDS-poison build (build variant "poison") fills what its kernels use: each kernel that has LDS has more LDS
writes or more barriers there than in the library (a fill is a loop and, but for a wave's own LDS, a barrier; the
library's own writes may be unrolled further).  On the CPU: the objects are disassembled, not run."""
import os
import re
import subprocess

import pytest

import test_isa_hazards as isa
from lds_staged_matrix_amd import build

READELF = os.path.join(isa.LLVM, "llvm-readelf")
UNITS = [os.path.splitext(s)[0] for s in build.SOURCES]


def kernels(obj, tmp_path):
    """{kernel: (bytes of LDS, LDS writes, barriers)} of the gfx950 code in an object."""
    fat, co = tmp_path / "fat.bin", tmp_path / "co.o"
    subprocess.run(["objcopy", "-O", "binary", "--only-section=.hip_fatbin", obj, str(fat)], check=True)
    subprocess.run([isa.BUNDLER, "--unbundle", "--type=o", f"--input={fat}", "--targets=hipv4-amdgcn-amd-amdhsa--gfx950",
                    f"--output={co}"], check=True)
    notes = subprocess.run([READELF, "--notes", str(co)], check=True, capture_output=True, text=True).stdout
    lds = {}
    for entry in notes.split("- .agpr_count")[1:]:
        name = re.search(r"\.symbol:\s+'?([^'\s]+)\.kd'?", entry)[1]
        lds[name] = int(re.search(r"\.group_segment_fixed_size:\s+(\d+)", entry)[1])
    writes, barriers, name = dict.fromkeys(lds, 0), dict.fromkeys(lds, 0), None
    text = subprocess.run([isa.OBJDUMP, "-d", "--mcpu=gfx950", str(co)], check=True, capture_output=True, text=True).stdout
    for line in text.splitlines():
        start = re.match(r"[0-9a-f]+ <(\S+)>:", line)
        if start:
            name = start[1] if start[1] in lds else None
        elif name:
            writes[name] += line.lstrip().startswith("ds_write")
            barriers[name] += line.lstrip().startswith("s_barrier")
    return {k: (lds[k], writes[k], barriers[k]) for k in lds}


@isa.needs_tools
@pytest.mark.parametrize("unit", UNITS)
def test_every_kernel_with_lds_is_poisoned(unit, tmp_path):
    paths = [os.path.join(build.OBJ_DIR, unit + s + ".o") for s in ("", "_poison")]
    if not all(map(os.path.exists, paths)):
        pytest.skip("library objects not built")
    plain, poison = (kernels(p, tmp_path) for p in paths)
    assert plain and plain.keys() == poison.keys()
    bare = [k for k, (size, writes, barriers) in poison.items() if size > 0 and writes <= plain[k][1] and barriers <= plain[k][2]]
    assert not bare, bare
