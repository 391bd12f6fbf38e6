"""What the built kernels' own metadata says (the code objects inside libper.so)."""
import os
import re
import subprocess

import pytest
import yaml

from sum_tree_sampling_amd import build, per

LLVM = "/opt/rocm/llvm/bin"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{kernel: bytes of static LDS} of libper.so's gfx950 code objects."""
    if not os.path.exists(per.LIB_PATH):
        build.build()
    d = tmp_path_factory.mktemp("co")
    fat = str(d / "fat")
    subprocess.run([LLVM + "/llvm-objcopy", "--dump-section", ".hip_fatbin=" + fat, per.LIB_PATH, str(d / "rest")],
                   check=True)
    data = open(fat, "rb").read()
    out = {}
    starts = [m.start() for m in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", data)]
    for k, at in enumerate(starts):  # one bundle per source
        one = str(d / ("b%d" % k))
        with open(one, "wb") as f:
            f.write(data[at:starts[k + 1] if k + 1 < len(starts) else len(data)])
        subprocess.run([LLVM + "/clang-offload-bundler", "--type=o", "--unbundle", "--input=" + one,
                        "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", "--output=" + one + ".co"], check=True)
        notes = subprocess.run([LLVM + "/llvm-readelf", "--notes", one + ".co"], capture_output=True, text=True,
                               check=True).stdout
        meta = yaml.safe_load(notes.split("---", 1)[1].rsplit("...", 1)[0])
        out.update((q[".name"], q[".group_segment_fixed_size"]) for q in meta["amdhsa.kernels"])
    return out


def test_dynamic_lds_is_aligned(kernels):
    """The bitmap of the distillation's kernels is cleared 16 bytes at a time, and lies
    behind their static LDS."""
    found = {n: v for n, v in kernels.items() if re.search(r"distill_(row|part|grad|wave)_kernel", n)}
    assert len(found) > 50
    assert not {n: v for n, v in found.items() if v % 16}
