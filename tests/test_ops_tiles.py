"""The attention kernels' direct loads to shared memory, without a GPU: the bytes
they fetch (zo_tile.h, compiled for the host under the sanitizers), and that their
instructions leave the range check to the lane's offset."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_sharded_mixed_step_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_loads_stay_inside_their_rows(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not found")
    exe = str(tmp_path / "tile_checks")
    subprocess.run([HIPCC, "--cuda-host-only", "-x", "hip", "-O1", "-g", "-std=c++17",
                    "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                    "-Xarch_host", "-fno-sanitize-recover=all", "-I", CSRC,
                    os.path.join(ROOT, "tests", "sanitize", "tile_checks.cpp"), "-o", exe],
                   check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1"))
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr[-4000:]


def test_loads_that_may_end_early_have_no_scalar_offset():
    """The descriptors of start_near end with the last row that is there: a part of the
    offset that the range check might not count would reach past it."""
    text = open(os.path.join(CSRC, "zo_attn.h")).read()
    body = re.search(r"void start_near\(.*?\n  \}\n", text, re.S).group(0)
    calls = set(re.findall(r"lds_load\w+", body))
    assert calls
    for name in calls:
        forms = re.findall(r"void %s\([^)]*u32x4 buffer.*?\n\}\n" % name, text, re.S)
        assert forms and all(re.search(r"%2, 0 offen lds", x) for x in forms), name
