"""Registers that the 4-bit cache write leaves to memory: its kernels of large writes run 32
warps an SM at 64 registers a thread, and rows with a scale a channel lost time to spills when their
quotients went by pairs (int4 952 / 1124 bytes spilled and read back, by pairs 1176 / 1548)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "paged_quantized_kv_gqa_gb300")
# (4-bit format, a scale a channel) of units of 32 positions: bytes stored, bytes loaded
MOST = {("0", "0"): (176, 120), ("0", "1"): (960, 1140), ("1", "0"): (220, 164), ("1", "1"): (920, 1110)}


@pytest.fixture(scope="module")
def spills(tmp_path_factory):
    import importlib.util
    spec = importlib.util.spec_from_file_location("pa_build_for_spills", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    r = subprocess.run([build._nvcc(), *build.ARCH, *build.FLAGS, "-Xptxas", "-v", "-I", build.INCLUDE, "-I", build.CSRC, "-c",
                        os.path.join(build.CSRC, "pa_cache4.cu"), "-o", str(tmp_path_factory.mktemp("o") / "x.o")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    found = {}
    for m in re.finditer(r"cache_append4_kernelILi(\d)ELb(\d)ELi32E[\s\S]*?(\d+) bytes spill stores, (\d+) bytes spill loads",
                         r.stdout + r.stderr):
        found.setdefault(m.group(1, 2), (int(m.group(3)), int(m.group(4))))
    return found


@pytest.mark.parametrize("kernel", sorted(MOST))
def test_spills(spills, kernel):
    assert all(a <= b for a, b in zip(spills[kernel], MOST[kernel])), spills
