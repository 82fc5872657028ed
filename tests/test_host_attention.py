"""The attention operators' host layer under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: the library's
sources compiled for the host alone, launches recorded instead of run (as tests/test_host_sanitized.py), driven by
tests/host/attn_check.cpp over workspaces, grids, empty axes and failed launches."""

from __future__ import annotations

import os
import re
import subprocess

import pytest

from test_host_sanitized import HOST, SAN_HOST, SAN_LINK, _clangxx, _run
from tiled_genome_diffusion_amd import build as libbuild


@pytest.fixture(scope="module")
def attn_check_exe(tmp_path_factory):
    work = str(tmp_path_factory.mktemp("attn_check"))
    inc = ["-I", os.path.join(libbuild.ROOT, "include"), "-I", libbuild.CSRC, "-I", HOST]
    common = ["-O1", "-g", "-std=c++17", "-ffp-contract=off"]
    objs = []
    names = ("api.hip", "step.hip", "chain.hip", "seam.hip", "mds.hip", "stitch.hip", "api_attn.hip", "attn_fwd.hip",
             "attn_bwd.hip", "norm_rope.hip")
    for s in [os.path.join(libbuild.CSRC, n) for n in names] + [os.path.join(HOST, "hip_stub.cpp")]:
        o = os.path.join(work, os.path.basename(s) + ".o")
        _run([libbuild.hipcc(), "-x", "hip", "--offload-host-only", *common, *SAN_HOST, *inc, "-c", s, "-o", o], work)
        objs.append(o)
    o = os.path.join(work, "attn_check.o")
    _run([_clangxx(), *common, *SAN_LINK, *inc, "-I", "/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", "-c",
          os.path.join(HOST, "attn_check.cpp"), "-o", o], work)
    objs.append(o)
    syms = set()
    for obj in objs:
        syms.update(re.findall(r"\b(__hip_fatbin_\w+)", _run(["nm", "-u", obj], work).stdout))
    stub_c = os.path.join(work, "fatbin_stub.c")
    with open(stub_c, "w") as f:
        f.writelines(f"const char {s}[16] = {{0}};\n" for s in sorted(syms))
    o = os.path.join(work, "fatbin_stub.o")
    _run([_clangxx(), "-x", "c", "-c", stub_c, "-o", o], work)
    exe = os.path.join(work, "attn_check")
    _run([_clangxx(), *SAN_LINK, "-o", exe, *objs, o], work)
    return exe


def test_attention_host_layer_clean_under_asan_and_ubsan(attn_check_exe):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([attn_check_exe], capture_output=True, text=True, env=env, timeout=600)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "host checks passed" in res.stdout
    assert "runtime error" not in res.stderr and "AddressSanitizer" not in res.stderr
