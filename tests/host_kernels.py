"""Compiles a tensor-core kernel's source for the host (tests/cuda_host/tc_emu)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "gated_delta_rule_132_b200", "csrc")
HEADERS = ("kda_attn.cuh", "kda_attn_rows.cuh", "kda_attn_tc.cuh", "kda_internal.cuh")
_STRING = r'"(?:[^"\\]|\\.)*"'
_ASM = re.compile(r'\basm\s*(?:volatile\s*)?\((?:[^()"]|%s|\((?:[^()"]|%s)*\))*\);' % (_STRING, _STRING))
_LAUNCH = re.compile(r"(\w+(?:<[^<>;]*>)?)<<<(.+?)>>>\(", re.S)


def _asm(m):
    text = m.group(0)
    part = re.search(r'"bar\.sync (\d+), (\d+);"', text)
    if part:
        return f"emu::part_sync({part[1]}, {part[2]});"
    return "" if "griddepcontrol" in text else "emu::absent();"


def for_host(text):
    """The source with launches and inline PTX under the emulation's names."""
    return _LAUNCH.sub(r"emu::launch(\1, \2, ", _ASM.sub(_asm, text))


def build(folder, kernels, driver):
    """The library of `driver` (tests/cuda_host) with the sources that it includes."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not available")
    emu = os.path.join(HERE, "cuda_host", "tc_emu")
    # all beside one another: quoted includes are looked for there first
    for f in os.listdir(emu):
        shutil.copy(os.path.join(emu, f), folder)
    for f in ("attn_host.h", driver):
        shutil.copy(os.path.join(HERE, "cuda_host", f), folder)
    for name in kernels + HEADERS:
        with open(os.path.join(CSRC, name)) as f:
            (folder / name).write_text(for_host(f.read()))
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    so = str(folder / (driver + ".so"))
    subprocess.run([gxx, "-O2", "-fno-strict-aliasing", "-std=c++17", "-w", "-fPIC", "-shared", "-I", cuda, "-I",
                    os.path.join(ROOT, "include"), "-o", so, str(folder / driver)], check=True)
    return ctypes.CDLL(so)
