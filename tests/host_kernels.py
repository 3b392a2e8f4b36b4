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
HEADERS = ("kda_attn.cuh", "kda_attn_rows.cuh", "kda_attn_tc.cuh", "kda_attn_tree.cuh", "kda_internal.cuh")
_LAUNCH = re.compile(r"(\w+(?:<[^<>;]*>)?)<<<(.+?)>>>\(", re.S)


def _end(text, at):
    """Behind the parenthesis that closes the one at `at`."""
    depth, quoted = 0, False
    while True:
        c = text[at]
        if quoted:
            at += c == "\\"
            quoted = c != '"'
        elif c == '"':
            quoted = True
        else:
            depth += (c == "(") - (c == ")")
        at += 1
        if not depth:
            return at


def _asm(text):
    """One asm statement under the emulation's names."""
    part = re.search(r'"bar\.sync (\d+), (?:(\d+);"|%0;"\s*::"n"\((.+)\) : )', text)
    if part:
        return f"emu::part_sync({part[1]}, {part[2] or part[3]});"
    if '"cp.async.cg.shared.global [%0], [%1], 16, %2;"' in text:
        args = [text[m.end() - 1:_end(text, m.end() - 1)] for m in re.finditer(r'"[rl]"\(', text)]
        return f"tc::copy16({', '.join(args)});"
    return "" if "griddepcontrol" in text else "emu::absent();"


def for_host(text):
    """The source with launches, inline PTX and shared memory under the emulation's names."""
    text = text.replace("extern __shared__", "extern").replace("__shared__", "static")
    out, at = [], 0
    for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", text):
        end = text.index(";", _end(text, m.end() - 1)) + 1
        out += [text[at:m.start()], _asm(text[m.start():end])]
        at = end
    return _LAUNCH.sub(r"emu::launch(\1, \2, ", "".join(out) + text[at:])


def build(folder, kernels, *drivers):
    """The library of `drivers` (tests/cuda_host) with the sources that they include."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not available")
    emu = os.path.join(HERE, "cuda_host", "tc_emu")
    # all beside one another: quoted includes are looked for there first
    for f in os.listdir(emu):
        shutil.copy(os.path.join(emu, f), folder)
    for f in ("attn_host.h",) + drivers:
        shutil.copy(os.path.join(HERE, "cuda_host", f), folder)
    for name in kernels + HEADERS:
        with open(os.path.join(CSRC, name)) as f:
            (folder / name).write_text(for_host(f.read()))
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    so = str(folder / (drivers[0] + ".so"))
    subprocess.run([gxx, "-O1", "-fno-strict-aliasing", "-std=c++17", "-w", "-fPIC", "-shared", "-I", cuda, "-I",
                    os.path.join(ROOT, "include"), "-o", so] + [str(folder / f) for f in drivers], check=True)
    return ctypes.CDLL(so)
