"""Device functions compiled as plain C++, to be run lane by lane on the CPU."""
from __future__ import annotations

import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_sampling_gb300", "csrc")


def function(file: str, name: str) -> str:
    """The definition of `name` in csrc/`file`, from its template head or first line to its closing brace."""
    text = open(os.path.join(CSRC, file), encoding="utf-8").read()
    m = re.search(r"^(template <[^\n]*>\n)?__device__ [^\n;]*\b" + name + r"\([^;{]*\)\n?\{.*?^\}\n", text, flags=re.M | re.S)
    assert m, name
    return m.group(0)


def run(source: str, tmp_path, *args: str, include=(CSRC,)) -> str:
    """Compile C++ source with the host compiler, run it, return what it prints."""
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(source)
    subprocess.run(["g++", "-O1", "-std=c++17", "-w", *[f"-I{i}" for i in include], "-o", str(exe), str(src)], check=True)
    return subprocess.run([str(exe), *args], check=True, capture_output=True, text=True).stdout
