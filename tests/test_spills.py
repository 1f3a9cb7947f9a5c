"""Registers of the bias and dropout kernels: they share their source with the plain and the windowed ones and sit at the
register limit of their launch bounds, so that an expression added for another instantiation can make them spill (96 and
92 bytes in place of 32 and 12 made the bias-only forward 1.13x slower).  What ptxas reports, without a GPU."""
import os
import re
import subprocess

import pytest

from io_aware_exact_32_b200 import build

KERNELS = {  # instantiation: bytes of spill stores and loads it may have
    "fa_fwd_kernel<128, false, true>": (32, 12),
    "fa_fwd_kernel<64, false, true>": (44, 28),
    "fa_bwd_main_kernel<128, true, true>": (0, 0),
    "fa_bwd_main_kernel<64, true, true>": (0, 0),
}


@pytest.fixture(scope="module")
def report(tmp_path_factory):
    try:
        nvcc = build._nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    folder = tmp_path_factory.mktemp("spills")
    source = folder / "kernels.cu"
    source.write_text("#include <cuda.h>\n" +
                      "".join(f'#include "{os.path.join(build.CSRC, n)}"\n' for n in ("fwd_sm100.cuh", "bwd_sm100.cuh")) +
                      "extern const void* const kernels[] = {" + ", ".join(f"(const void*)fa::{k}" for k in KERNELS) + "};\n")
    flags = [f for f in build.NVCC_FLAGS if f != "-shared"]
    run = subprocess.run([nvcc, *flags, "-Xptxas", "-v", "-c", "-o", str(folder / "kernels.o"), str(source)],
                         capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]
    text = run.stdout + run.stderr
    found = {}
    for entry, rest in re.findall(r"Compiling entry function '(\S+)'(.*?)(?=Compiling entry function|\Z)", text, re.S):
        m = re.search(r"(\d+) bytes spill stores, (\d+) bytes spill loads", rest)
        found[entry] = (int(m[1]), int(m[2]))
    return found


@pytest.mark.parametrize("kernel", KERNELS)
def test_spills(report, kernel):
    name, args = re.fullmatch(r"(\w+)<(.*)>", kernel).groups()
    mangled = name + "I" + "".join(f"Li{a}E" if a.isdigit() else f"Lb{int(a == 'true')}E" for a in args.split(", "))
    hits = [v for k, v in report.items() if mangled in k]
    assert len(hits) == 1
    assert hits[0] <= KERNELS[kernel] and hits[0][1] <= KERNELS[kernel][1], hits
