"""The RMS norm, the 8-bit and the grouped layer operators on the CPU: the C ABI's
refusals under AddressSanitizer and UndefinedBehaviorSanitizer (the entry points' sources
linked with launchers that do nothing), the Python layer's checks, the tile that sizes
take, and the direct-to-LDS loads of the kernels in their gfx950 assembly.
"""

import ctypes
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from muon_newton_schulz_04_amd import binding as B
from muon_newton_schulz_04_amd import layers as L
from test_abi_sanitize import CSRC, NATIVE, ROCM, ROOT, _have_toolchain
from test_kernel_assembly import _compile, _have_hipcc, _instructions, check_m0_use

INC = [f"-I{ROCM}/include", f"-I{ROOT}/include", f"-I{CSRC}", "-D__HIP_PLATFORM_AMD__"]


@pytest.mark.skipif(not _have_toolchain(), reason="g++ / gcc / ROCm HIP runtime not available")
@pytest.mark.skipif(torch.cuda.is_available(), reason="the check's addresses are made up: for hosts without a GPU")
def test_abi_under_asan_and_ubsan(tmp_path):
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]
    objs = []

    def build(src):
        o = str(tmp_path / (os.path.basename(src) + ".o"))
        cc, std = ("gcc", "-std=c99") if src.endswith(".c") else ("g++", "-std=c++17")
        subprocess.run([cc, std, "-Wall", *san, *INC, "-c", src, "-o", o], check=True)
        return o

    srcs = [os.path.join(CSRC, s) for s in ("layers.cpp", "layers_scaled.cpp", "layers_grouped.cpp")]
    srcs += [os.path.join(NATIVE, s) for s in ("layer_stubs.cpp", "scaled_stubs.cpp", "scaled_check.c")]
    with ThreadPoolExecutor(len(srcs)) as ex:
        objs = list(ex.map(build, srcs))
    exe = str(tmp_path / "scaled_check")
    subprocess.run(["g++", *san, *objs, "-o", exe, f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib", "-lm"],
                   check=True)
    env = dict(os.environ)
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=0:halt_on_error=1"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "all expectations hold" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr


def test_struct_sizes_match_c_layout():
    assert ctypes.sizeof(B.muon_rmsnorm) == 7 * 8 + 2 * 4
    assert ctypes.sizeof(B.muon_eight) == 3 * 8 + 2 * 4
    assert ctypes.sizeof(B.muon_grouped) == 8 * 8 + 2 * 4


def test_cpu_tensors_are_refused():
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(2, 16, 32, dtype=torch.bfloat16)
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    x8 = x.to(torch.float8_e4m3fn), torch.ones(1, 4)
    for call in (lambda: L.rmsnorm_forward(x), lambda: L.rmsnorm_backward(x, x, x), lambda: L.quantize_fp8(x),
                 lambda: L.quantize_fp8_weight(x), lambda: L.linear_fp8_forward(x8, x8),
                 lambda: L.linear_fp8_grad_input(x8, x8), lambda: L.grouped_linear_forward(x, w, off),
                 lambda: L.grouped_linear_grad_input(x, w, off), lambda: L.grouped_linear_grad_weight(x, x, off)):
        with pytest.raises(ValueError, match="expected a GPU tensor"):
            call()


# the kinds of tile, in the order of layers.hpp's TileKind
KINDS = ["tall", "square", "square groups", "small", "small groups", "few 16", "few 32"]


def plans(tmp_path, lines):
    """The kind of tile that the entry points' sources take for each line, and the pieces."""
    exe = str(tmp_path / "scaled_plan")
    srcs = [os.path.join(NATIVE, s) for s in ("scaled_plan.cpp", "layer_stubs.cpp", "scaled_stubs.cpp")]
    subprocess.run(["g++", "-std=c++17", "-O1", *INC, *srcs, os.path.join(CSRC, "layers.cpp"), "-o", exe,
                    f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib"], check=True)
    text = "".join(" ".join(str(v) for v in line) + "\n" for line in lines)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    got = [[int(v) for v in o.split()] for o in out if o]
    return [KINDS[k] + (f" in {p}" if p > 1 else "") for k, p in got]


@pytest.mark.skipif(not _have_toolchain(), reason="g++ / ROCm HIP runtime not available")
def test_every_tile_is_taken_by_a_tested_size(tmp_path):
    """The sizes that test_scaled_tiles_gpu.py runs on the GPU take the tile that they
    stand for, so that another choice of plan cannot leave a kernel untested."""
    from test_scaled_tiles_gpu import EIGHT, GROUPED, line_of
    got = plans(tmp_path, [line_of(c) for c in EIGHT + GROUPED])
    assert got == [c[-1] for c in EIGHT + GROUPED]
    assert {c[-1] for c in EIGHT} == set(KINDS)
    for op in ("forward", "grad input"):
        assert {c[-1] for c in GROUPED if c[0] == op} == set(KINDS)
    weight = {c[-1] for c in GROUPED if c[0] == "grad weight"}
    assert {c.split(" in ")[0] for c in weight} == {"tall", "square", "small"}
    assert {c.split(" in ")[0] for c in weight if " in " in c} == {"tall", "square", "small"}


@pytest.mark.skipif(not _have_hipcc(), reason="hipcc not available")
def test_m0_written_only_by_the_lds_load_helpers(tmp_path):
    srcs = ("kernels_scaled.hip", "kernels_grouped.hip")
    with ThreadPoolExecutor(len(srcs)) as ex:
        listings = list(ex.map(lambda s: _compile(s, str(tmp_path)), srcs))
    for src, asm in zip(srcs, listings):
        pairs, problems = check_m0_use(_instructions(asm))
        assert pairs > 0, f"{src}: no direct-to-LDS loads found (the check would be vacuous)"
        assert not problems, f"{src}: " + "; ".join(problems[:10])
