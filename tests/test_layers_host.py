"""The layer operators on the CPU: the C ABI's refusals and workspace sizes
under AddressSanitizer and UndefinedBehaviorSanitizer (layers.cpp linked with
launchers that do nothing), the Python layer's checks, and the direct-to-LDS
loads of the product kernels in their gfx950 assembly.
"""

import ctypes
import os
import subprocess

import pytest
import torch

from muon_newton_schulz_04_amd import binding as B
from muon_newton_schulz_04_amd import layers as L
from test_abi_sanitize import CSRC, NATIVE, ROCM, ROOT, _have_toolchain
from test_kernel_assembly import _compile, _have_hipcc, _instructions, check_m0_use


@pytest.mark.skipif(not _have_toolchain(), reason="g++ / gcc / ROCm HIP runtime not available")
@pytest.mark.skipif(torch.cuda.is_available(), reason="the check's addresses are made up: for hosts without a GPU")
def test_layer_abi_under_asan_and_ubsan(tmp_path):
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]
    inc = [f"-I{ROCM}/include", f"-I{ROOT}/include", f"-I{CSRC}", "-D__HIP_PLATFORM_AMD__"]
    objs = []
    for cc, std, src in (("g++", "-std=c++17", os.path.join(CSRC, "layers.cpp")),
                         ("g++", "-std=c++17", os.path.join(NATIVE, "layer_stubs.cpp")),
                         ("gcc", "-std=c99", os.path.join(NATIVE, "layer_check.c"))):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        subprocess.run([cc, std, "-Wall", *san, *inc, "-c", src, "-o", objs[-1]], check=True)
    exe = str(tmp_path / "layer_check")
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
    assert ctypes.sizeof(B.muon_linear) == 6 * 8 + 2 * 4
    assert ctypes.sizeof(B.muon_epilogue) == 2 * 4 + 5 * 8
    assert ctypes.sizeof(B.muon_layernorm) == 6 * 8 + 2 * 4


def test_errors_are_explained():
    d = B.muon_linear(4, 0, 8, 0, 0, 0, B.MUON_TYPE_BF16, 0)
    s, _ = B.muon_linear_workspace_bytes(d, B.MUON_LINEAR_FORWARD, 0, 0)
    assert s == B.MUON_E_SHAPE and "features" in B.muon_op_last_error()


def test_cpu_tensors_are_refused():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expected a GPU tensor"):
        L.linear_forward(x, w)
    with pytest.raises(ValueError, match="expected a GPU tensor"):
        L.linear_grad_input(x, w)
    with pytest.raises(ValueError, match="expected a GPU tensor"):
        L.linear_grad_weight(x, x)
    with pytest.raises(ValueError, match="expected a GPU tensor"):
        L.layernorm_forward(x)
    with pytest.raises(ValueError, match="expected a GPU tensor"):
        L.layernorm_backward(x, x, x, x)


@pytest.mark.skipif(not _have_hipcc(), reason="hipcc not available")
def test_m0_written_only_by_the_lds_load_helper(tmp_path):
    pairs, problems = check_m0_use(_instructions(_compile("kernels_linear.hip", str(tmp_path))))
    assert pairs > 0, "no direct-to-LDS loads found (the check would be vacuous)"
    assert not problems, "; ".join(problems[:10])
