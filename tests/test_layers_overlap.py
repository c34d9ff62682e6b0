"""In-place calls of the layer operators: the output may be the tensor of the
residual (`add`), but not where that is an operand too.
"""

import os
import subprocess

import pytest
import torch

from muon_newton_schulz_04_amd import binding as B
from muon_newton_schulz_04_amd import layers as L
from test_abi_sanitize import CSRC, NATIVE, ROCM, ROOT, _have_toolchain


def run_native(tmp_path, check):
    """Builds `check` (a C source under tests/native) with layers.cpp and
    launchers that do nothing, under the sanitizers, and runs it."""
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]
    inc = [f"-I{ROCM}/include", f"-I{ROOT}/include", f"-I{CSRC}", "-D__HIP_PLATFORM_AMD__"]
    objs = []
    for cc, std, src in (("g++", "-std=c++17", os.path.join(CSRC, "layers.cpp")),
                         ("g++", "-std=c++17", os.path.join(NATIVE, "layer_stubs.cpp")),
                         ("gcc", "-std=c99", os.path.join(NATIVE, check))):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        subprocess.run([cc, std, "-Wall", *san, *inc, "-c", src, "-o", objs[-1]], check=True)
    exe = str(tmp_path / "check")
    subprocess.run(["g++", *san, *objs, "-o", exe, f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib"], check=True)
    env = dict(os.environ)
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=0:halt_on_error=1"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    return subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)


@pytest.mark.skipif(not _have_toolchain(), reason="g++ / gcc / ROCm HIP runtime not available")
@pytest.mark.skipif(torch.cuda.is_available(), reason="the check's addresses are made up: for hosts without a GPU")
def test_output_over_an_operand_is_refused_even_at_the_residuals_address(tmp_path):
    r = run_native(tmp_path, "layer_overlap_check.c")
    assert r.returncode == 0, r.stdout + r.stderr
    assert "all expectations hold" in r.stdout


@pytest.mark.gpu
def test_in_place_over_the_residual_alone():
    """A square layer's sum over its own input is refused and leaves it as it
    was; over a residual of its own it is the separate call's result."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(40, 64, generator=g).bfloat16().cuda()
    w = (torch.randn(64, 64, generator=g) / 8).bfloat16().cuda()
    keep = x.clone()
    for layout in ("in_out", "out_in"):
        for call in (lambda: L.linear_forward(x, w, residual=x, out=x, weight_layout=layout),
                     lambda: L.linear_grad_input(x, w, add=x, out=x, weight_layout=layout),
                     lambda: L.linear_forward(x, w, residual=w[:40], out=w[:40], weight_layout=layout)):
            with pytest.raises(B.MuonError, match="overlaps"):
                call()
        assert torch.equal(x, keep)
        want = L.linear_forward(x, w, residual=x, weight_layout=layout)
        res = x.clone()
        assert L.linear_forward(x, w, residual=res, out=res, weight_layout=layout) is res
        assert torch.equal(res, want)
        want = L.linear_grad_input(x, w, add=x, weight_layout=layout)
        res = x.clone()
        L.linear_grad_input(x, w, add=res, out=res, weight_layout=layout)
        assert torch.equal(res, want)
    stats = torch.zeros(40, device="cuda"), torch.ones(40, device="cuda")
    with pytest.raises(B.MuonError, match="overlaps"):
        L.layernorm_backward(x, w[:40], *stats, add=x, out=x)
    with pytest.raises(B.MuonError, match="overlaps"):
        L.layernorm_backward(w[:40], x, *stats, add=x, out=x)
    assert torch.equal(x, keep)
