"""Decode-layer operators: what can be held without a GPU, beside the refusals."""
import os
import subprocess
import sys

import pytest
import torch

import bench
import chunked_gated_delta_14_b200 as gdn
import chunked_gated_delta_14_b200.layer as L
from chunked_gated_delta_14_b200 import build as gbuild

CSRC = os.path.join(os.path.dirname(os.path.abspath(gdn.__file__)), "csrc")


@pytest.mark.parametrize("name", ["gdn_recurrent_pool.cu", "gdn_rows_int8.cu", "gdn_int8_matmul.cu"])
def test_no_read_only_loads_where_kernels_begin_early(name):
    """The read-only path is for data that is constant while the kernel lives; a kernel launched
    early lives while the one ahead still writes its operands."""
    source = open(os.path.join(CSRC, name)).read()
    assert "grid_wait" in source
    for load in ("__ldg", "ld.global.nc", "__restrict__"):
        assert load not in source, load


WORDS = r"""
#include <cstdio>
#include "gdn_internal.cuh"
#include "gdn_serve.cuh"
// Stand-ins for the four kernels' error words: read and cleared as on the device.
static unsigned words[4];
static unsigned take(int i) { const unsigned v = words[i]; words[i] = 0; return v; }
namespace gdn {
unsigned int tc_read_and_clear_error(cudaStream_t, cudaError_t *e) { *e = cudaSuccess; return take(0); }
unsigned int fused_read_and_clear_error(cudaError_t *e) { *e = cudaSuccess; return take(1); }
unsigned int pool_read_and_clear_error(cudaError_t *e) { *e = cudaSuccess; return take(2); }
unsigned int int8_matmul_read_and_clear_error(cudaError_t *e) { *e = cudaSuccess; return take(3); }
}
int main() {
    for (int set = 0; set < 16; ++set) {
        for (int i = 0; i < 4; ++i) words[i] = set >> i & 1;
        int reports = 0;
        while (gdn_device_check(nullptr) != GDN_OK && reports < 5) ++reports;
        printf("%d\n", reports);
    }
}
"""


def test_device_check_reports_every_word(tmp_path):
    """Words of several kernels set at once: each call reports one, and none is lost."""
    (tmp_path / "main.cu").write_text(WORDS)
    exe = str(tmp_path / "words")
    subprocess.check_call([gbuild.NVCC, *gbuild.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", gbuild.INCLUDE, "-I", CSRC,
                           str(tmp_path / "main.cu"), os.path.join(CSRC, "gdn_api.cu"), "-o", exe,
                           "-Xlinker", "--unresolved-symbols=ignore-all"])
    out = subprocess.check_output([exe]).decode().split()
    assert out == [str(bin(i).count("1")) for i in range(16)]


@pytest.fixture
def binding_elsewhere(tmp_path, monkeypatch):
    """build.py's binding in a folder of its own, made by a compiler that writes a line each time."""
    cxx = tmp_path / "cxx"
    cxx.write_text("#!/bin/sh\nwhile [ \"$1\" != -o ]; do shift; done\necho built > \"$2\"\necho run >> " + str(tmp_path / "runs") + "\n")
    cxx.chmod(0o755)
    monkeypatch.setenv("CXX", str(cxx))
    monkeypatch.setattr(gbuild, "BINDING", str(tmp_path / "_layer.so"))
    runs = tmp_path / "runs"
    return lambda: len(runs.read_text().split()) if runs.exists() else 0


def test_binding_is_rebuilt_for_another_torch(binding_elsewhere, monkeypatch):
    assert not gbuild.binding_is_current()
    for _ in range(2):
        gbuild.build_binding()
    assert binding_elsewhere() == 1 and gbuild.binding_is_current()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert not gbuild.binding_is_current()
    gbuild.build_binding()
    assert binding_elsewhere() == 2 and gbuild.binding_is_current()


def test_binding_of_another_torch_is_not_used(monkeypatch):
    monkeypatch.setattr(L, "_quick", None)
    gbuild.build_binding()
    from chunked_gated_delta_14_b200 import _layer
    assert L._bind_quick() is _layer and _layer.built_for == gbuild.binding_for()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert L._bind_quick() is L._NoQuick


@pytest.mark.parametrize("cxx", ["/bin/false", "/nowhere/cxx"])
def test_library_builds_without_a_host_compiler_for_the_binding(binding_elsewhere, cxx, monkeypatch, capsys):
    monkeypatch.setenv("CXX", cxx)
    assert gbuild.build() == gbuild.LIB and os.path.exists(gbuild.LIB)
    assert "not built" in capsys.readouterr().err and not gbuild.binding_is_current()


def test_bench_says_what_the_layer_finds_in_l2():
    assert "> 126 MB" in bench.layer_l2(256, 16, 128)
    assert "stay in" in bench.layer_l2(4, 16, 128)


def test_bench_refuses_the_layer_without_decode(monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["bench.py", "--layer"])
    with pytest.raises(SystemExit) as e:
        bench.main()
    assert e.value.code == 2 and "--decode" in capsys.readouterr().err
