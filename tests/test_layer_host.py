"""Decode-layer operators: what can be held without a GPU, beside the refusals."""
import os
import subprocess

import pytest

import chunked_gated_delta_14_b200 as gdn
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
