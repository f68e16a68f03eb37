"""Decode-layer operators: what can be held without a GPU, beside the refusals."""
import os

import pytest

import chunked_gated_delta_14_b200 as gdn

CSRC = os.path.join(os.path.dirname(os.path.abspath(gdn.__file__)), "csrc")


@pytest.mark.parametrize("name", ["gdn_recurrent_pool.cu", "gdn_rows_int8.cu", "gdn_int8_matmul.cu"])
def test_no_read_only_loads_where_kernels_begin_early(name):
    """The read-only path is for data that is constant while the kernel lives; a kernel launched
    early lives while the one ahead still writes its operands."""
    source = open(os.path.join(CSRC, name)).read()
    assert "grid_wait" in source
    for load in ("__ldg", "ld.global.nc", "__restrict__"):
        assert load not in source, load
