"""A launch has fewer than 2^32 threads: on the CPU, what the dense entries plan
for sizes that would pass it, or refuse before any device work."""
import ctypes

import pytest

import int8_convolution_forward_amd as ci8
from int8_convolution_forward_amd import dense

BF16 = 3
FAKE = 0x1000000  # aligned, never dereferenced


def mat(r, c):
    return (FAKE, r, c, c, 1, BF16)


def linear_size(m, n, k):
    args = dense._pack_linear(*mat(m, k), *mat(n, k), *mat(m, n), *dense._NO_MAT, *dense._NO_MAT, *dense._NO_VEC,
                              *dense._NO_VEC, *dense._NO_VEC, 0)
    n = ctypes.c_size_t()
    return ci8.STATUS[dense.lib.dense_linear_workspace_size(args, n)], args


@pytest.mark.parametrize("n,kernel", [(1 << 25, "skinny"), ((1 << 25) + 1, "gemm"), (1 << 26, "gemm"), (1 << 30, "gemm")])
def test_few_rows_and_many_columns(n, kernel):
    """1024 threads for 16 columns are 2^32 for 2^26."""
    status, args = linear_size(4, n, 8)
    assert status == "CONV_I8_OK"
    buf = ctypes.create_string_buffer(512)
    assert dense.lib.dense_linear_plan(args, buf, 512) == 0
    fields = ci8.plan_fields(buf.value.decode())
    assert fields["kernel"] == kernel
    if kernel == "gemm":
        assert int(fields["tiles"]) * int(fields["split"]) * 256 < 1 << 32


def test_copies_and_tiles_past_a_launch_are_refused():
    """Copies of more than 64 GiB, and more tiles than a launch has workgroups."""
    assert linear_size(1 << 28, 48, 33)[0] == "CONV_I8_OK"
    assert linear_size(1 << 30, 48, 33)[0] == "CONV_I8_ERR_UNSUPPORTED"
    assert linear_size(1 << 30, 1 << 14, 64)[0] == "CONV_I8_ERR_UNSUPPORTED"


def test_norm_gradients_of_very_wide_and_very_many_rows():
    """Their partial sums' size: the widest row, and narrow rows by the workgroup."""
    none, stat = dense._NO_VEC, lambda m: (FAKE, m, 5)
    for m, d, most in ((1, 1 << 30, 2 * 4 << 30), ((1 << 22) + 3, 7, 512 * 2 * 8 * 4), (1 << 30, 1, 512 * 2 * 8 * 4)):
        args = dense._pack_norm_backward(*mat(m, d), *mat(m, d), *mat(m, d), *none, *stat(m), *stat(m), FAKE, d, BF16, FAKE, d,
                                         BF16)
        n = ctypes.c_size_t()
        assert dense.lib.dense_layer_norm_backward_workspace_size(args, n) == 0
        assert 0 < n.value <= most
