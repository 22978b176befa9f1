"""Limits of the adapter and block-norm entry points that the kernels' arithmetic sets, on the host.  No pointer
below is ever dereferenced: every call is refused before anything is launched."""
import ctypes
import os
import re

import pytest
import torch

SHAPE, DEVICE = 2, 5
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "nq.h")


@pytest.fixture(scope="module")
def nq():
    from rank_binary_factorized_b200 import nq as mod
    return mod


def _limit(name):
    with open(HEADER) as f:
        return int(re.search(r"#define %s (\d+)" % name, f.read()).group(1))


@pytest.mark.parametrize("n,rank,d", [(1, 1, 1), (3, 16, 8), (16384, 8, 8)])
def test_adapter_rows_beyond_the_kernels_32_bit_counts_are_refused(nq, n, rank, d):
    """A group of 2^31 - 1 rows rounded up to a tile does not fit 32 bits: such a batch is refused, up to
    the documented limit it is taken, and there the counts fit."""
    most = _limit("NQ_ADAPTER_MAX_M")
    S = nq.nq_adapters(n, rank, d, d, 0x10000, d, 0x20000, rank, 0)
    lib = nq.raw_lib()
    for M in (most + 1, 2 ** 31 - 128, 2 ** 31 - 1):
        assert lib.nq_adapter_forward(ctypes.byref(S), 0x40000, 0x50000, 0x60000, 0x70000, 0x80000, 0, M, None) == SHAPE
        assert lib.nq_adapter_backward(ctypes.byref(S), 0x40000, 0x50000, 0x60000, 0x70000, 0x80000, 0x90000, 0xA0000,
                                       0xB0000, 0xC0000, M, 0xD0000, 1 << 62, None) == SHAPE
        assert lib.nq_adapter_workspace_bytes(ctypes.byref(S), M) == 0
    assert lib.nq_adapter_workspace_bytes(ctypes.byref(S), most) > 0
    if not torch.cuda.is_available():  # nothing here is launched
        assert lib.nq_adapter_forward(ctypes.byref(S), 0x40000, 0x50000, 0x60000, 0x70000, 0x80000, 0, most, None) == DEVICE
    padded = most + 15 * _limit("NQ_ADAPTER_MAX_N")
    assert most + 127 < 2 ** 31 and 2 * padded < 2 ** 31


def test_adapter_columns_beyond_the_kernels_32_bit_counts_are_refused(nq):
    """The last tile of columns below 2^31 does not fit 32 bits when it is rounded up."""
    most = _limit("NQ_ADAPTER_MAX_D")
    lib = nq.raw_lib()
    for d_in, d_out in ((2 ** 31 - 8, 64), (64, 2 ** 31 - 8), (most + 8, 64), (64, most + 8), (most, most)):
        S = nq.nq_adapters(1, 8, d_in, d_out, 0x10000, d_in, 0x20000, 8, 0)
        taken = max(d_in, d_out) <= most
        assert (lib.nq_adapter_workspace_bytes(ctypes.byref(S), 4) > 0) == taken
        if not taken or not torch.cuda.is_available():
            want = DEVICE if taken else SHAPE
            assert lib.nq_adapter_forward(ctypes.byref(S), 0x40000, 0x50000, 0x60000, 0x70000, 0x80000, 0, 4, None) == want
            assert lib.nq_adapter_backward(ctypes.byref(S), 0x40000, 0x50000, 0x60000, 0x70000, 0x80000, 0x90000, 0xA0000,
                                           0xB0000, 0xC0000, 4, 0xD0000, 1 << 62, None) == want
    assert most + 2047 < 2 ** 31
