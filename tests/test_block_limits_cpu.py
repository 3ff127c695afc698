"""Sizes at the edges of the block-128 and norm calls' index ranges and overlap rules, refused or
accepted on the host (pointers are only compared)."""
import ctypes
import os

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
E4M3, F32, BF16 = 0, 0, 1
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    from precision_block_amax_amd import build as libbuild
    if not os.path.exists(libbuild.LIB_PATH):
        libbuild.build()
    import precision_block_amax_amd as mx
    return mx.lib()


@pytest.mark.parametrize("out", [F32, BF16])
def test_block_gemm_longest_k(L, out):
    """The kernels count K, rounded up to whole blocks, in 31 bits: a K above 2^31 - 128 would round to 2^31
    and past it, so it is refused, not answered with zeros."""
    for K in ((1 << 31) - 127, (1 << 31) - 1, 1 << 31, 1 << 40):
        args = [P(1 << 44), K, P(1 << 45), 1, E4M3, P(1 << 46), K, P(1 << 47), 1, E4M3, 0, 1, 1, K, P(1 << 32), out, 1, None]
        assert L.mx_block_gemm(*args) == UNSUPPORTED, K
