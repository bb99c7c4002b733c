"""The gated delta rule's limits on sizes are those that include/gated_delta.h states (nothing here is launched: fake
device pointers, and every call ends at a host check)."""
import ctypes
import os

import pytest

from quaternion_cumprod_autodiff_amd import capi
from quaternion_cumprod_autodiff_amd.build import LIB_PATH

E_SHAPE, E_ALIAS = -2, -5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB_PATH):
        from quaternion_cumprod_autodiff_amd.build import build
        build()
    return capi.load()


def dims(B, T, Hk, Hv, K, V, N=None):
    d = capi.GdrDims(B, T, Hk, Hv, K, V, B if N is None else N)
    d.q_stride[:] = d.k_stride[:] = (T * Hk * K, Hk * K, K)
    d.v_stride[:] = (T * Hv * V, Hv * V, V)
    d.packed, d.scale = int(N is not None), 1.0
    return d


@pytest.mark.parametrize("size,ok", [
    ((1, 1, 16384, 16384, 1, 1024), True),          # 2^20 of (sequence, head, 16 columns)
    ((8, 1, 16384, 16384, 1, 1008), True),          # 63 * 2^17, just below 2^23
    ((8, 1, 16384, 16384, 1, 1024), False),         # 2^23
    ((1, 1, 1, 16384, 1, 1008), True),              # one key head is rounded up to eight
    ((1, 1, 1, 16384, 1, 1024), False),
    ((1, 1, 1 << 20, 1 << 20, 1, 16), True),
    ((1, 1, 1 << 20, 1 << 21, 1, 16), False),       # heads
    ((1, 1, (1 << 20) + 8, (1 << 20) + 8, 1, 16), False),
    ((1, 64 * 511, 16384, 16384, 1, 1), True),      # chunks: 511 * 2^14
    ((1, 64 * 511 + 1, 16384, 16384, 1, 1), False),
], ids=str)
def test_rule_takes_what_the_header_says(lib, size, ok):
    d = dims(*size)
    for n in (lib.gdr_workspace_bytes(d, 0), lib.gdr_workspace_bytes(d, 1), lib.gdr_saved_bytes(d)):
        assert (n > 0) == ok


def test_packed_chunks_count_a_slot_more_for_each_sequence(lib):
    assert lib.gdr_workspace_bytes(dims(1, 64 * 500, 16384, 16384, 1, 1, N=11), 0) > 0
    assert lib.gdr_workspace_bytes(dims(1, 64 * 500, 16384, 16384, 1, 1, N=12), 0) == 0


@pytest.mark.parametrize("n,code", [(1082401, E_ALIAS), (1082402, E_SHAPE)])
def test_step_takes_what_the_header_says(lib, n, code):
    """31 pieces of 32 columns: 1082401 rows are 2^25 - 1 of them, and are refused for out in the states alone."""
    p = [ctypes.c_void_p(0x10_0000_0000 * i) for i in range(8)]
    out = ctypes.c_void_p(p[6].value + 16)
    assert lib.gdr_step(dims(n, 1, 1, 1, 1, 992), *p[1:6], p[6], n, 992, p[7], out, None) == code
