"""Sizes that the headers of linear attention with decays and layer norm refuse, without a GPU: fake device pointers,
and every call returns before any HIP call."""
import ctypes
import os

import pytest

from quaternion_cumprod_autodiff_amd import capi
from quaternion_cumprod_autodiff_amd.build import LIB_PATH

E_SHAPE, E_ALIAS = -2, -5
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB_PATH):
        from quaternion_cumprod_autodiff_amd.build import build
        build()
    return capi.load()


def P(n, by=0):
    return ctypes.c_void_p(0x1000_0000_0000 * n + by)


def step(lib, n, heads, V, slots, out):
    d = capi.DcaDims(n, 1, 1, heads, 1, V, n)
    d.q_stride[:] = d.k_stride[:] = (1, 1, 1)
    d.v_stride[:] = (heads * V, heads * V, V)
    d.dtype, d.scale, d.packed, d.head_decay = BF16, 1.0, 0, 1
    return lib.dca_step(d, P(1), P(2), P(3), P(4), P(5), n, heads * V, slots, out, None)


@pytest.mark.parametrize("n,heads,V", [((1 << 20) + 1, 1, 32), ((1 << 18) + 1, 16, 16), ((1 << 19) + 1, 1, 97), ((1 << 25), 1, 1)], ids=str)
def test_a_step_refuses_more_slots_than_it_can_look_through(lib, n, heads, V):
    """A row looks through the slots of those before it, once for each head and 32 columns: 2^40 at most, an eighth of a
    second.  Without slots there is nothing to look through, and such sizes are refused for out in the states alone."""
    assert step(lib, n, heads, V, P(7), P(8)) == E_SHAPE
    assert step(lib, n, heads, V, None, P(5, 16)) == E_ALIAS


@pytest.mark.parametrize("B,T,N,heads,K,V,dtype,states", [
    (4, 4096, 4, 32, 128, 128, BF16, 4 * 64 * 32 * 128 * 128),
    (2, 65, 2, 3, 33, 65, BF16, 2 * 2 * 3 * 64 * 128),
    (2, 65, 2, 3, 32, 64, F32, 2 * 3 * 3 * 32 * 64),
    (1, 12288, 64, 2, 128, 128, BF16, (192 + 64) * 2 * 128 * 128),
    (1, 1000, 7, 1, 64, 20, F16, (31 + 7) * 64 * 64),
], ids=str)
def test_a_training_step_keeps_the_states_that_are_documented(lib, B, T, N, heads, K, V, dtype, states):
    """A float32 state for each chunk of 64 tokens (32): N ceil(T / C) of them, of packed sequences floor(T / C) + N."""
    d = capi.DcaDims(B, T, heads, heads, K, V, N)
    d.q_stride[:] = d.k_stride[:] = (T * heads * K, heads * K, K)
    d.v_stride[:] = (T * heads * V, heads * V, V)
    d.dtype, d.scale, d.packed, d.head_decay = dtype, 1.0, int(N != B), 0
    assert 4 * states <= lib.dca_saved_bytes(d) < 4 * states + 512
    assert lib.dca_workspace_bytes(d, 1) >= 4 * states
