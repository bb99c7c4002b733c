"""The language-model operators without a GPU: their oracles against
differences, the header's names, and the C entry points' refusals (fake device
pointers: every one of these calls returns before any HIP call)."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from oracle import lm_ops as ref
from quaternion_cumprod_autodiff_amd import autograd, capi
from quaternion_cumprod_autodiff_amd.build import LIB_PATH

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, E_NULL, E_SHAPE, E_ALIGN, E_DTYPE, E_ALIAS, E_WS, E_HIP, E_OPT = 0, -1, -2, -3, -4, -5, -6, -7, -8


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB_PATH):
        from quaternion_cumprod_autodiff_amd.build import build
        build()
    return capi.load()


def test_headers_declare_what_the_binding_uses(lib):
    names = set()
    for h in ("gated_delta.h", "qk_norm.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", h)).read(), flags=re.S)
        names |= set(re.findall(r"\b((?:gdr|qkn)_\w+)\s*\(", text))
    assert sorted(names) == sorted(capi.LM_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names == set(re.findall(r"\bT ((?:gdr|qkn)_\w+)", out))


# ------------------------------------------------------------------ the oracles

def central(f, x, d, eps=1e-5):
    """The directional derivative of the number f(x) along d."""
    return (f(x + eps * d) - f(x - eps * d)) / (2 * eps)


@pytest.mark.parametrize("lengths", [None, [3, 0, 1, 2]])
def test_rule_oracle_gradients_match_differences(lengths):
    rng = np.random.default_rng(5)
    B, T, Hk, Hv, K, V = (2, 5, 2, 4, 3, 4) if lengths is None else (1, 7, 1, 3, 4, 2)
    N = B if lengths is None else len(lengths)
    x = [rng.standard_normal(s) for s in [(B, T, Hk, K)] * 2 + [(B, T, Hv, V)]]
    x += [-rng.random((B, T, Hv)), rng.random((B, T, Hv)), rng.standard_normal((N, Hv, K, V))]
    w_out, w_fin = rng.standard_normal((B, T, Hv, V)), rng.standard_normal((N, Hv, K, V))

    def loss(*a):
        out, fin = ref.gdr_fwd(*a, 0.7, lengths)
        return (out * w_out).sum() + (fin * w_fin).sum()

    grads = ref.gdr_bwd(*x, 0.7, w_out, w_fin, lengths)
    for i, g in enumerate(grads):
        d = rng.standard_normal(x[i].shape)
        want = central(lambda y: loss(*x[:i], y, *x[i + 1:]), x[i], d)
        assert abs((g * d).sum() - want) <= 1e-7 * (1 + abs(want)), i


def test_rule_oracle_by_hand():
    # One head, K = 1, V = 1: S = a S; u = b (v - S k); S += k u; o = s S q.
    one = lambda *v: np.array(v, dtype=np.float64).reshape(1, -1, 1, 1)
    out, fin = ref.gdr_fwd(one(1, 2), one(1, 0.5), one(3, 5), np.log(one(0.5, 0.25))[..., 0], one(1, 0.5)[..., 0],
                           np.array([[[[2.0]]]]), 10.0)
    # t = 0: S = 1, u = 3 - 1 = 2, S = 3, o = 30;  t = 1: S = .75, u = .5 (5 - .375) = 2.3125, S = 1.90625, o = 38.125
    assert out.ravel().tolist() == [30.0, 38.125] and fin.ravel().tolist() == [1.90625]


@pytest.mark.parametrize("kind", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_oracle_gradients_match_differences(kind, interleaved):
    rng = np.random.default_rng(7)
    x, w, dy = rng.standard_normal((2, 3, 2, 10)), rng.standard_normal(10), rng.standard_normal((2, 3, 2, 10))
    angle = rng.standard_normal((5, 3))
    pos = rng.integers(0, 5, (2, 3))
    how = (np.cos(angle), np.sin(angle), pos, kind, 1e-3, interleaved)
    dx, dw = ref.qkn_bwd(x, w, *how, dy)
    for i, g in enumerate((dx, dw)):
        d = rng.standard_normal(g.shape)
        f = (lambda y: (ref.qkn_fwd(y, w, *how) * dy).sum()) if i == 0 else (lambda y: (ref.qkn_fwd(x, y, *how) * dy).sum())
        want = central(f, (x, w)[i], d)
        assert abs((g * d).sum() - want) <= 1e-7 * (1 + abs(want))


# ------------------------------------------------------------------ refusals in C

def P(n):
    return ctypes.c_void_p(0x10_0000_0000 * n)


def dims(B=2, T=3, Hk=2, Hv=4, K=16, V=8, N=None, dtype=1, **strides):
    d = capi.GdrDims(B, T, Hk, Hv, K, V, B if N is None else N)
    d.q_stride[:] = strides.get("q", (T * Hk * K, Hk * K, K))
    d.k_stride[:] = strides.get("k", (T * Hk * K, Hk * K, K))
    d.v_stride[:] = strides.get("v", (T * Hv * V, Hv * V, V))
    d.dtype, d.scale = dtype, 1.0
    return d


def step(lib, d, p=(1, 2, 3, 4, 5, 6), n_slots=9, slot_stride=4 * 16 * 8, slots=7, out=8):
    ptr = [None if x is None else (x if isinstance(x, ctypes.c_void_p) else P(x)) for x in (*p, slots, out)]
    return lib.gdr_step(d, *ptr[:6], n_slots, slot_stride, ptr[6], ptr[7], None)


def test_step_refusals(lib):
    assert step(lib, None) == E_NULL
    for i in range(6):
        assert step(lib, dims(), p=tuple(None if j == i else j + 1 for j in range(6))) == E_NULL
    assert step(lib, dims(), out=None) == E_NULL
    for bad in (dict(B=-1), dict(T=-1), dict(Hk=0), dict(Hv=0), dict(Hv=3), dict(K=0), dict(K=129), dict(V=0), dict(V=1025),
                dict(N=3), dict(q=(-1, 1, 1)), dict(v=(1 << 60, 1 << 60, 1)), dict(B=1 << 30, T=1 << 30)):
        assert step(lib, dims(**bad)) == E_SHAPE, bad
    assert step(lib, dims(dtype=3)) == E_DTYPE
    assert step(lib, dims(), n_slots=-1) == E_SHAPE
    assert step(lib, dims(), slot_stride=4 * 16 * 8 - 1) == E_SHAPE        # slots that overlap
    assert step(lib, dims(), n_slots=1, slots=None) == E_SHAPE             # fewer slots than rows
    off = lambda n, by: ctypes.c_void_p(P(n).value + by)
    assert step(lib, dims(), p=(off(1, 1), 2, 3, 4, 5, 6)) == E_ALIGN
    assert step(lib, dims(), p=(1, 2, 3, 4, 5, off(6, 2))) == E_ALIGN
    assert step(lib, dims(), out=off(3, 16)) == E_ALIAS                    # out over value
    assert step(lib, dims(), out=off(6, 16)) == E_ALIAS                    # out over the states
    assert step(lib, dims(), slots=off(6, 64)) == E_ALIAS                  # slots in the states
    # nothing to do: no pointer is looked at
    assert step(lib, dims(B=0), p=(None,) * 6, out=None) == OK
    assert step(lib, dims(T=0), p=(None,) * 6, out=None) == OK


def whole(lib, d, p=tuple(range(1, 12)), ws_bytes=None):
    """gdr_fwd: query, key, value, log_decay, beta, offsets, initial_state, out, final_state, saved, workspace."""
    ptr = [None if x is None else (x if isinstance(x, ctypes.c_void_p) else P(x)) for x in p]
    return lib.gdr_fwd(d, *ptr, lib.gdr_workspace_bytes(d, 0) if ws_bytes is None else ws_bytes, None)


def whole_bwd(lib, d, p=tuple(range(1, 17)), ws_bytes=None):
    """gdr_bwd: query .. beta, offsets, saved, d_out, d_final, six gradients, workspace."""
    ptr = [None if x is None else (x if isinstance(x, ctypes.c_void_p) else P(x)) for x in p]
    return lib.gdr_bwd(d, *ptr, lib.gdr_workspace_bytes(d, 1) if ws_bytes is None else ws_bytes, None)


def but(i, x, n=11):
    return tuple(x if j == i else j + 1 for j in range(n))


def test_rule_refusals(lib):
    assert whole(lib, None) == E_NULL and whole_bwd(lib, None) == E_NULL
    for i in (0, 1, 2, 3, 4, 7):
        assert whole(lib, dims(), p=but(i, None)) == E_NULL, i
    packed = dims(B=1, T=9, N=3)
    packed.packed = 1
    assert whole(lib, packed, p=but(5, None)) == E_NULL
    for bad in (dict(B=-1), dict(T=-1), dict(Hv=3), dict(K=0), dict(K=129), dict(V=1025), dict(N=3), dict(k=(1, 1, -1)),
                dict(B=1 << 30, T=1 << 30), dict(T=1 << 31)):
        assert whole(lib, dims(**bad)) == E_SHAPE, bad
        assert lib.gdr_saved_bytes(dims(**bad)) == 0 and lib.gdr_workspace_bytes(dims(**bad), 1) == 0
    two = dims(B=2, N=3)
    two.packed = 1
    assert whole(lib, two) == E_SHAPE                                   # packed rows lie in a batch of one
    assert whole(lib, dims(dtype=-1)) == E_DTYPE
    assert whole(lib, dims(), p=but(10, None)) == E_WS
    assert whole(lib, dims(), ws_bytes=lib.gdr_workspace_bytes(dims(), 0) - 1) == E_WS
    off = lambda n, by: ctypes.c_void_p(P(n).value + by)
    for i, by in ((0, 1), (3, 2), (5, 2), (6, 2), (7, 1), (8, 2), (9, 64), (10, 128)):
        assert whole(lib, dims(), p=but(i, off(i + 1, by))) == E_ALIGN, i
    assert whole(lib, dims(), p=but(7, 3)) == E_ALIAS                   # out over value
    assert whole(lib, dims(), p=but(8, 7)) == E_ALIAS                   # final over initial state
    assert whole(lib, dims(), p=but(9, 11)) == E_ALIAS                  # saved over the workspace
    assert whole(lib, dims(B=0), p=(None,) * 10 + (11,)) == OK
    assert whole_bwd(lib, dims(), p=tuple(range(1, 10)) + (None,) * 6 + (16,)) == OK    # nothing wanted
    for i in (0, 6, 7):
        assert whole_bwd(lib, dims(), p=but(i, None, 16)) == E_NULL, i
    assert whole_bwd(lib, dims(), p=but(15, None, 16)) == E_WS
    assert whole_bwd(lib, dims(), ws_bytes=lib.gdr_workspace_bytes(dims(), 1) - 1) == E_WS
    assert whole_bwd(lib, dims(), p=but(9, 8, 16)) == E_ALIAS           # d_query over d_out
    assert whole_bwd(lib, dims(), p=but(14, 7, 16)) == E_ALIAS          # d_initial over saved
    assert whole_bwd(lib, dims(), p=but(6, off(7, 16), 16)) == E_ALIGN


def qdims(B=2, T=3, Hq=4, Hk=2, D=32, R=16, Pn=64, dtype=1, kind=0, eps=1e-6, **strides):
    d = capi.QknDims(B, T, Hq, Hk, D, R, Pn)
    d.q_stride[:] = strides.get("q", (T * Hq * D, Hq * D, D))
    d.k_stride[:] = strides.get("k", (T * Hk * D, Hk * D, D))
    d.dtype, d.kind, d.eps = dtype, kind, eps
    return d


def norm(lib, d, p=(1, 2, 3, 4, 5, 6, 7, 8, 9)):
    return lib.qkn_fwd(d, *[None if x is None else (x if isinstance(x, ctypes.c_void_p) else P(x)) for x in p], None)


def norm_bwd(lib, d, p=tuple(range(1, 14)), ws=14, ws_bytes=None):
    ptr = [None if x is None else (x if isinstance(x, ctypes.c_void_p) else P(x)) for x in (*p, ws)]
    return lib.qkn_bwd(d, *ptr, lib.qkn_workspace_bytes(d) if ws_bytes is None else ws_bytes, None)


def test_norm_refusals(lib):
    assert norm(lib, None) == E_NULL
    for i in (0, 1, 4, 5, 7, 8):
        assert norm(lib, qdims(), p=tuple(None if j == i else j + 1 for j in range(9))) == E_NULL, i
    for bad in (dict(B=-1), dict(D=0), dict(D=1025), dict(R=-2), dict(R=15), dict(R=34), dict(Pn=-1), dict(Pn=0),
                dict(q=(1, -1, 1)), dict(B=1 << 30, T=1 << 30)):
        assert norm(lib, qdims(**bad)) == E_SHAPE, bad
    assert norm(lib, qdims(Pn=2), p=(1, 2, 3, 4, 5, 6, None, 8, 9)) == E_SHAPE    # fewer table rows than tokens
    assert norm(lib, qdims(dtype=3)) == E_DTYPE
    assert norm(lib, qdims(kind=2)) == E_OPT
    assert norm(lib, qdims(eps=-1.0)) == E_OPT and norm(lib, qdims(eps=float("nan"))) == E_OPT
    off = lambda n, by: ctypes.c_void_p(P(n).value + by)
    assert norm(lib, qdims(), p=(off(1, 1), 2, 3, 4, 5, 6, 7, 8, 9)) == E_ALIGN
    assert norm(lib, qdims(), p=(1, 2, 3, 4, off(5, 2), 6, 7, 8, 9)) == E_ALIGN
    assert norm(lib, qdims(), p=(1, 2, 3, 4, 5, 6, 7, 1, 9)) == E_ALIAS
    assert norm(lib, qdims(), p=(1, 2, 3, 4, 5, 6, 7, 8, 8)) == E_ALIAS
    assert norm(lib, qdims(B=0), p=(None,) * 9) == OK
    assert lib.qkn_workspace_bytes(qdims(D=0)) == 0
    assert norm_bwd(lib, qdims(), p=(*range(1, 10), None, None, None, None)) == OK    # nothing wanted
    assert norm_bwd(lib, qdims(), ws=None) == E_WS
    assert norm_bwd(lib, qdims(), ws_bytes=lib.qkn_workspace_bytes(qdims()) - 1) == E_WS
    assert norm_bwd(lib, qdims(), p=(1, 2, None, *range(4, 14))) == E_NULL            # gradient of an absent weight
    assert norm_bwd(lib, qdims(), p=(*range(1, 8), None, *range(9, 14))) == E_NULL
    assert norm_bwd(lib, qdims(), p=(*range(1, 10), 1, 11, 12, 13)) == E_ALIAS
    assert norm_bwd(lib, qdims(), p=(*range(1, 10), 10, 11, 14, 13)) == E_ALIAS       # weight gradient over the workspace


# ------------------------------------------------------------------ refusals in Python

def cpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_python_refuses_host_tensors_and_gradients():
    q, v, g, s = cpu(1, 2, 1, 4), cpu(1, 2, 1, 4), cpu(1, 2, 1), cpu(1, 1, 4, 4)
    with pytest.raises(ValueError, match="GPU"):
        autograd.gated_delta_step(q, q, v, g, g, s)
    with pytest.raises(ValueError, match="GPU"):
        autograd.qk_norm_rotate(q, q)
    with pytest.raises(ValueError, match="GPU"):
        autograd.gated_delta_rule(q, q, v, g, g, s)
    with pytest.raises(ValueError, match="no gradient"):
        autograd.gated_delta_step(q.clone().requires_grad_(), q, v, g, g, s)
    with pytest.raises(ValueError, match="detach"):
        autograd.qk_norm_rotate(q, q, cos=cpu(2, 2).requires_grad_(), sin=cpu(2, 2))
