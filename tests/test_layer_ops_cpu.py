"""Linear attention with decays, its decoding step and layer norm without a GPU:
their oracles against differences, the headers' names, and the refusals in C
(fake device pointers: every one of these calls returns before any HIP call)
and in Python."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

from oracle import layer_ops as ref
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
    for h in ("decay_attention.h", "layer_norm.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", h)).read(), flags=re.S)
        names |= set(re.findall(r"\b((?:dca|lnm)_\w+)\s*\(", text))
    assert sorted(names) == sorted(capi.LAYER_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names == set(re.findall(r"\bT ((?:dca|lnm)_\w+)", out))


# ------------------------------------------------------------------ the oracles

def central(f, x, d, eps=1e-5):
    """The directional derivative of the number f(x) along d."""
    return (f(x + eps * d) - f(x - eps * d)) / (2 * eps)


@pytest.mark.parametrize("by_head", [False, True])
@pytest.mark.parametrize("lengths", [None, [3, 0, 1, 2]])
def test_attention_oracle_gradients_match_differences(lengths, by_head):
    rng = np.random.default_rng(5)
    B, T, Hk, Hv, K, V = (2, 5, 2, 4, 3, 4) if lengths is None else (1, 7, 1, 3, 4, 2)
    N = B if lengths is None else len(lengths)
    x = [rng.standard_normal(s) for s in [(B, T, Hk, K)] * 2 + [(B, T, Hv, V)]]
    x += [-rng.random((Hv,) if by_head else (B, T, Hv)), rng.standard_normal((N, Hv, K, V))]
    w_out, w_fin = rng.standard_normal((B, T, Hv, V)), rng.standard_normal((N, Hv, K, V))

    def loss(*a):
        out, fin = ref.dca_fwd(*a, 0.7, lengths)
        return (out * w_out).sum() + (fin * w_fin).sum()

    grads = ref.dca_bwd(*x, 0.7, w_out, w_fin, lengths)
    for i, g in enumerate(grads):
        assert g.shape == x[i].shape
        d = rng.standard_normal(x[i].shape)
        want = central(lambda y: loss(*x[:i], y, *x[i + 1:]), x[i], d)
        assert abs((g * d).sum() - want) <= 1e-7 * (1 + abs(want)), i


def test_attention_oracle_by_hand():
    # One head, K = 1, V = 1: S = a S + k v; o = s S q.
    one = lambda *v: np.array(v, dtype=np.float64).reshape(1, -1, 1, 1)
    out, fin = ref.dca_fwd(one(1, 2), one(1, 0.5), one(3, 5), np.log(one(0.5, 0.25))[..., 0], np.array([[[[2.0]]]]), 10.0)
    # t = 0: S = 1 + 3 = 4, o = 40;  t = 1: S = 1 + 2.5 = 3.5, o = 70
    assert out.ravel().tolist() == [40.0, 70.0] and fin.ravel().tolist() == [3.5]


@pytest.mark.parametrize("by_head", [False, True])
def test_norm_oracle_gradients_match_differences(by_head):
    rng = np.random.default_rng(7)
    x, dy = rng.standard_normal((2, 3, 4, 5)), rng.standard_normal((2, 3, 4, 5))
    shape = (4, 5) if by_head else (5,)
    w, b = rng.standard_normal(shape), rng.standard_normal(shape)
    grads = ref.lnm_bwd(x, w, 1e-3, dy, by_head)
    for i, g in enumerate(grads):
        at = [x, w, b]
        assert g.shape == at[i].shape
        d = rng.standard_normal(g.shape)
        want = central(lambda y: (ref.lnm_fwd(*at[:i], y, *at[i + 1:], 1e-3) * dy).sum(), at[i], d)
        assert abs((g * d).sum() - want) <= 1e-7 * (1 + abs(want)), i


def test_norm_oracle_by_hand():
    # mean 2, variance 2/3 + 1/3 = 1 with eps
    assert np.allclose(ref.lnm_fwd(np.array([1.0, 2.0, 3.0]), np.array([1.0, 2.0, 3.0]), np.array([0.0, 0.5, 0.0]), 1 / 3), [-1, 0.5, 3])


# ------------------------------------------------------------------ refusals in C

def P(n):
    return ctypes.c_void_p(0x10_0000_0000 * n)


def off(n, by):
    return ctypes.c_void_p(P(n).value + by)


def pointers(p):
    return [None if x is None else (x if isinstance(x, ctypes.c_void_p) else P(x)) for x in p]


def but(i, x, n):
    return tuple(x if j == i else j + 1 for j in range(n))


def dims(B=2, T=3, Hk=2, Hv=4, K=16, V=8, N=None, dtype=1, packed=0, head=0, **strides):
    d = capi.DcaDims(B, T, Hk, Hv, K, V, B if N is None else N)
    d.q_stride[:] = strides.get("q", (T * Hk * K, Hk * K, K))
    d.k_stride[:] = strides.get("k", (T * Hk * K, Hk * K, K))
    d.v_stride[:] = strides.get("v", (T * Hv * V, Hv * V, V))
    d.dtype, d.scale, d.packed, d.head_decay = dtype, 1.0, packed, head
    return d


def step(lib, d, p=(1, 2, 3, 4, 5), n_slots=9, slot_stride=4 * 16 * 8, slots=7, out=8):
    ptr = pointers((*p, slots, out))
    return lib.dca_step(d, *ptr[:5], n_slots, slot_stride, ptr[5], ptr[6], None)


def test_step_refusals(lib):
    assert step(lib, None) == E_NULL
    for i in range(5):
        assert step(lib, dims(), p=but(i, None, 5)) == E_NULL
    assert step(lib, dims(), out=None) == E_NULL
    for bad in (dict(B=-1), dict(T=-1), dict(Hk=0), dict(Hv=0), dict(Hv=3), dict(K=0), dict(K=129), dict(V=0), dict(V=1025),
                dict(N=3), dict(q=(-1, 1, 1)), dict(v=(1 << 60, 1 << 60, 1)), dict(B=1 << 30, T=1 << 30)):
        assert step(lib, dims(**bad)) == E_SHAPE, bad
    assert step(lib, dims(dtype=3)) == E_DTYPE
    assert step(lib, dims(), n_slots=-1) == E_SHAPE
    assert step(lib, dims(), slot_stride=4 * 16 * 8 - 1) == E_SHAPE        # slots that overlap
    assert step(lib, dims(), n_slots=1, slots=None) == E_SHAPE             # fewer slots than rows
    assert step(lib, dims(), p=(off(1, 1), 2, 3, 4, 5)) == E_ALIGN
    assert step(lib, dims(), p=(1, 2, 3, off(4, 2), 5)) == E_ALIGN
    assert step(lib, dims(), p=(1, 2, 3, 4, off(5, 2))) == E_ALIGN
    assert step(lib, dims(), out=off(3, 16)) == E_ALIAS                    # out over value
    assert step(lib, dims(), out=off(5, 16)) == E_ALIAS                    # out over the states
    assert step(lib, dims(), slots=off(5, 64)) == E_ALIAS                  # slots in the states
    assert step(lib, dims(head=1), out=off(4, 8)) == E_ALIAS               # out over the heads' four decays
    # nothing to do: no pointer is looked at
    assert step(lib, dims(B=0), p=(None,) * 5, out=None) == OK
    assert step(lib, dims(T=0), p=(None,) * 5, out=None) == OK


@pytest.mark.parametrize("n,code", [(1082401, E_ALIAS), (1082402, E_SHAPE)])
def test_step_takes_what_the_header_says(lib, n, code):
    """31 pieces of 32 columns: 1082401 rows are 2^25 - 1 of them, and are refused for out in the states alone."""
    assert step(lib, dims(n, 1, 1, 1, 1, 992), n_slots=n, slot_stride=992, out=off(5, 16)) == code


def whole(lib, d, p=tuple(range(1, 11)), ws_bytes=None):
    """dca_fwd: query, key, value, log_decay, offsets, initial_state, out, final_state, saved, workspace."""
    return lib.dca_fwd(d, *pointers(p), lib.dca_workspace_bytes(d, 0) if ws_bytes is None else ws_bytes, None)


def whole_bwd(lib, d, p=tuple(range(1, 15)), ws_bytes=None):
    """dca_bwd: query .. log_decay, offsets, saved, d_out, d_final, five gradients, workspace."""
    return lib.dca_bwd(d, *pointers(p), lib.dca_workspace_bytes(d, 1) if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("head", [0, 1])
def test_attention_refusals(lib, head):
    make = lambda **kw: dims(head=head, **kw)
    assert whole(lib, None) == E_NULL and whole_bwd(lib, None) == E_NULL
    for i in (0, 1, 2, 3, 6):
        assert whole(lib, make(), p=but(i, None, 10)) == E_NULL, i
    assert whole(lib, make(B=1, T=9, N=3, packed=1), p=but(4, None, 10)) == E_NULL
    for bad in (dict(B=-1), dict(T=-1), dict(Hv=3), dict(K=0), dict(K=129), dict(V=1025), dict(N=3), dict(k=(1, 1, -1)),
                dict(B=1 << 30, T=1 << 30), dict(T=1 << 31), dict(B=2, N=3, packed=1), dict(B=1, T=9, N=-1, packed=1)):
        assert whole(lib, make(**bad)) == E_SHAPE, bad
        assert lib.dca_saved_bytes(make(**bad)) == 0 and lib.dca_workspace_bytes(make(**bad), 1) == 0
    assert whole(lib, make(dtype=-1)) == E_DTYPE
    assert whole(lib, make(), p=but(9, None, 10)) == E_WS
    assert whole(lib, make(), ws_bytes=lib.dca_workspace_bytes(make(), 0) - 1) == E_WS
    for i, by in ((0, 1), (3, 2), (4, 2), (5, 2), (6, 1), (7, 2), (8, 64), (9, 128)):
        assert whole(lib, make(), p=but(i, off(i + 1, by), 10)) == E_ALIGN, i
    assert whole(lib, make(), p=but(6, 3, 10)) == E_ALIAS                   # out over value
    assert whole(lib, make(), p=but(7, 6, 10)) == E_ALIAS                   # final over initial state
    assert whole(lib, make(), p=but(8, 10, 10)) == E_ALIAS                  # saved over the workspace
    assert whole(lib, make(B=0), p=(None,) * 9 + (10,)) == OK
    assert whole_bwd(lib, make(), p=tuple(range(1, 9)) + (None,) * 5 + (14,)) == OK    # nothing wanted
    for i in (0, 3, 5, 6):
        assert whole_bwd(lib, make(), p=but(i, None, 14)) == E_NULL, i
    assert whole_bwd(lib, make(), p=but(13, None, 14)) == E_WS
    assert whole_bwd(lib, make(), ws_bytes=lib.dca_workspace_bytes(make(), 1) - 1) == E_WS
    assert whole_bwd(lib, make(), p=but(8, 7, 14)) == E_ALIAS               # d_query over d_out
    assert whole_bwd(lib, make(), p=but(11, 4, 14)) == E_ALIAS              # d_log_decay over log_decay
    assert whole_bwd(lib, make(), p=but(12, 6, 14)) == E_ALIAS              # d_initial over saved
    assert whole_bwd(lib, make(), p=but(5, off(6, 16), 14)) == E_ALIGN
    assert whole_bwd(lib, make(), p=but(11, off(12, 2), 14)) == E_ALIGN


@pytest.mark.parametrize("size,ok", [
    ((1, 1, 16384, 16384, 1, 1024), True),          # 2^18 of (sequence, head, 64 columns)
    ((31, 1, 16384, 16384, 1, 1024), True),         # 31 * 2^18, just below 2^23
    ((32, 1, 16384, 16384, 1, 1024), False),        # 2^23
    ((1, 1, 1, 65536, 1, 1024), False),             # one key head is rounded up to eight: 8 * 2^20
    ((1, 1, 1, 65536, 1, 960), True),
    ((1, 1, 1 << 20, 1 << 20, 1, 64), True),
    ((1, 1, 1 << 20, 1 << 21, 1, 16), False),       # heads
    ((1, 32 * 511, 16384, 16384, 1, 1), True),      # chunks of 32: 511 * 2^14
    ((1, 32 * 511 + 1, 16384, 16384, 1, 1), False),
], ids=str)
def test_attention_takes_what_the_header_says(lib, size, ok):
    d = dims(*size)
    for n in (lib.dca_workspace_bytes(d, 0), lib.dca_workspace_bytes(d, 1), lib.dca_saved_bytes(d)):
        assert (n > 0) == ok


def test_packed_chunks_count_a_slot_more_for_each_sequence(lib):
    assert lib.dca_workspace_bytes(dims(1, 32 * 500, 16384, 16384, 1, 1, N=11, packed=1), 0) > 0
    assert lib.dca_workspace_bytes(dims(1, 32 * 500, 16384, 16384, 1, 1, N=12, packed=1), 0) == 0


def ldims(B=2, T=3, H=4, D=32, dtype=1, by_head=0, eps=1e-5, x=None):
    d = capi.LnmDims(B, T, H, D)
    d.x_stride[:] = x or (T * H * D, H * D, D)
    d.dtype, d.by_head, d.eps = dtype, by_head, eps
    return d


def norm(lib, d, p=(1, 2, 3, 4, 5)):
    return lib.lnm_fwd(d, *pointers(p), None)


def norm_bwd(lib, d, p=tuple(range(1, 8)), ws=8, ws_bytes=None):
    """lnm_bwd: x, weight, stats, d_y, d_x, d_weight, d_bias."""
    return lib.lnm_bwd(d, *pointers((*p, ws)), lib.lnm_workspace_bytes(d) if ws_bytes is None else ws_bytes, None)


def test_norm_refusals(lib):
    assert norm(lib, None) == E_NULL and norm_bwd(lib, None) == E_NULL and lib.lnm_workspace_bytes(None) == 0
    for i in (0, 3):
        assert norm(lib, ldims(), p=but(i, None, 5)) == E_NULL, i
    for bad in (dict(B=-1), dict(T=-1), dict(H=-1), dict(D=0), dict(D=16385), dict(x=(1, -1, 1)), dict(B=1 << 30, T=1 << 30),
                dict(H=(1 << 20) + 1), dict(H=1 << 20, D=2048, by_head=1)):
        assert norm(lib, ldims(**bad)) == E_SHAPE, bad
        assert lib.lnm_workspace_bytes(ldims(**bad)) == 0
    assert norm(lib, ldims(dtype=3)) == E_DTYPE
    assert norm(lib, ldims(eps=-1.0)) == E_OPT and norm(lib, ldims(eps=float("nan"))) == E_OPT
    for i, by in ((0, 1), (1, 1), (2, 1), (3, 1), (4, 8)):
        assert norm(lib, ldims(), p=but(i, off(i + 1, by), 5)) == E_ALIGN, i
    for p in ((1, 2, 3, 1, 5), (1, 2, 3, 2, 5), (1, 2, 3, 4, 1), (1, 2, 3, 4, 4)):
        assert norm(lib, ldims(), p=p) == E_ALIAS, p
    assert norm(lib, ldims(B=0), p=(None,) * 5) == OK
    assert norm_bwd(lib, ldims(), p=(1, 2, 3, 4, None, None, None)) == OK              # nothing wanted
    assert norm_bwd(lib, ldims(H=0, by_head=1), p=(None,) * 4 + (5, 6, 7)) == OK
    for i in (0, 1, 2, 3):                                                             # 1: gradient of an absent weight
        assert norm_bwd(lib, ldims(), p=but(i, None, 7)) == E_NULL, i
    assert norm_bwd(lib, ldims(), ws=None) == E_WS
    assert norm_bwd(lib, ldims(), ws_bytes=lib.lnm_workspace_bytes(ldims()) - 1) == E_WS
    assert norm_bwd(lib, ldims(), ws=off(8, 8)) == E_ALIGN
    for i, by in ((0, 1), (2, 8), (4, 1), (5, 1), (6, 1)):
        assert norm_bwd(lib, ldims(), p=but(i, off(i + 1, by), 7)) == E_ALIGN, i
    for i, x in ((4, 1), (4, 4), (5, 2), (6, 6), (5, 8), (4, 3)):
        assert norm_bwd(lib, ldims(), p=but(i, x, 7)) == E_ALIAS, (i, x)


# ------------------------------------------------------------------ refusals in Python

def cpu(*shape):
    return torch.zeros(*shape)


def test_python_refuses_host_tensors_and_gradients():
    q, v, g, s = cpu(1, 2, 1, 4), cpu(1, 2, 1, 4), cpu(1, 2, 1), cpu(1, 1, 4, 4)
    for decay in (g, cpu(1)):
        with pytest.raises(ValueError, match="GPU"):
            autograd.decay_attention(q, q, v, decay, s)
        with pytest.raises(ValueError, match="GPU"):
            autograd.decay_attention_step(q, q, v, decay, s)
    with pytest.raises(ValueError, match="GPU"):
        autograd.layer_norm(q)
    with pytest.raises(ValueError, match="no gradient"):
        autograd.decay_attention_step(q.clone().requires_grad_(), q, v, g, s)
    with pytest.raises(ValueError, match="axes"):
        autograd.layer_norm(torch.zeros(()))


@pytest.mark.parametrize("shape", [(2, 3, 0, 4, 5), (0, 2, 3, 4, 5), (2, 2, 3, 4, 0, 5)], ids=str)
def test_empty_rows_of_many_axes_reach_the_checks(shape):
    with pytest.raises(ValueError, match="GPU"):
        autograd.layer_norm(cpu(*shape))


@pytest.mark.parametrize("tracked", [False, True])
def test_forward_mode_is_refused_and_not_dropped(tracked):
    q, v, g, s = cpu(1, 2, 1, 4), cpu(1, 2, 1, 4), cpu(1, 2, 1), cpu(1, 1, 4, 4)
    args = {"query": q, "key": q.clone(), "value": v, "log_decay": g}
    dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))
    with forward_ad.dual_level():
        for name in args:
            duals = {n: dual(t) if n == name else t.clone().requires_grad_(tracked) for n, t in args.items()}
            with pytest.raises(NotImplementedError, match="forward"):
                autograd.decay_attention(**duals)
            with pytest.raises(NotImplementedError, match="forward"):
                autograd.decay_attention_step(**duals, state=s)
        with pytest.raises(NotImplementedError, match="forward"):
            autograd.decay_attention(**args, initial_state=dual(s))
        with pytest.raises(NotImplementedError, match="forward"):
            autograd.decay_attention_step(**args, state=dual(s))
        x, w = cpu(3, 4).requires_grad_(tracked), cpu(4)
        for call in (dict(x=dual(cpu(3, 4))), dict(x=x, weight=dual(w)), dict(x=x, bias=dual(w))):
            with pytest.raises(NotImplementedError, match="forward"):
                autograd.layer_norm(**call)
