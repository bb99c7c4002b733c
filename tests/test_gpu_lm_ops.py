"""Parity of the decoding step of the gated delta rule and of the query/key
norm with the float64 oracles (needs an MI355X).

Tolerance of an output, element by element: half a step of its type relative
to the value, for the one rounding, plus 1e-5 of the largest value for the
float32 arithmetic (sums of at most K + V + tokens products; the probabilistic
rounding model gives sqrt(6 (K + V + T)) 2^-24 <= 5e-6 at the largest sizes
here, the bound leaves a factor 2)."""
import numpy as np
import pytest
import torch

from oracle import lm_ops as ref
from quaternion_cumprod_autodiff_amd import capi, gated_delta_step, qk_norm_rotate

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def f64(t):
    return t.detach().double().cpu().numpy()


def close(label, got, want, rel=None, top=None):
    rel = torch.finfo(got.dtype).eps / 2 if rel is None else rel
    got, want = f64(got), np.asarray(want)
    assert got.shape == want.shape, (label, got.shape, want.shape)
    if not want.size:
        return
    top = float(np.abs(want).max()) if top is None else top
    off = np.abs(got - want) - rel * np.abs(want)
    assert np.isfinite(got).all() and off.max() <= 1e-5 * top + 1e-30, f"{label}: {off.max():.3e} over the rounding, largest {top:.3e}"


def randn(gen, shape, dtype=F32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=F32).to(dtype)


def unit(gen, shape, dtype):
    return torch.nn.functional.normalize(randn(gen, shape), dim=-1).to(dtype)


def step_inputs(B, T, Hk, Hv, K, V, pool, dtype, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    q, k, v = unit(gen, (B, T, Hk, K), dtype), unit(gen, (B, T, Hk, K), dtype), randn(gen, (B, T, Hv, V), dtype)
    g = -torch.rand(B, T, Hv, generator=gen, device=DEV)
    b = torch.rand(B, T, Hv, generator=gen, device=DEV)
    state = randn(gen, (pool, Hv, K, V))
    slots = torch.randperm(pool, generator=gen, device=DEV)[:B].to(torch.int32)
    return q, k, v, g, b, state, slots


def check_step(q, k, v, g, b, state, slots, scale=None, run=gated_delta_step):
    before = f64(state)
    rows = f64(slots).astype(int)
    want, fin = ref.gdr_fwd(*map(f64, (q, k, v, g, b)), before[rows], q.shape[-1] ** -0.5 if scale is None else scale)
    out = run(q, k, v, g, b, state, slots=slots, scale=scale)
    close("out", out, want)
    before[rows] = fin
    close("state", state, before)
    return out


STEPS = [(1, 1, 1, 1, 1, 1, 1), (3, 1, 2, 4, 128, 128, 5), (2, 5, 1, 3, 72, 100, 4), (4, 2, 2, 2, 64, 64, 4), (1, 3, 1, 1, 32, 33, 2),
         (2, 1, 3, 3, 127, 130, 9), (1, 2, 1, 2, 5, 1024, 1), (2, 9, 1, 1, 33, 4, 70), (70, 1, 1, 1, 16, 8, 300), (2, 1, 2, 2, 100, 64, 3)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("size", STEPS, ids=str)
def test_step(size, dtype):
    print(f"[step {size} {dtype}]", flush=True)
    check_step(*step_inputs(*size, dtype, seed=sum(size)))


def test_step_scale_strides_and_a_view_of_a_larger_pool():
    q, k, v, g, b, state, slots = step_inputs(3, 2, 2, 4, 64, 64, 6, BF16, seed=3)
    fused = torch.randn(3, 2, 8 * 64 + 3, device=DEV).to(BF16)     # rows whose starts are on 2 bytes only
    qs, ks, vs = fused[..., 1:129].unflatten(-1, (2, 64)), fused[..., 129:257].unflatten(-1, (2, 64)), fused[..., 257:513].unflatten(-1, (4, 64))
    qs.copy_(q), ks.copy_(k), vs.copy_(v)
    check_step(qs, ks, vs, g, b, state.clone(), slots, scale=0.3)
    layers = torch.randn(6, 3, 4, 64, 64, device=DEV)
    kept = layers.clone()
    check_step(q, k, v, g, b, layers[:, 1], slots)                  # one layer of a pool that holds three
    assert torch.equal(layers[:, 0], kept[:, 0]) and torch.equal(layers[:, 2], kept[:, 2])
    check_step(q[:, :, :1].expand(3, 2, 2, 64), k, v, g, b, state.clone(), slots)   # one query head for all


def test_step_skips_padding_and_later_rows_of_the_same_slot():
    q, k, v, g, b, state, _ = step_inputs(7, 2, 1, 2, 48, 40, 5, BF16, seed=8)
    slots = torch.tensor([3, -1, 0, 3, 5, 2 ** 31 - 1, 4], dtype=torch.int32, device=DEV)
    before = state.clone()
    out = gated_delta_step(q, k, v, g, b, state, slots=slots)
    run = [0, 2, 6]
    want, fin = ref.gdr_fwd(*(f64(x)[run] for x in (q, k, v, g, b)), f64(before)[[3, 0, 4]], 48 ** -0.5)
    close("out", out[run], want)
    assert not out[[1, 3, 4, 5]].any()
    close("state", state[[3, 0, 4]], fin)
    assert torch.equal(state[[1, 2]], before[[1, 2]])


def test_step_clears_a_state_at_a_decay_of_zero_and_keeps_it_at_beta_zero():
    q, k, v, g, b, state, slots = step_inputs(2, 1, 1, 2, 32, 16, 2, F32, seed=9)
    g[:] = -float("inf")
    check_step(q, k, v, g, b, state, slots)
    kept = state.clone()
    gated_delta_step(q, k, v, torch.zeros_like(g), torch.zeros_like(b), state, slots=slots)
    assert torch.equal(state, kept)


def test_step_with_nothing_to_do():
    q, k, v, g, b, state, slots = step_inputs(2, 3, 1, 2, 32, 16, 4, BF16)
    kept = state.clone()
    assert gated_delta_step(q[:0], k[:0], v[:0], g[:0], b[:0], state, slots=slots[:0]).shape == (0, 3, 2, 16)
    assert gated_delta_step(q[:, :0], k[:, :0], v[:, :0], g[:, :0], b[:, :0], state, slots=slots).shape == (2, 0, 2, 16)
    assert not gated_delta_step(q, k, v, g, b, state[:0], slots=slots).any()
    assert torch.equal(state, kept)


def test_step_on_many_large_states():
    # 136 MB of states, which pass by the caches, against the same rows in two calls of half as many
    args = step_inputs(70, 2, 4, 32, 128, 120, 70, BF16, seed=6)
    q, k, v, g, b, state, slots = args
    twin = state.clone()
    out = gated_delta_step(q, k, v, g, b, state, slots=slots)
    for rows in (slice(0, 35), slice(35, 70)):
        part = gated_delta_step(q[rows], k[rows], v[rows], g[rows], b[rows], twin, slots=slots[rows])
        assert torch.equal(part, out[rows])
    assert torch.equal(state, twin)


def test_step_on_another_stream_and_in_a_graph():
    size = (5, 1, 2, 4, 128, 128, 8)
    q, k, v, g, b, state, slots = step_inputs(*size, BF16, seed=4)
    twin, third = state.clone(), state.clone()
    want = [gated_delta_step(q, k, v, g, b, state, slots=slots).clone() for _ in range(4)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        got = capi.gdr_step(q, k, v, g, b, twin, slots, stream=side)
        side.synchronize()
        assert torch.equal(got, want[i])
    assert torch.equal(twin, state)
    start = third.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gated_delta_step(q, k, v, g, b, third, slots=slots)
    third.copy_(start)
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
    assert torch.equal(third, state)


def test_step_refusals():
    q, k, v, g, b, state, slots = step_inputs(2, 1, 2, 4, 32, 16, 4, BF16)
    call = lambda **kw: gated_delta_step(**{**dict(query=q, key=k, value=v, log_decay=g, beta=b, state=state, slots=slots), **kw})
    for kw in (dict(key=k[:, :, :1]), dict(value=v[:, :, :3]), dict(value=v[:1]), dict(log_decay=g[:1]), dict(log_decay=g.to(BF16)),
               dict(beta=b.double()), dict(state=state.to(BF16)), dict(state=state[:, :, :, :8]), dict(state=state.transpose(2, 3)),
               dict(slots=slots.long()), dict(slots=slots[:1]), dict(slots=None, state=state[:1]), dict(query=q[0]),
               dict(query=q.transpose(2, 3)), dict(log_decay=g.cpu())):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    for kw in (dict(key=k.to(F16)), dict(query=q.double(), key=k.double(), value=v.double())):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(capi.QuatCumprodError):                       # a slot that every row shares
        call(state=state[:1].expand(4, 4, 32, 16))
    torch.cuda.synchronize()


# ------------------------------------------------------------------------ norms

def norm_inputs(B, T, Hq, Hk, D, R, table, dtype, weights, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    q, k = randn(gen, (B, T, Hq, D), dtype), randn(gen, (B, T, Hk, D), dtype)
    wq, wk = (randn(gen, (D,), dtype), randn(gen, (D,), dtype)) if weights else (None, None)
    cos = sin = pos = None
    if R:
        angle = randn(gen, (table, R // 2)) * 3
        cos, sin = angle.cos(), angle.sin()
        pos = torch.randint(0, table, (B, T), generator=gen, device=DEV, dtype=torch.int32)
    return q, k, wq, wk, cos, sin, pos


def host(t):
    return None if t is None else (f64(t) if t.is_floating_point() else t.cpu().numpy())


def largest_term(x, w, cos, sin, pos, kind, eps, interleaved, dy):
    """The gradient of a head is dx = r dh - x r^3 c / size, a projection: its two terms cancel (fully for one element,
    where dx = r dh eps r^2).  In float32 each term carries its own few roundings of 2^-24, so the error of dx is
    that share of the terms, however small their difference: the 1e-5 is of the largest |r dh| + |x r^3 c / size|."""
    size = x.shape[-1] if kind == "rms" else 1
    r = 1 / np.sqrt((x * x).sum(-1, keepdims=True) / size + eps)
    dn = dy if cos is None else ref._turn(dy, cos, sin, ref._rows(x, pos), interleaved, -1.0)
    dh = dn if w is None else dn * w
    return float((np.abs(r * dh) + np.abs(x) * r ** 3 * np.abs((dh * x).sum(-1, keepdims=True)) / size).max())


def check_norm(q, k, wq, wk, cos, sin, pos, kind="rms", eps=1e-6, interleaved=False, seed=1):
    how = (host(cos), host(sin), host(pos), kind, eps, interleaved)
    leaves = [t.detach().requires_grad_() if t is not None else None for t in (q, k, wq, wk)]
    qo, ko = qk_norm_rotate(*leaves, cos, sin, pos, kind=kind, eps=eps, interleaved=interleaved)
    close("query", qo, ref.qkn_fwd(f64(q), host(wq), *how))
    close("key", ko, ref.qkn_fwd(f64(k), host(wk), *how))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dq, dk = randn(gen, qo.shape, q.dtype), randn(gen, ko.shape, q.dtype)
    some = [t for t in leaves if t is not None]
    grads = dict(zip([n for n, t in zip("qkwz", leaves) if t is not None], torch.autograd.grad([qo, ko], some, [dq, dk])))
    for x, w, d, a, c in ((q, wq, dq, "q", "w"), (k, wk, dk, "k", "z")):
        want, want_w = ref.qkn_bwd(f64(x), host(w), *how, f64(d))
        close("gradient " + a, grads[a], want, top=largest_term(f64(x), host(w), *how, f64(d)))
        if w is not None:
            close("gradient " + c, grads[c], want_w)
    return qo, ko


NORMS = [(1, 1, 1, 1, 1, 0, 1), (2, 3, 4, 2, 128, 128, 9), (1, 70, 2, 1, 128, 64, 500), (3, 7, 5, 3, 90, 42, 8), (1, 5, 1, 2, 64, 0, 1),
         (1, 9, 3, 1, 256, 256, 20), (2, 2, 1, 1, 512, 16, 3), (1, 3, 2, 1, 1024, 1024, 3), (1, 3, 1, 1, 1023, 1000, 3), (1, 4, 2, 2, 2, 2, 4),
         (1, 11, 2, 1, 80, 80, 12), (1, 2, 3, 1, 300, 6, 2), (1, 1200, 3, 2, 16, 16, 50)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size", NORMS, ids=str)
def test_norm(size, interleaved, dtype):
    print(f"[norm {size} {interleaved} {dtype}]", flush=True)
    check_norm(*norm_inputs(*size, dtype, True, seed=sum(size)), interleaved=interleaved)
    check_norm(*norm_inputs(*size, dtype, False, seed=sum(size)), kind="l2", eps=1e-3, interleaved=interleaved)


@pytest.mark.parametrize("size", [(1, 8300, 3, 2, 6, 4, 50), (2, 16500, 8, 4, 128, 128, 300), (1, 33000, 7, 2, 128, 64, 300)], ids=str)
def test_norm_of_many_heads_equals_its_parts(size):
    """Calls so large that a group takes four heads in a row, against slices of their tokens small enough for one each."""
    print(f"[norm {size}]", flush=True)
    q, k, wq, wk, cos, sin, pos = norm_inputs(*size, BF16, True, seed=3)
    whole = [t.detach().requires_grad_() for t in (q, k, wq, wk)]
    out = qk_norm_rotate(*whole, cos, sin, pos)
    cot = [torch.randn_like(t) for t in out]
    grads = torch.autograd.grad(out, whole, cot)
    half = 2.0 ** -8
    sums = [torch.zeros(size[4], dtype=torch.float64, device=DEV) for _ in range(2)]
    step = 700
    for t0 in range(0, size[1], step):
        cut = slice(t0, t0 + step)
        leaves = [t[:, cut].detach().float().requires_grad_() for t in (q, k)] + [t.detach().float().requires_grad_() for t in (wq, wk)]
        part = qk_norm_rotate(*leaves, cos, sin, pos[:, cut].contiguous())
        pg = torch.autograd.grad(part, leaves, [c[:, cut].float() for c in cot])
        for a, b in zip((*out, *grads[:2]), (*part, *pg[:2])):         # the part in float32: the whole rounds once more
            a, b = a[:, cut].double(), b.double()
            assert ((a - b).abs() <= half * b.abs() + 1e-5 * b.abs().max()).all()
        for s, g in zip(sums, pg[2:]):
            s += g.double()
    for a, b in zip(grads[2:], sums):
        assert ((a.double() - b).abs() <= half * b.abs() + 1e-5 * b.abs().max()).all()


def test_norm_of_strided_views_positions_of_64_bits_and_none():
    q, k, wq, wk, cos, sin, pos = norm_inputs(2, 6, 4, 2, 64, 32, 30, BF16, True, seed=2)
    for lead in (0, 8, 1):                                           # rows on 16 bytes, and on 2
        fused = torch.zeros(2, 6, lead + 6 * 64 + 8, device=DEV, dtype=BF16)
        qs, ks = fused[..., lead:lead + 256].unflatten(-1, (4, 64)), fused[..., lead + 256:lead + 384].unflatten(-1, (2, 64))
        qs.copy_(q), ks.copy_(k)
        check_norm(qs, ks, wq, wk, cos, sin, pos.long())
    check_norm(q.transpose(1, 2).contiguous().transpose(1, 2), k, wq, wk, cos, sin, None)     # heads before tokens
    check_norm(q[:, :1].expand(2, 6, 4, 64), k, wq, None, cos, sin, pos)
    got = qk_norm_rotate(q.transpose(2, 3).contiguous().transpose(2, 3), k, wq, wk, cos, sin, pos)
    assert all(torch.equal(a, b) for a, b in zip(got, qk_norm_rotate(q, k, wq, wk, cos, sin, pos)))


def test_norm_of_a_position_outside_the_table_is_nan_and_of_a_zero_head_zero():
    q, k, wq, wk, cos, sin, pos = norm_inputs(1, 4, 2, 1, 64, 64, 10, BF16, True)
    pos[0] = torch.tensor([0, 10, -1, 9], dtype=torch.int32)
    q[0, 0] = 0
    qo, ko = qk_norm_rotate(q, k, wq, wk, cos, sin, pos)
    assert qo[0, 1:3].isnan().all() and ko[0, 1:3].isnan().all()
    assert not qo[0, [0, 3]].isnan().any() and not ko[0, [0, 3]].isnan().any() and not qo[0, 0].any()


def test_norm_with_nothing_to_do_and_of_one_side_alone():
    q, k, wq, wk, cos, sin, pos = norm_inputs(2, 3, 4, 2, 64, 64, 10, BF16, True)
    a, b = qk_norm_rotate(q[:, :0], k[:, :0], wq, wk, cos, sin, pos[:, :0])
    assert a.shape == (2, 0, 4, 64) and b.shape == (2, 0, 2, 64)
    leaf = wq.clone().requires_grad_()
    a, b = qk_norm_rotate(q[:, :0], k[:, :0], leaf, wk)
    assert not torch.autograd.grad([a, b], [leaf], [a.detach(), b.detach()])[0].any()
    a, b = qk_norm_rotate(q, k[:, :, :0], wq, wk, cos, sin, pos)
    assert torch.equal(a, qk_norm_rotate(q, k, wq, wk, cos, sin, pos)[0]) and b.numel() == 0
    leaf = k.clone().requires_grad_()                                 # only one input's gradient, one output's cotangent
    a, b = qk_norm_rotate(q, leaf, wq, wk, cos, sin, pos)
    g, = torch.autograd.grad(b.float().square().sum(), [leaf])
    want, _ = ref.qkn_bwd(f64(k), f64(wk), f64(cos), f64(sin), host(pos), "rms", 1e-6, False, f64(2 * b.float()).astype(np.float32).astype(np.float64))
    close("gradient k", g, want, rel=torch.finfo(BF16).eps)           # the cotangent is rounded once too


def test_norm_in_a_graph_and_twice_the_same_bits():
    args = norm_inputs(2, 130, 8, 2, 128, 128, 256, BF16, True, seed=5)
    d = [torch.randn_like(t) for t in args[:2]]
    want = capi.qkn_fwd(*args) + capi.qkn_bwd(*args, *d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = capi.qkn_fwd(*args) + capi.qkn_bwd(*args, *d)
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        again = capi.qkn_fwd(*args) + capi.qkn_bwd(*args, *d)
        assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_norm_refusals():
    q, k, wq, wk, cos, sin, pos = norm_inputs(2, 3, 4, 2, 64, 32, 10, BF16, True)
    call = lambda **kw: qk_norm_rotate(**{**dict(query=q, key=k, query_weight=wq, key_weight=wk, cos=cos, sin=sin, positions=pos), **kw})
    for kw in (dict(key=k[:1]), dict(key=k[..., :32]), dict(query=q[0]), dict(query_weight=wq[:5]), dict(key_weight=wk.float()), dict(sin=None),
               dict(cos=None, sin=None), dict(cos=cos.to(BF16)), dict(sin=sin[:5]), dict(cos=cos[:2], sin=sin[:2], positions=None),
               dict(positions=pos[:1]), dict(positions=pos.float()), dict(kind="max"), dict(eps=-1.0), dict(cos=torch.zeros(4, 40, device=DEV), sin=torch.zeros(4, 40, device=DEV)),
               dict(query=q.double(), key=k.double()), dict(key=k.to(F16)), dict(positions=pos.cpu())):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    torch.cuda.synchronize()
