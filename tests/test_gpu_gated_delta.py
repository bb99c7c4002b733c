"""Parity of the whole-sequence gated delta rule and its VJP with the float64
oracle (needs an MI355X).

Tolerance of an output, element by element: half a step of its type relative
to the value, for the one rounding, plus 1e-5 of the largest value for the
float32 arithmetic.  Products are exact to 2^-23 (three bfloat16 parts hold 24
bits; the dropped products are below 2^-24) and are summed in float32 over at
most K + V + 64 terms a chunk; the decays forget a chunk's error.  The
probabilistic rounding model gives sqrt(6 (K + V + 64)) 2^-23 <= 6e-6 at the
largest sizes here, and the bound leaves less than a factor 2."""
import numpy as np
import pytest
import torch

from oracle import lm_ops as ref
from quaternion_cumprod_autodiff_amd import capi, gated_delta_rule, gated_delta_step, qk_norm_rotate

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def f64(t):
    return t.detach().double().cpu().numpy()


def close(label, got, want):
    rel = torch.finfo(got.dtype).eps / 2
    got, want = f64(got), np.asarray(want)
    assert got.shape == want.shape, (label, got.shape, want.shape)
    if not want.size:
        return 0.0
    top = float(np.abs(want).max())
    off = float((np.abs(got - want) - rel * np.abs(want)).max())
    assert np.isfinite(got).all() and off <= 1e-5 * top + 1e-30, f"{label}: {off:.3e} over the rounding, largest {top:.3e}"
    return max(off, 0.0) / max(top, 1e-30)


def randn(gen, shape, dtype=F32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=F32).to(dtype)


def unit(gen, shape, dtype):
    return torch.nn.functional.normalize(randn(gen, shape), dim=-1).to(dtype)


def inputs(B, T, Hk, Hv, K, V, dtype, N=None, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    N = B if N is None else N
    q, k, v = unit(gen, (B, T, Hk, K), dtype), unit(gen, (B, T, Hk, K), dtype), randn(gen, (B, T, Hv, V), dtype)
    rate = torch.logspace(-2, 0.5, Hv, device=DEV)
    g = -torch.rand(B, T, Hv, generator=gen, device=DEV) * rate
    b = torch.rand(B, T, Hv, generator=gen, device=DEV)
    return [q, k, v, g, b, randn(gen, (N, Hv, K, V))], [randn(gen, (B, T, Hv, V), dtype), randn(gen, (N, Hv, K, V))]


NAMES = ("query", "key", "value", "log_decay", "beta", "initial_state")


def check(args, cot, lengths=None, scale=None, tail=0):
    """Forward without and with gradients, and all six gradients, against the oracle."""
    offsets = None
    if lengths is not None:
        offsets = torch.tensor(np.cumsum([0] + list(lengths)), dtype=torch.int32, device=DEV)
    sc = args[0].shape[-1] ** -0.5 if scale is None else scale
    out, state = gated_delta_rule(*args, scale=scale, offsets=offsets)
    leaves = [t.detach().requires_grad_() for t in args]
    out2, state2 = gated_delta_rule(*leaves, scale=scale, offsets=offsets)
    assert torch.equal(out, out2) and torch.equal(state, state2)
    grads = torch.autograd.grad([out2, state2], leaves, cot)
    x = [f64(t) for t in args]
    r_out, r_state = ref.gdr_fwd(*x, sc, lengths)
    errs = {"out": close("out", out, r_out), "state": close("state", state, r_state)}
    for name, got, want in zip(NAMES, grads, ref.gdr_bwd(*x, sc, *[f64(t) for t in cot], lengths)):
        errs[name] = close("gradient of " + name, got, want)
    print("  over the rounding, of the largest:", {n: f"{e:.1e}" for n, e in errs.items()}, flush=True)
    if tail:
        assert not out[:, -tail:].any() and not any(g[:, -tail:].any() for g in grads[:5])
    return out, state, grads


SIZES = [(1, 1, 1, 1, 1, 1), (2, 3, 1, 2, 5, 7), (1, 64, 1, 1, 32, 16), (1, 65, 2, 2, 64, 64), (2, 130, 1, 3, 128, 128), (1, 63, 2, 4, 33, 20),
         (1, 200, 1, 1, 127, 130), (1, 129, 1, 2, 100, 1), (3, 17, 2, 2, 16, 300), (1, 70, 1, 1, 8, 1024), (1, 192, 1, 2, 65, 48), (2, 33, 3, 3, 96, 24)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_rule(size, dtype):
    print(f"[rule {size} {dtype}]", flush=True)
    check(*inputs(*size, dtype, seed=sum(size)))


PACKED = [([5, 0, 1, 64, 65, 0, 130], 0), ([1], 3), ([0, 0], 5), ([63, 1, 1, 63, 128], 70), ([1] * 9, 0), ([200, 7], 1)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("lengths,tail", PACKED, ids=str)
def test_packed(lengths, tail, dtype):
    print(f"[packed {lengths} + {tail} {dtype}]", flush=True)
    args, cot = inputs(1, sum(lengths) + tail, 2, 4, 40, 24, dtype, N=len(lengths), seed=len(lengths))
    for t in args[:5] + cot[:1]:
        if tail:
            t[:, -tail:] = float("nan")                       # rows of no sequence are not read
    x = [t.clone() for t in args]
    out, state, grads = check_packed(args, cot, lengths, tail)
    assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(x, args))
    for n, length in enumerate(lengths):
        if not length:
            assert torch.equal(state[n], args[5][n]) and torch.equal(grads[5][n], cot[1][n])


def check_packed(args, cot, lengths, tail):
    if not tail:
        return check(args, cot, lengths)
    end = sum(lengths)
    cut = [t[:, :end] for t in args[:5]] + [args[5]]
    want = check([t.contiguous() for t in cut], [cot[0][:, :end].contiguous(), cot[1]], lengths) if end else None
    offsets = torch.tensor(np.cumsum([0] + list(lengths)), dtype=torch.int32, device=DEV)
    leaves = [t.detach().requires_grad_() for t in args]
    out, state = gated_delta_rule(*leaves, offsets=offsets)
    grads = torch.autograd.grad([out, state], leaves, cot)
    assert not out[:, end:].any() and not any(g[:, end:].any() for g in grads[:5])
    if want is not None:
        assert torch.equal(out[:, :end], want[0]) and torch.equal(state, want[1])
        assert all(torch.equal(a[:, :end], b) for a, b in zip(grads[:5], want[2][:5])) and torch.equal(grads[5], want[2][5])
    kept = torch.full_like(out, 5.0)
    capi.gdr_fwd(*args, offsets=offsets, out=kept)
    assert (kept[:, end:] == 5.0).all() and torch.equal(kept[:, :end], out[:, :end])
    return out, state, grads


PAIRED = [(2, 70, 4, 40, 64, 64, None), (1, 130, 3, 66, 32, 60, None), (3, 65, 2, 24, 128, 128, None), (1, 40, 1, 130, 100, 32, None),
          (1, 203, 2, 10, 40, 96, [64, 0, 1, 65, 70])]


@pytest.mark.parametrize("size", PAIRED, ids=str)
def test_many_heads_of_two_strips_to_a_block(size):
    """More strips of columns than compute units, an even number to a head: the passes take two at once.  Whole
    rows on 16 bytes and rows that are not, each count of key blocks, and a batch packed into one row."""
    print(f"[paired {size}]", flush=True)
    B, T, Hk, Hv, K, V, lengths = size
    check(*inputs(B, T, Hk, Hv, K, V, BF16, N=None if lengths is None else len(lengths), seed=Hv), lengths)


@pytest.mark.parametrize("dtype", [F32, F16], ids=str)
@pytest.mark.parametrize("size", [(3, 67, 4, 24, 64, 64), (1, 129, 2, 68, 27, 60), (2, 66, 2, 34, 128, 64), (5, 40, 7, 7, 48, 128)], ids=str)
def test_many_heads_of_two_strips_to_a_block_of_other_types(size, dtype):
    print(f"[paired {size} {dtype}]", flush=True)
    check(*inputs(*size, dtype, seed=size[3]))


def test_two_strips_to_a_block_equal_one_bit_for_bit():
    """The strips of a block share operands and nothing else: 33 sequences of 2 heads in one call, and one by one."""
    args, cot = inputs(33, 70, 1, 2, 64, 64, BF16, seed=5)
    leaves = [t.clone().requires_grad_() for t in args]
    whole = gated_delta_rule(*leaves)
    grads = torch.autograd.grad(whole, leaves, cot)
    for n in (0, 17, 32):
        one = [t[n:n + 1].clone().requires_grad_() for t in args]
        part = gated_delta_rule(*one)
        pg = torch.autograd.grad(part, one, [c[n:n + 1] for c in cot])
        for a, b in zip((*whole, *grads), (*part, *pg)):
            assert torch.equal(a[n:n + 1], b)


def test_packed_equals_a_batch_bit_for_bit():
    args, cot = inputs(3, 100, 1, 2, 64, 32, BF16, seed=11)
    leaves = [t.clone().requires_grad_() for t in args]
    a = gated_delta_rule(*leaves)
    ga = torch.autograd.grad(a, leaves, cot)
    offsets = torch.tensor([0, 100, 200, 300], dtype=torch.int32, device=DEV)
    flat = [t.reshape(1, -1, *t.shape[2:]).requires_grad_() for t in args[:5]] + [args[5].clone().requires_grad_()]
    b = gated_delta_rule(*flat, offsets=offsets)
    gb = torch.autograd.grad(b, flat, [cot[0].reshape(b[0].shape), cot[1]])
    for x, y in zip((*a, *ga), (*b, *gb)):
        assert torch.equal(x.reshape(-1), y.reshape(-1))


def test_offsets_out_of_range_stay_inside_the_tensors():
    args, cot = inputs(1, 150, 1, 2, 32, 16, BF16, N=3, seed=12)
    for bad in ([0, 150, 100, 50], [-5, 70, 90, 150], [0, 70, 90, 10 ** 9], [150, 100, 50, 0]):
        leaves = [t.clone().requires_grad_() for t in args]
        out, state = gated_delta_rule(*leaves, offsets=torch.tensor(bad, dtype=torch.int32, device=DEV))
        torch.autograd.grad([out, state], leaves, cot)
        torch.cuda.synchronize()
    # clamped offsets at both ends are the whole rows
    want = gated_delta_rule(*args, offsets=torch.tensor([0, 70, 90, 150], dtype=torch.int32, device=DEV))
    got = gated_delta_rule(*args, offsets=torch.tensor([-5, 70, 90, 10 ** 9], dtype=torch.int32, device=DEV))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_alike_keys_at_full_strength():
    # The triangular system's powers grow as binomials here: substitution has to hold.
    args, cot = inputs(1, 128, 1, 1, 32, 32, F32, seed=13)
    args[1][:] = args[1][:, :1]
    args[3][:] = 0
    args[4][:] = 1
    check(args, cot)


def test_decays_of_zero_and_far_below_and_betas_of_zero():
    args, cot = inputs(1, 150, 1, 2, 32, 32, F32, seed=14)
    g, b = args[3], args[4]
    g[0, [3, 64, 65, 100], 0] = -float("inf")
    g[0, [10, 70], 1] = -5000.0
    g[0, 20:40] = -80.0
    b[0, 5:30:3] = 0
    x = [f64(t) for t in args]
    with np.errstate(invalid="ignore"):
        check(args, cot)
    assert np.isfinite(x[0]).all()
    args[3] = torch.full_like(g, -float("inf"))
    check(args, cot)


def test_scale_strides_shared_and_absent_inputs():
    args, cot = inputs(2, 70, 2, 4, 64, 64, BF16, seed=15)
    for lead in (0, 8, 1):                                    # rows on 16 bytes, and on 2
        fused = torch.zeros(2, 70, lead + 512 + 8, device=DEV, dtype=BF16)
        parts = [fused[..., lead:lead + 128].unflatten(-1, (2, 64)), fused[..., lead + 128:lead + 256].unflatten(-1, (2, 64)),
                 fused[..., lead + 256:lead + 512].unflatten(-1, (4, 64))]
        for p, t in zip(parts, args):
            p.copy_(t)
        check(parts + args[3:], cot, scale=0.25)
    heads_first = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in args[:5]]
    check(heads_first + args[5:], cot)
    a = gated_delta_rule(*args[:5])
    b = gated_delta_rule(*args[:5], torch.zeros_like(args[5]))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # one key head for both (a broadcast input): its gradient is the sum
    leaf = args[1][:, :, :1].clone().requires_grad_()
    out, state = gated_delta_rule(args[0], leaf.expand(2, 70, 2, 64), *args[2:])
    got, = torch.autograd.grad([out, state], [leaf], cot)
    x = [f64(t) for t in (args[0], leaf.expand(2, 70, 2, 64), *args[2:])]
    want = ref.gdr_bwd(*x, 64 ** -0.5, *[f64(t) for t in cot])[1].sum(2, keepdims=True)
    top = np.abs(want).max()                                  # two heads' gradients rounded, then their sum
    assert np.abs(f64(got) - want).max() <= 3 * 2.0 ** -8 * top + 1e-5 * top


def test_gradients_of_some_inputs_and_of_one_output():
    args, cot = inputs(1, 100, 1, 2, 48, 40, F32, seed=16)
    x = [f64(t) for t in args]
    zero = [np.zeros(c.shape) for c in cot]
    for only in range(2):
        want = ref.gdr_bwd(*x, 48 ** -0.5, *[f64(c) if i == only else z for i, (c, z) in enumerate(zip(cot, zero))])
        for i in range(6):
            leaves = [t.clone().requires_grad_(j == i) for j, t in enumerate(args)]
            got, = torch.autograd.grad(gated_delta_rule(*leaves)[only], [leaves[i]], cot[only])
            close(f"output {only}, gradient of {NAMES[i]}", got, want[i])


def test_gradients_against_differences():
    args, cot = inputs(1, 90, 1, 2, 32, 16, F32, seed=17)
    gen = torch.Generator(device=DEV).manual_seed(1)
    leaves = [t.clone().requires_grad_() for t in args]
    loss = lambda *a: sum((x.double() * c).sum() for x, c in zip(gated_delta_rule(*a), cot))
    grads = torch.autograd.grad(loss(*leaves), leaves)
    for i, g in enumerate(grads):
        d = randn(gen, args[i].shape)
        if i == 3:
            d = d * args[i].abs().clamp(max=0.1)
        h = 1e-2
        up, down = (loss(*[t + s * h * d if j == i else t for j, t in enumerate(args)]) for s in (1, -1))
        want, got = float((up - down) / (2 * h)), float((g.double() * d.double()).sum())
        # h^2 of the third derivative, and float32 outputs' 2^-24 over h
        assert abs(got - want) <= 5e-3 * (abs(want) + float((g * d).norm())), (NAMES[i], got, want)


def test_with_nothing_to_do():
    args, cot = inputs(2, 5, 1, 2, 16, 8, BF16, seed=18)
    cut = [t[:, :0].contiguous().requires_grad_() for t in args[:5]] + [args[5].clone().requires_grad_()]
    out, state = gated_delta_rule(*cut)
    assert out.shape == (2, 0, 2, 8) and torch.equal(state, args[5])
    grads = torch.autograd.grad([out, state], cut, [out.detach(), cot[1]])
    assert torch.equal(grads[5], cot[1]) and grads[0].shape == (2, 0, 1, 16)
    out, state = gated_delta_rule(*[t[:0] for t in args])
    assert out.shape == (0, 5, 2, 8) and state.shape == (0, 2, 16, 8)
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, state = gated_delta_rule(*[t[:1] for t in args[:5]], args[5][:0], offsets=none)
    assert not out.any() and state.shape == (0, 2, 16, 8)


def test_long_sequence_in_pieces_and_against_the_step():
    args, _ = inputs(1, 1500, 1, 2, 128, 128, BF16, seed=19)
    out, state = gated_delta_rule(*args)
    cut = 777
    o1, s1 = gated_delta_rule(*[t[:, :cut] for t in args[:5]], args[5])
    o2, s2 = gated_delta_rule(*[t[:, cut:] for t in args[:5]], s1)
    half = 2.0 ** -8
    both, top = torch.cat([o1, o2], 1).double(), out.double().abs().max()
    # the same sums, chunked elsewhere: each side rounds once, at its own place
    assert ((both - out.double()).abs() <= 2 * half * out.double().abs() + 2e-5 * top).all()
    assert (s2 - state).abs().max() <= 2e-5 * state.abs().max()
    pool = s1.clone()
    steps = [gated_delta_step(*[t[:, i:i + 5].contiguous() for t in args[:5]], pool) for i in range(cut, 1500, 5) if i + 5 <= 1500]
    n = 5 * len(steps)
    got = torch.cat(steps, 1).double()
    assert ((got - o2[:, :n].double()).abs() <= 2 * half * o2[:, :n].double().abs() + 2e-5 * top).all()


def test_a_layer_from_norm_to_prompt_to_tokens():
    """The operators as a layer runs them: unit heads from one fused projection, a packed prompt, then tokens one by one on
    the pooled states, against the oracles' chain; and its gradients through both."""
    gen = torch.Generator(device=DEV).manual_seed(20)
    Hk, Hv, K, V, lengths = 2, 4, 64, 48, [70, 3, 129]
    T = sum(lengths)
    rows = randn(gen, (1, T, 2 * Hk * K))
    q, k = rows[..., :Hk * K].unflatten(-1, (Hk, K)), rows[..., Hk * K:].unflatten(-1, (Hk, K))
    v, g, b = randn(gen, (1, T, Hv, V)), -torch.rand(1, T, Hv, generator=gen, device=DEV), torch.rand(1, T, Hv, generator=gen, device=DEV)
    angle = randn(gen, (200, 16)) * 3
    pos = torch.cat([torch.arange(n) for n in lengths])[None].to(DEV)
    offsets = torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32, device=DEV)
    leaves = [t.detach().requires_grad_() for t in (q, k, v, g, b)]
    qn, kn = qk_norm_rotate(leaves[0], leaves[1], None, None, angle.cos(), angle.sin(), pos, kind="l2")
    out, state = gated_delta_rule(qn, kn, *leaves[2:], offsets=offsets)
    cot = [randn(gen, out.shape), randn(gen, state.shape)]
    grads = torch.autograd.grad([out, state], leaves, cot)
    how = (None, f64(angle.cos()), f64(angle.sin()), pos.cpu().numpy(), "l2", 1e-6, False)
    rq, rk = ref.qkn_fwd(f64(q), *how), ref.qkn_fwd(f64(k), *how)
    s0 = np.zeros((3, Hv, K, V))
    rest = [f64(t) for t in (v, g, b)]
    r_out, r_state = ref.gdr_fwd(rq, rk, *rest, s0, K ** -0.5, lengths)
    close("out", out, r_out)
    close("state", state, r_state)
    dq, dk, dv, dg, db, _ = ref.gdr_bwd(rq, rk, *rest, s0, K ** -0.5, *[f64(c) for c in cot], lengths)
    want = [ref.qkn_bwd(f64(q), *how, dq)[0], ref.qkn_bwd(f64(k), *how, dk)[0], dv, dg, db]
    for name, x, y in zip(NAMES, grads, want):
        close("gradient of " + name, x, y)
    pool = torch.zeros(5, Hv, K, V, device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    pool[slots.long()] = state.detach()
    for step in range(3):
        x = [randn(gen, (3, 1, h, w)) for h, w in ((Hk, K), (Hk, K), (Hv, V))]
        gb = [-torch.rand(3, 1, Hv, generator=gen, device=DEV), torch.rand(3, 1, Hv, generator=gen, device=DEV)]
        at = torch.tensor([[n + step] for n in lengths], device=DEV)
        qn, kn = qk_norm_rotate(x[0], x[1], None, None, angle.cos(), angle.sin(), at, kind="l2")
        got = gated_delta_step(qn, kn, x[2], *gb, pool, slots=slots)
        how = (None, f64(angle.cos()), f64(angle.sin()), at.cpu().numpy(), "l2", 1e-6, False)
        r, r_state = ref.gdr_fwd(ref.qkn_fwd(f64(x[0]), *how), ref.qkn_fwd(f64(x[1]), *how), f64(x[2]), *map(f64, gb), r_state, K ** -0.5)
        close(f"token {step}", got, r)
    close("pool", pool[slots.long()], r_state)


def test_streams_graphs_and_bits():
    args, cot = inputs(2, 200, 2, 4, 128, 64, BF16, seed=21)
    call = lambda **kw: (lambda o: o[:2] + capi.gdr_bwd(*args[:5], o[2], *cot, **kw))(capi.gdr_fwd(*args, want_saved=True, **kw))
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, here = call(stream=side), call()                     # two calls at once, workspaces of their own
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(here, want))
    graphs, outs = [], []
    for _ in range(2):                                        # two captures of one pool, replayed in turn
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], pool=graphs[0].pool() if len(graphs) > 1 else None):
            outs.append(call())
    for _ in range(3):
        for graph, out in zip(graphs, outs):
            for t in out:
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(call(), want))


def test_a_training_step_of_a_layer_captured_and_replayed():
    args, cot = inputs(2, 90, 2, 4, 64, 32, BF16, seed=31)
    leaves = [t.clone().requires_grad_() for t in args]

    def step():
        q, k = qk_norm_rotate(*leaves[:2], kind="l2")
        out, state = gated_delta_rule(q, k, *leaves[2:])
        return [t.detach() for t in (out, state, *torch.autograd.grad([out, state], leaves, cot))]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))


def test_a_scale_or_eps_in_a_tensor_is_read_at_each_call():
    args, cot = inputs(1, 20, 1, 2, 16, 16, F32, seed=9)
    scale, eps = torch.tensor(0.5), torch.tensor(0.25)
    leaves = [t.clone().requires_grad_() for t in args]
    out = gated_delta_rule(*leaves, scale=scale)
    first = gated_delta_step(*args[:5], args[5].clone(), scale=scale)
    normed = qk_norm_rotate(*leaves[:2], eps=eps)
    scale.fill_(2.0)
    eps.fill_(4.0)
    want = gated_delta_rule(*leaves, scale=0.5)
    for a, b in zip(torch.autograd.grad(out, leaves, cot), torch.autograd.grad(want, leaves, cot)):
        assert torch.equal(a, b)                     # the backward pass keeps the forward's
    want = torch.autograd.grad(qk_norm_rotate(*leaves[:2], eps=0.25), leaves[:2], args[:2])
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(normed, leaves[:2], args[:2]), want))
    assert torch.equal(gated_delta_rule(*args, scale=scale)[0], gated_delta_rule(*args, scale=2.0)[0])
    second = gated_delta_step(*args[:5], args[5].clone(), scale=scale)
    assert torch.equal(second, gated_delta_step(*args[:5], args[5].clone(), scale=2.0)) and not torch.equal(first, second)
    assert torch.equal(qk_norm_rotate(*args[:2], eps=eps)[0], qk_norm_rotate(*args[:2], eps=4.0)[0])


def test_refusals():
    args, cot = inputs(2, 5, 2, 4, 16, 8, BF16, seed=22)
    q, k, v, g, b, s = args
    offsets = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    call = lambda **kw: gated_delta_rule(**{**dict(query=q, key=k, value=v, log_decay=g, beta=b, initial_state=s), **kw})
    for kw in (dict(key=k[:1]), dict(key=k[..., :8]), dict(value=v[:, :, :3]), dict(value=v[:, :4]), dict(log_decay=g.to(BF16)),
               dict(beta=b.double()), dict(beta=b[:, :4]), dict(initial_state=s[:1]), dict(initial_state=s.to(BF16)), dict(offsets=offsets),
               dict(query=q[0]), dict(query=q.double(), key=k.double(), value=v.double()), dict(key=k.to(F16)), dict(initial_state=s.cpu()),
               dict(query=torch.zeros(2, 5, 2, 200, device=DEV, dtype=BF16), key=torch.zeros(2, 5, 2, 200, device=DEV, dtype=BF16)),
               dict(value=torch.zeros(2, 5, 4, 1025, device=DEV, dtype=BF16))):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    one = [t[:1] for t in args]
    for bad in (offsets.long(), offsets.cpu(), offsets[None], offsets[:0]):
        with pytest.raises(ValueError):
            gated_delta_rule(*one, offsets=bad)
    saved = capi.gdr_fwd(*args, want_saved=True)[2]
    with pytest.raises(ValueError):
        capi.gdr_bwd(*args[:5], saved[:-1], *cot)
    with pytest.raises(RuntimeError):                         # the gradient's own gradient
        leaf = q.clone().requires_grad_()
        d, = torch.autograd.grad(call(query=leaf)[0].float().sum(), [leaf], create_graph=True)
        d.sum().backward()
    torch.cuda.synchronize()
