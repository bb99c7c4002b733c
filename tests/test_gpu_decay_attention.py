"""Parity of linear attention with decays, its VJP and its decoding step with
the float64 oracle (needs an MI355X).

Tolerance of an output, element by element: half a step of its type relative
to the value, for the one rounding, plus 1e-5 of the largest value for the
rest.  Of the rest: float32 sums of at most K + V + 64 products a chunk, which
the decays forget, are off by sqrt(6 (K + V + 64)) 2^-23 <= 6e-6 of it in the
probabilistic rounding model at the largest sizes here, and where the output
has 16 bits its computed operands keep two bfloat16 parts, off by 2^-18 each, a
thousandth of the output's own step."""
import numpy as np
import pytest
import torch

from oracle import layer_ops as ref
from oracle import lm_ops
from quaternion_cumprod_autodiff_amd import capi, decay_attention, decay_attention_step, layer_norm, qk_norm_rotate

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAMES = ("query", "key", "value", "log_decay", "initial_state")


def f64(t):
    return t.detach().double().cpu().numpy()


def close(label, got, want, top=None):
    rel, low = torch.finfo(got.dtype).eps / 2, torch.finfo(got.dtype).smallest_normal      # below it steps stay those of it
    got, want = f64(got), np.asarray(want)
    assert got.shape == want.shape, (label, got.shape, want.shape)
    if not want.size:
        return 0.0
    top = float(np.abs(want).max()) if top is None else top
    off = float((np.abs(got - want) - rel * np.maximum(np.abs(want), low)).max())
    assert np.isfinite(got).all() and off <= 1e-5 * top + 1e-30, f"{label}: {off:.3e} over the rounding, largest {top:.3e}"
    return max(off, 0.0) / max(top, 1e-30)


def randn(gen, shape, dtype=F32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=F32).to(dtype)


def inputs(B, T, Hk, Hv, K, V, dtype, N=None, seed=0, head=False):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    N = B if N is None else N
    q, k, v = randn(gen, (B, T, Hk, K), dtype), (randn(gen, (B, T, Hk, K)) * K ** -0.5).to(dtype), randn(gen, (B, T, Hv, V), dtype)
    rate = torch.logspace(-2, 0.5, Hv, device=DEV)
    g = -rate if head else -torch.rand(B, T, Hv, generator=gen, device=DEV) * rate
    return [q, k, v, g, randn(gen, (N, Hv, K, V))], [randn(gen, (B, T, Hv, V), dtype), randn(gen, (N, Hv, K, V))]


def offsets_of(lengths):
    return torch.tensor(np.cumsum([0] + list(lengths)), dtype=torch.int32, device=DEV)


def check(args, cot, lengths=None, scale=None):
    """Forward without and with gradients, and all five gradients, against the oracle."""
    offsets = None if lengths is None else offsets_of(lengths)
    sc = args[0].shape[-1] ** -0.5 if scale is None else scale
    out, state = decay_attention(*args, scale=scale, offsets=offsets)
    leaves = [t.detach().requires_grad_() for t in args]
    out2, state2 = decay_attention(*leaves, scale=scale, offsets=offsets)
    assert torch.equal(out, out2) and torch.equal(state, state2)
    grads = torch.autograd.grad([out2, state2], leaves, cot)
    x = [f64(t) for t in args]
    r_out, r_state = ref.dca_fwd(*x, sc, lengths)
    errs = {"out": close("out", out, r_out), "state": close("state", state, r_state)}
    for name, got, want in zip(NAMES, grads, ref.dca_bwd(*x, sc, *[f64(t) for t in cot], lengths)):
        errs[name] = close("gradient of " + name, got, want)
    print("  over the rounding, of the largest:", {n: f"{e:.1e}" for n, e in errs.items()}, flush=True)
    return out, state, grads


SIZES = [(1, 1, 1, 1, 1, 1), (2, 3, 1, 2, 5, 7), (1, 64, 1, 1, 32, 16), (1, 65, 2, 2, 64, 64), (2, 130, 1, 3, 128, 128), (1, 63, 2, 4, 33, 20),
         (1, 200, 1, 1, 127, 130), (1, 129, 1, 2, 100, 1), (3, 17, 2, 2, 16, 300), (1, 70, 1, 1, 8, 1024), (1, 192, 1, 2, 65, 48), (2, 33, 3, 3, 96, 24),
         (1, 31, 1, 1, 128, 72), (1, 32, 1, 2, 24, 65)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_attention(size, dtype):
    print(f"[attention {size} {dtype}]", flush=True)
    check(*inputs(*size, dtype, seed=sum(size), head=size[1] % 2 == 0))


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("size", [(1, 1500, 1, 2, 64, 32), (2, 1025, 2, 2, 40, 100), (1, 833, 1, 2, 128, 128)], ids=str)
def test_sequences_in_segments(size, head, dtype):
    """Long enough that few heads are cut into several segments, the last of them ragged."""
    print(f"[segments {size} {head} {dtype}]", flush=True)
    check(*inputs(*size, dtype, seed=size[1], head=head))


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("size", [(5, 300, 16, 32, 32, 40), (2, 333, 8, 128, 64, 128), (4, 450, 4, 24, 100, 130), (9, 290, 30, 30, 24, 50)], ids=str)
def test_many_heads_and_sequences(size, dtype):
    """Enough of them that the forward pass or the backward states' pass goes without segments, or both do."""
    print(f"[many {size} {dtype}]", flush=True)
    check(*inputs(*size, dtype, seed=size[1]))


PACKED = [([5, 0, 1, 64, 65, 0, 130], 0), ([1], 3), ([0, 0], 5), ([63, 1, 1, 63, 128], 70), ([1] * 9, 0), ([200, 7], 1), ([900, 0, 3, 640, 257], 30)]


@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("lengths,tail", PACKED, ids=str)
def test_packed(lengths, tail, dtype, head):
    """Packed sequences; rows behind the last are neither read (they hold NaN) nor written."""
    print(f"[packed {lengths} + {tail} {dtype} {head}]", flush=True)
    end = sum(lengths)
    args, cot = inputs(1, end + tail, 2, 4, 40, 24, dtype, N=len(lengths), seed=len(lengths), head=head)
    if tail:
        for t in args[:3 if head else 4] + cot[:1]:
            t[:, end:] = float("nan")
    cut = [t[:, :end].contiguous() for t in args[:3]] + [args[3] if head else args[3][:, :end].contiguous(), args[4]]
    want = check(cut, [cot[0][:, :end].contiguous(), cot[1]], lengths) if end else None
    offsets = offsets_of(lengths)
    leaves = [t.detach().requires_grad_() for t in args]
    out, state = decay_attention(*leaves, offsets=offsets)
    grads = torch.autograd.grad([out, state], leaves, cot)
    rows = grads[:3] if head else grads[:4]
    assert not out[:, end:].any() and not any(g[:, end:].any() for g in rows)
    if want is not None:
        # Where the rows behind the end change the segments, the sums are joined elsewhere; else bits are equal.
        half = torch.finfo(dtype).eps
        assert ((out[:, :end].double() - want[0].double()).abs() <= half * want[0].double().abs() + 2e-5 * want[0].abs().max()).all()
        assert ((state - want[1]).abs() <= 2e-5 * want[1].abs().max()).all()
        for a, b in zip(grads[:3], want[2][:3]):
            assert ((a[:, :end].double() - b.double()).abs() <= half * b.double().abs() + 2e-5 * b.abs().max()).all()
    else:
        assert not (grads[3].any() if head else grads[3].any())
    kept = torch.full_like(out, 5.0)
    capi.dca_fwd(*args, offsets=offsets, out=kept)
    assert (kept[:, end:] == 5.0).all() and torch.equal(kept[:, :end], out[:, :end])
    for n, length in enumerate(lengths):
        if not length:
            assert torch.equal(state[n], args[4][n]) and torch.equal(grads[4][n], cot[1][n])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("lengths", [[128, 256, 0, 129, 127, 1, 640, 0, 0, 383], [7] * 140 + [1000] + [5] * 40, [1] + [255] * 4 + [0] * 3 + [257, 513, 2],
                                     [0, 700, 0] + [3] * 200], ids=lambda x: f"{len(x)} sequences")
def test_packed_sequences_of_unlike_length(lengths, dtype):
    """Ends at, before and behind the places where segments may meet; a long sequence among many short ones."""
    print(f"[packed {len(lengths)} {dtype}]", flush=True)
    args, cot = inputs(1, sum(lengths), 2, 4, 40, 24, dtype, N=len(lengths), seed=len(lengths))
    check(args, cot, lengths)


def test_packed_equals_a_batch_bit_for_bit():
    args, cot = inputs(3, 128, 1, 2, 64, 32, BF16, seed=11)
    leaves = [t.clone().requires_grad_() for t in args]
    a = decay_attention(*leaves)
    ga = torch.autograd.grad(a, leaves, cot)
    flat = [t.reshape(1, -1, *t.shape[2:]).requires_grad_() for t in args[:4]] + [args[4].clone().requires_grad_()]
    b = decay_attention(*flat, offsets=offsets_of([128] * 3))
    gb = torch.autograd.grad(b, flat, [cot[0].reshape(b[0].shape), cot[1]])
    for x, y in zip((*a, *ga), (*b, *gb)):
        assert torch.equal(x.reshape(-1), y.reshape(-1))


@pytest.mark.parametrize("T", [150, 1500])
def test_offsets_out_of_range_stay_inside_the_tensors(T):
    args, cot = inputs(1, T, 1, 2, 32, 16, BF16, N=3, seed=12)
    for bad in ([0, T, 100, 50], [-5, 70, 90, T], [0, 70, 90, 10 ** 9], [T, 100, 50, 0], [T, 0, T, 0], [-2 ** 31, 2 ** 31 - 1, -1, 2 ** 31 - 1]):
        leaves = [t.clone().requires_grad_() for t in args]
        out, state = decay_attention(*leaves, offsets=torch.tensor(bad, dtype=torch.int32, device=DEV))
        torch.autograd.grad([out, state], leaves, cot)
        torch.cuda.synchronize()
    want = decay_attention(*args, offsets=torch.tensor([0, 70, 90, T], dtype=torch.int32, device=DEV))
    got = decay_attention(*args, offsets=torch.tensor([-5, 70, 90, 10 ** 9], dtype=torch.int32, device=DEV))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_decays_of_zero_and_far_below():
    args, cot = inputs(1, 150, 1, 2, 32, 32, F32, seed=14)
    g = args[3]
    g[0, [3, 64, 65, 100], 0] = -float("inf")
    g[0, [10, 70], 1] = -5000.0
    g[0, 20:40] = -80.0
    grads = check(args, cot)[2]
    assert not grads[3][0, [3, 64, 65, 100], 0].any()         # a decay of exactly nothing has a gradient of exactly nothing
    args[3] = torch.full_like(g, -float("inf"))
    check(args, cot)
    args[3] = torch.zeros_like(g)
    check(args, cot)
    for value in (0.0, -40.0, -float("inf")):
        args[3] = torch.tensor([value, -0.1], device=DEV)
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
    heads_first = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in args[:4]]
    check(heads_first + args[4:], cot, scale=-1.5)
    a = decay_attention(*args[:4])
    b = decay_attention(*args[:4], torch.zeros_like(args[4]))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert not decay_attention(*args, scale=0.0)[0].any()
    # one key head for both (a broadcast input): its gradient is the sum
    leaf = args[1][:, :, :1].clone().requires_grad_()
    out, state = decay_attention(args[0], leaf.expand(2, 70, 2, 64), *args[2:])
    got, = torch.autograd.grad([out, state], [leaf], cot)
    x = [f64(t) for t in (args[0], leaf.expand(2, 70, 2, 64), *args[2:])]
    want = ref.dca_bwd(*x, 64 ** -0.5, *[f64(t) for t in cot])[1].sum(2, keepdims=True)
    top = np.abs(want).max()                                  # two heads' gradients rounded, then their sum
    assert np.abs(f64(got) - want).max() <= 3 * 2.0 ** -8 * top + 1e-5 * top


def test_rows_far_apart():
    """Tokens and heads 16 MiB apart: offsets pass 32 bits, within a chunk too."""
    args, cot = inputs(1, 70, 2, 2, 32, 40, BF16, seed=23)
    room = torch.zeros(150 * 2 ** 23, device=DEV, dtype=BF16)
    far = []
    for i, t in enumerate(args[:3]):
        view = room[i * 2 ** 10:].as_strided(t.shape, (0, 2 ** 24, 2 ** 23, 1))
        view.copy_(t)
        far.append(view)
    want = decay_attention(*args)
    got = decay_attention(*far, *args[3:])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    leaves, there = [t.clone().requires_grad_() for t in args], [t.detach().requires_grad_() for t in far + args[3:]]
    a = torch.autograd.grad(decay_attention(*leaves), leaves, cot)
    b = torch.autograd.grad(decay_attention(*there), there, cot)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    step = [t[:, :1] for t in far] + [args[3][:, :1].contiguous()]
    near = [t[:, :1].contiguous() for t in args[:4]]
    assert torch.equal(decay_attention_step(*step, args[4].clone()), decay_attention_step(*near, args[4].clone()))


@pytest.mark.parametrize("head", [False, True])
def test_gradients_of_some_inputs_and_of_one_output(head):
    args, cot = inputs(1, 100, 1, 2, 48, 40, F32, seed=16, head=head)
    x = [f64(t) for t in args]
    zero = [np.zeros(c.shape) for c in cot]
    for only in range(2):
        want = ref.dca_bwd(*x, 48 ** -0.5, *[f64(c) if i == only else z for i, (c, z) in enumerate(zip(cot, zero))])
        for i in range(5):
            leaves = [t.clone().requires_grad_(j == i) for j, t in enumerate(args)]
            out = decay_attention(*leaves)[only]
            if not out.requires_grad:
                continue
            got = torch.autograd.grad(out, [leaves[i]], cot[only], allow_unused=True)[0]
            close(f"output {only}, gradient of {NAMES[i]}", got, want[i])


def test_gradients_against_differences():
    args, cot = inputs(1, 90, 1, 2, 32, 16, F32, seed=17)
    gen = torch.Generator(device=DEV).manual_seed(1)
    leaves = [t.clone().requires_grad_() for t in args]
    loss = lambda *a: sum((x.double() * c).sum() for x, c in zip(decay_attention(*a), cot))
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


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("g0", [-3.0, -8.0, -20.0, -40.0])
def test_gradients_of_uniform_strong_decays(g0, dtype):
    """The gradient of log_decay scales with exp(log_decay): nothing that does not carry the decay may be left in it."""
    args, cot = inputs(1, 150, 1, 2, 64, 48, dtype, seed=int(-g0))
    args[3].fill_(g0)
    check(args, cot)


@pytest.mark.parametrize("K", [24, 128])
def test_gradients_of_strong_decays_among_weak_ones(K):
    """At the tokens whose decay is strong the gradient is far below the others': it is held to its own size."""
    args, cot = inputs(2, 200, 2, 2, K, 32, F32, seed=K)
    strong = [0, 5, 31, 32, 63, 64, 90, 127, 128, 191, 192, 199]
    args[3] = args[3].clamp(min=-0.1)
    args[3][:, strong] = -25.0
    args[3][:, [30, 150]] = -float("inf")
    got = check(args, cot)[2][3]
    want = ref.dca_bwd(*[f64(t) for t in args], K ** -0.5, *[f64(c) for c in cot])[3]
    for t in strong:
        close(f"token {t}", got[:, t], want[:, t])
    assert not got[:, [30, 150]].any()


@pytest.mark.parametrize("head", [False, True])
def test_with_nothing_to_do(head):
    args, cot = inputs(2, 5, 1, 2, 16, 8, BF16, seed=18, head=head)
    cut = [t[:, :0].contiguous().requires_grad_() for t in args[:3]] + [(args[3] if head else args[3][:, :0].contiguous()).clone().requires_grad_(),
                                                                       args[4].clone().requires_grad_()]
    out, state = decay_attention(*cut)
    assert out.shape == (2, 0, 2, 8) and torch.equal(state, args[4])
    grads = torch.autograd.grad([out, state], cut, [out.detach(), cot[1]])
    assert torch.equal(grads[4], cot[1]) and grads[0].shape == (2, 0, 1, 16)
    if head:
        want = ref.dca_bwd(*[f64(t) for t in cut], 0.25, np.zeros((2, 0, 2, 8)), f64(cot[1]))[3]
        assert not grads[3].any() and not want.any()
    empty = [t[:0] for t in args[:3]] + [args[3] if head else args[3][:0], args[4][:0]]
    out, state = decay_attention(*empty)
    assert out.shape == (0, 5, 2, 8) and state.shape == (0, 2, 16, 8)
    if head:
        leaf = args[3].clone().requires_grad_()
        out = decay_attention(*empty[:3], leaf, empty[4])
        assert not torch.autograd.grad(out, [leaf], [t.detach() for t in out])[0].any()
    long, _ = inputs(1, 300, 1, 2, 16, 8, BF16, seed=24, head=head)          # no sequence among many rows
    leaves = [t.clone().requires_grad_() for t in long[:4]] + [long[4][:0].clone().requires_grad_()]
    out, state = decay_attention(*leaves, offsets=torch.zeros(1, dtype=torch.int32, device=DEV))
    grads = torch.autograd.grad([out, state], leaves, [torch.ones_like(out), torch.ones_like(state)])
    assert not out.any() and state.shape == (0, 2, 16, 8) and not any(g.any() for g in grads)
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, state = decay_attention(*[t[:1] for t in args[:3]], args[3] if head else args[3][:1], args[4][:0], offsets=none)
    assert not out.any() and state.shape == (0, 2, 16, 8)


def test_long_sequence_in_pieces_and_against_the_step():
    args, _ = inputs(1, 1500, 1, 2, 128, 128, BF16, seed=19)
    out, state = decay_attention(*args)
    cut = 777
    o1, s1 = decay_attention(*[t[:, :cut] for t in args[:4]], args[4])
    o2, s2 = decay_attention(*[t[:, cut:] for t in args[:4]], s1)
    half = 2.0 ** -8
    both, top = torch.cat([o1, o2], 1).double(), out.double().abs().max()
    # the same sums, chunked elsewhere: each side rounds once, at its own place
    assert ((both - out.double()).abs() <= 2 * half * out.double().abs() + 2e-5 * top).all()
    assert (s2 - state).abs().max() <= 2e-5 * state.abs().max()
    pool = s1.clone()
    steps = [decay_attention_step(*[t[:, i:i + 5].contiguous() for t in args[:4]], pool) for i in range(cut, 1500, 5) if i + 5 <= 1500]
    n = 5 * len(steps)
    got = torch.cat(steps, 1).double()
    assert ((got - o2[:, :n].double()).abs() <= 2 * half * o2[:, :n].double().abs() + 2e-5 * top).all()


# ------------------------------------------------------------------ the decoding step

def step_inputs(B, T, Hk, Hv, K, V, pool, dtype, seed=0, head=False):
    args, _ = inputs(B, T, Hk, Hv, K, V, dtype, seed=seed, head=head)
    gen = torch.Generator(device=DEV).manual_seed(seed + 1)
    return args[:4] + [randn(gen, (pool, Hv, K, V))], torch.randperm(pool, generator=gen, device=DEV)[:B].to(torch.int32)


def check_step(args, slots, scale=None):
    state = args[4]
    before = state.clone()
    rows = torch.arange(args[0].shape[0], device=DEV) if slots is None else slots.long()
    out = decay_attention_step(*args, slots=slots, scale=scale)
    sc = args[0].shape[-1] ** -0.5 if scale is None else scale
    want, want_state = ref.dca_fwd(*[f64(t) for t in args[:4]], f64(before[rows]), sc)
    close("out", out, want)
    close("state", state[rows], want_state)
    rest = torch.ones(len(state), dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert torch.equal(state[rest], before[rest])


@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 1, 1, 1), (3, 1, 2, 4, 128, 128, 5), (2, 4, 1, 3, 72, 100, 7), (5, 7, 2, 2, 33, 17, 5), (4, 1, 1, 1, 64, 200, 4),
                                  (1, 2, 4, 8, 24, 40, 3), (2, 1, 1, 2, 8, 1024, 2)], ids=str)
def test_step(size, dtype, head):
    print(f"[step {size} {dtype} {head}]", flush=True)
    args, slots = step_inputs(*size, dtype, seed=sum(size), head=head)
    check_step(args, slots)


def test_step_without_slots_with_strides_padding_and_doubles():
    args, _ = step_inputs(4, 2, 2, 4, 64, 32, 6, BF16, seed=3)
    check_step(args, None, scale=2.0)
    whole = torch.zeros(6, 2, 4, 64, 32, device=DEV)
    whole[:, 1] = args[4]
    check_step(args[:4] + [whole[:, 1]], torch.tensor([5, 0, 3, 1], dtype=torch.int32, device=DEV))
    assert not whole[:, 0].any()
    fused = torch.cat([t.flatten(2) for t in args[:3]], -1)
    parts = [fused[..., :128].unflatten(-1, (2, 64)), fused[..., 128:256].unflatten(-1, (2, 64)), fused[..., 256:].unflatten(-1, (4, 32))]
    check_step(parts + args[3:], None)
    slots = torch.tensor([2, -1, 2, 6], dtype=torch.int32, device=DEV)      # padding, a slot named before, one outside
    before = args[4].clone()
    out = decay_attention_step(*args, slots=slots)
    want, want_state = ref.dca_fwd(*[f64(t[:1]) for t in args[:4]], f64(before[2:3]), 64 ** -0.5)
    close("out", out[:1], want)
    close("state", args[4][2:3], want_state)
    assert not out[1:].any() and torch.equal(args[4][[0, 1, 3, 4, 5]], before[[0, 1, 3, 4, 5]])
    version = args[4]._version
    decay_attention_step(*args)
    assert args[4]._version > version


def test_step_on_states_beyond_2_to_the_31_elements():
    """The last slots of a pool of 9.7 GB."""
    args, _ = step_inputs(2, 1, 1, 32, 128, 128, 1, BF16, seed=5)
    pool = torch.zeros(4600, 32, 128, 128, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(7)
    pool[[4599, 4097]] = randn(gen, (2, 32, 128, 128))
    slots = torch.tensor([4599, 4097], dtype=torch.int32, device=DEV)
    before = pool[slots.long()].clone()
    out = decay_attention_step(*args[:4], pool, slots=slots)
    want, want_state = ref.dca_fwd(*[f64(t) for t in args[:4]], f64(before), 128 ** -0.5)
    close("out", out, want)
    close("state", pool[slots.long()], want_state)
    assert not pool[:4097].any() and not pool[4098:4599].any()


# ------------------------------------------------------------------ inputs that are not finite

@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("dtype,K,V,Hk,Hv,T", [(F32, 40, 24, 1, 2, 150), (BF16, 128, 32, 2, 4, 150), (F16, 64, 100, 1, 3, 150), (BF16, 20, 64, 1, 40, 150),
                                              (BF16, 32, 128, 1, 1, 900)], ids=str)
def test_what_is_not_finite_reaches_no_earlier_token(dtype, K, V, Hk, Hv, T, saved):
    """out of token t depends on tokens up to t: what comes before a NaN or an infinity keeps its bits, and from there on
    its head (a value: its column; a query: its token) is not finite, the final state neither."""
    clean = inputs(1, T, Hk, Hv, K, V, dtype, seed=K)[0]
    run = lambda a: capi.dca_fwd(*a, want_saved=saved)[:2]
    want, want_state = run(clean)
    group = Hv // Hk
    for t, bad in ((0, float("nan")), (5, float("inf")), (17, float("nan")), (31, -float("inf")), (63, float("nan")), (64, float("inf")), (T - 1, float("nan"))):
        for which in range(4):
            args = [x.clone() for x in clean]
            h, c = (t + which) % args[which].shape[2], (7 * t + which) % args[which].shape[-1]
            if which < 3:
                args[which][0, t, h, c] = bad
            else:
                args[which][0, t, h] = float("nan") if bad < 0 else bad      # a decay of -inf is an input like others
            out, state = run(args)
            hit = torch.zeros(T, Hv, V, dtype=torch.bool, device=DEV)
            heads = slice(h * group, (h + 1) * group) if which < 2 else h
            if which == 0:
                hit[t, heads] = True
            elif which == 2:
                hit[t:, h, c] = True
            else:
                hit[t:, heads] = True
            assert torch.equal(out[0][~hit], want[0][~hit]), (t, which)
            assert not out[0][hit].isfinite().any(), (t, which)
            gone = torch.zeros(Hv, K, V, dtype=torch.bool, device=DEV)       # as by the recurrence: a key's row, a value's column
            if which == 1:
                gone[heads, c] = True
            elif which == 2:
                gone[h, :, c] = True
            elif which == 3:
                gone[h] = True
            assert torch.equal(state[0][~gone], want_state[0][~gone]) and not state[0][gone].isfinite().any(), (t, which)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_a_batch_with_garbage_behind_each_end(dtype):
    clean = inputs(3, 140, 1, 2, 64, 48, dtype, seed=1)[0]
    ends = [1, 77, 130]
    args = [x.clone() for x in clean]
    for n, end in enumerate(ends):
        for x, junk in zip(args[:4], (float("nan"), float("inf"), float("nan"), float("nan"))):
            x[n, end:] = junk
    out, want = decay_attention(*args)[0], decay_attention(*clean)[0]
    for n, end in enumerate(ends):
        assert torch.equal(out[n, :end], want[n, :end]) and not out[n, end:].isfinite().any()


def test_a_packed_sequence_that_is_not_finite_leaves_the_others_alone():
    lengths = [70, 1, 700, 61]
    clean, cot = inputs(1, sum(lengths), 2, 4, 40, 32, BF16, N=4, seed=2)
    offsets = offsets_of(lengths)

    def run(args):
        leaves = [t.clone().requires_grad_() for t in args]
        got = decay_attention(*leaves, offsets=offsets)
        return (*got, *torch.autograd.grad(got, leaves, cot))

    want = run(clean)
    args = [x.clone() for x in clean]
    for x in args[:4]:
        x[0, 71:771] = float("nan")
    got = run(args)
    for i in (0, 2, 3, 4, 5):
        assert torch.equal(got[i][:, :71], want[i][:, :71]) and torch.equal(got[i][:, 771:], want[i][:, 771:])
    assert got[0][:, 71:771].isnan().all()
    for i in (1, 6):
        assert torch.equal(got[i][[0, 1, 3]], want[i][[0, 1, 3]])
    assert got[1][2].isnan().all()


# ------------------------------------------------------------------ together, streams, graphs

def test_a_layer_from_norms_to_prompt_to_tokens():
    """The operators as a layer runs them: a norm of the rows, heads with rotation, a packed prompt, a norm of each head
    with weights of its own, then tokens one by one on the pooled states; against the oracles' chain, with its gradients."""
    gen = torch.Generator(device=DEV).manual_seed(20)
    H, K, V, lengths = 3, 64, 48, [70, 3, 129]
    T, D = sum(lengths), 3 * (2 * 64 + 48)
    x, w, b = randn(gen, (1, T, D)) * 2 + 1, 1 + 0.1 * randn(gen, (D,)), 0.1 * randn(gen, (D,))
    g, hw = -torch.rand(H, generator=gen, device=DEV), 1 + 0.1 * randn(gen, (H, V))
    angle = randn(gen, (200, 16)) * 3
    tables = (angle.cos(), angle.sin())

    def layer(x, w, b, g, hw, pos, attend):
        rows = layer_norm(x, w, b)
        q, k = rows[..., :H * K].unflatten(-1, (H, K)), rows[..., H * K:2 * H * K].unflatten(-1, (H, K))
        q, k = qk_norm_rotate(q, k, None, None, *tables, pos, kind="l2")
        out, state = attend(q, k, rows[..., 2 * H * K:].unflatten(-1, (H, V)), g)
        return layer_norm(out, hw, eps=1e-3), state

    def oracle(x, w, b, g, hw, pos, s0, lens):
        rows = ref.lnm_fwd(x, w, b, 1e-5)
        how = (None, f64(tables[0]), f64(tables[1]), pos, "l2", 1e-6, False)
        raw = rows[..., :H * K].reshape(*rows.shape[:2], H, K), rows[..., H * K:2 * H * K].reshape(*rows.shape[:2], H, K)
        q, k = (lm_ops.qkn_fwd(y, *how) for y in raw)
        v = rows[..., 2 * H * K:].reshape(*rows.shape[:2], H, V)
        out, state = ref.dca_fwd(q, k, v, g, s0, K ** -0.5, lens)
        return (rows, raw, how, q, k, v, out), ref.lnm_fwd(out, hw, None, 1e-3), state

    pos = torch.cat([torch.arange(n) for n in lengths])[None].to(DEV)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, g, hw)]
    y, state = layer(*leaves, pos, lambda *a: decay_attention(*a, offsets=offsets_of(lengths)))
    cot = [randn(gen, y.shape), randn(gen, state.shape)]
    grads = torch.autograd.grad([y, state], leaves, cot)
    f = [f64(t) for t in (x, w, b, g, hw)]
    s0 = np.zeros((3, H, K, V))
    (rows, raw, how, q, k, v, out), want, r_state = oracle(*f, pos.cpu().numpy(), s0, lengths)
    # An error of 1e-5 of the largest out, divided by the smallest deviation of a head: `by` times 1e-5.  A norm turns an
    # error e of its row into at most (2 + |h|) r e, that is 2 |y| r e for |h| >= 2, and adds 1e-5 of its own.
    near = lambda out: 3e-5 * max(1.0, np.abs(out).max() / np.sqrt(out.var(-1) + 1e-3).min())
    by = near(out)
    assert np.abs(f64(y) - want).max() <= by * np.abs(want).max()
    close("state", state, r_state)
    d_out, d_hw, _ = ref.lnm_bwd(out, f[4], 1e-3, f64(cot[0]), True)
    dq, dk, dv, dg, _ = ref.dca_bwd(q, k, v, f[3], s0, K ** -0.5, d_out, f64(cot[1]), lengths)
    parts = [lm_ops.qkn_bwd(y, *how, d)[0] for y, d in zip(raw, (dq, dk))] + [dv]
    dx, dw, db = ref.lnm_bwd(f[0], f[1], 1e-5, np.concatenate([p.reshape(1, T, -1) for p in parts], -1))
    for name, a, c in zip(("x", "weight", "bias", "log_decay", "weights of heads"), grads, (dx, dw, db, dg, d_hw)):
        # What reaches the attention is off as y is; it, the two norms of heads and rows add 1e-5 each.
        assert np.abs(f64(a) - c).max() <= (by + 4e-5) * np.abs(c).max(), name
    pool = torch.zeros(5, H, K, V, device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    pool[slots.long()] = state.detach()
    for step in range(3):
        x = randn(gen, (3, 1, D)) * 2 + 1
        at = torch.tensor([[n + step] for n in lengths], device=DEV)
        y, _ = layer(x, w, b, g, hw, at, lambda *a: (decay_attention_step(*a, pool, slots=slots), None))
        (*_, out), want, r_state = oracle(f64(x), *f[1:], at.cpu().numpy(), r_state, None)
        assert np.abs(f64(y) - want).max() <= near(out) * np.abs(want).max()
    close("pool", pool[slots.long()], r_state)


@pytest.mark.parametrize("T,head", [(200, False), (1300, True)])
def test_streams_graphs_and_bits(T, head):
    args, cot = inputs(2, T, 2, 4, 128, 64, BF16, seed=21, head=head)
    call = lambda **kw: (lambda o: o[:2] + capi.dca_bwd(*args[:4], o[2], *cot, **kw))(capi.dca_fwd(*args, want_saved=True, **kw))
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
    gen = torch.Generator(device=DEV).manual_seed(31)
    args, cot = inputs(2, 90, 2, 4, 64, 32, BF16, seed=31, head=True)
    leaves = [t.clone().requires_grad_() for t in args + [1 + 0.1 * randn(gen, (4, 32), BF16), 0.1 * randn(gen, (4, 32), BF16)]]

    def step():
        out, state = decay_attention(*leaves[:5])
        y = layer_norm(out, *leaves[5:])
        return [t.detach() for t in (y, state, *torch.autograd.grad([y, state], leaves, cot))]

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


def test_a_decoding_step_captured_and_replayed():
    args, slots = step_inputs(3, 1, 2, 4, 64, 64, 6, BF16, seed=8, head=True)
    start = args[4].clone()
    want = [decay_attention_step(*args, slots=slots) for _ in range(3)]
    end = args[4].clone()
    args[4].copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = decay_attention_step(*args, slots=slots)
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, w)
    assert torch.equal(args[4], end)


def test_a_result_does_not_depend_on_the_sequences_beside_it():
    """As long as the segments are the same, a sequence of a batch has the bits that it has alone."""
    args, cot = inputs(9, 90, 2, 4, 64, 48, BF16, seed=25)
    leaves = [t.clone().requires_grad_() for t in args]
    whole = decay_attention(*leaves)
    grads = torch.autograd.grad(whole, leaves, cot)
    for n in (0, 4, 8):
        one = [t[n:n + 1].clone().requires_grad_() for t in args]
        part = decay_attention(*one)
        for a, b in zip((*whole, *grads), (*part, *torch.autograd.grad(part, one, [c[n:n + 1] for c in cot]))):
            assert torch.equal(a[n:n + 1], b)


def test_a_scale_in_a_tensor_is_read_at_each_call():
    args, cot = inputs(1, 20, 1, 2, 16, 16, F32, seed=9)
    scale = torch.tensor(0.5)
    leaves = [t.clone().requires_grad_() for t in args]
    out = decay_attention(*leaves, scale=scale)
    scale.fill_(2.0)
    for a, b in zip(torch.autograd.grad(out, leaves, cot), torch.autograd.grad(decay_attention(*leaves, scale=0.5), leaves, cot)):
        assert torch.equal(a, b)                     # the backward pass keeps the forward's
    assert torch.equal(decay_attention(*args, scale=scale)[0], decay_attention(*args, scale=2.0)[0])


def test_refusals():
    args, cot = inputs(2, 5, 2, 4, 16, 8, BF16, seed=22)
    q, k, v, g, s = args
    offsets = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    call = lambda **kw: decay_attention(**{**dict(query=q, key=k, value=v, log_decay=g, initial_state=s), **kw})
    for kw in (dict(key=k[:1]), dict(key=k[..., :8]), dict(value=v[:, :, :3]), dict(value=v[:, :4]), dict(log_decay=g.to(BF16)),
               dict(log_decay=g[:, :4]), dict(log_decay=g[0, 0, :3]), dict(log_decay=g[0]), dict(log_decay=g[0, 0, 0]), dict(log_decay=g.cpu()),
               dict(initial_state=s[:1]), dict(initial_state=s.to(BF16)), dict(offsets=offsets),
               dict(query=q[0]), dict(query=q.double(), key=k.double(), value=v.double()), dict(key=k.to(F16)), dict(initial_state=s.cpu()),
               dict(query=torch.zeros(2, 5, 2, 200, device=DEV, dtype=BF16), key=torch.zeros(2, 5, 2, 200, device=DEV, dtype=BF16)),
               dict(value=torch.zeros(2, 5, 4, 1025, device=DEV, dtype=BF16))):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    one = [t[:1] for t in args]
    for bad in (offsets.long(), offsets.cpu(), offsets[None], offsets[:0]):
        with pytest.raises(ValueError):
            decay_attention(*one, offsets=bad)
    saved = capi.dca_fwd(*args, want_saved=True)[2]
    with pytest.raises(ValueError):
        capi.dca_bwd(*args[:4], saved[:-1], *cot)
    with pytest.raises(RuntimeError):                         # the gradient's own gradient
        leaf = q.clone().requires_grad_()
        d, = torch.autograd.grad(call(query=leaf)[0].float().sum(), [leaf], create_graph=True)
        d.sum().backward()
    for kw in (dict(state=s[:1]), dict(state=s.to(BF16)), dict(slots=offsets.long()), dict(slots=offsets[:1]), dict(log_decay=g[:, :1])):
        with pytest.raises((ValueError, TypeError)):
            decay_attention_step(**{**dict(query=q, key=k, value=v, log_decay=g, state=s), **kw})
    torch.cuda.synchronize()
