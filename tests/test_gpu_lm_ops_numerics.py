"""Where the gated delta rule, its decoding step and the query/key norm lose bits, range or bookkeeping, if they do:
each against the float64 oracle's value or formula (needs an MI355X)."""
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


def close(label, got, want, top=None):
    """Half a step of the type for its one rounding, and 1e-5 of the largest value for the float32 arithmetic, as derived
    beside the operators' other tests."""
    rel = torch.finfo(got.dtype).eps / 2
    got, want = f64(got), np.asarray(want)
    top = float(np.abs(want).max()) if top is None else top
    off = float((np.abs(got - want) - rel * np.abs(want)).max())
    assert np.isfinite(got).all() and off <= 1e-5 * top, f"{label}: {off:.3e} over the rounding, largest {top:.3e}"


def randn(gen, shape, dtype=F32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=F32).to(dtype)


def unit(gen, shape, dtype):
    return torch.nn.functional.normalize(randn(gen, shape), dim=-1).to(dtype)


# ------------------------------------------------------------------ whole significands

def nearly_equal(gen, shape):
    """Float32 numbers in [1, 2) with random last bits, and the same moved by 2^-17: the difference is exact, and two
    bfloat16 parts, whose last step there is 2^-16, cannot tell how large it is."""
    a = (1 + 0.9 * torch.rand(shape, generator=gen, device=DEV)).double()
    a = (a * 2 ** 22).round() / 2 ** 22
    return a.float(), (a + 2.0 ** -17).float()


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("K", [32, 64, 128])
def test_differences_of_state_rows_keep_the_last_bits(K, dtype):
    """out = S_0 - S_1, rows of the initial state that are alike to 2^-17 of their size.  Six products of parts and their
    float32 sums are off by at most 6 * 2^-24 * (1 + 1 + 2 * 2) * 2 / 2 < 2^-20; a part left out costs 2^-17 or more."""
    gen = torch.Generator(device=DEV).manual_seed(K)
    T, V = 70, 48
    q, k, v = torch.zeros(1, T, 1, K, device=DEV, dtype=dtype), torch.zeros(1, T, 1, K, device=DEV, dtype=dtype), torch.zeros(1, T, 1, V, device=DEV, dtype=dtype)
    q[..., 1], q[..., K - 1] = 1, -1
    g = b = torch.zeros(1, T, 1, device=DEV)
    s = torch.zeros(1, 1, K, V, device=DEV)
    s[0, 0, K - 1], s[0, 0, 1] = nearly_equal(gen, (V,))
    out, state = gated_delta_rule(q, k, v, g, b, s, scale=1.0)
    want = (s[0, 0, 1].double() - s[0, 0, K - 1].double()).expand(1, T, 1, V)
    assert torch.equal(state, s)
    assert ((out.double() - want).abs() <= 2.0 ** -20).all(), float((out.double() - want).abs().max())


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_differences_of_updates_keep_the_last_bits(dtype):
    """The same for two updates within a chunk: u_0 = b_0, u_1 = b_1 (values of 1, keys that are unit vectors), and later
    queries read u_0 - u_1."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    T, K, V, H = 40, 64, 16, 24
    q, k = (torch.zeros(1, T, 1, K, device=DEV, dtype=dtype) for _ in range(2))
    v = torch.ones(1, T, H, V, device=DEV, dtype=dtype)
    k[0, 0, 0, 0] = k[0, 1, 0, 1] = 1
    q[0, 2:, 0, 0], q[0, 2:, 0, 1] = -1, 1
    g, b = torch.zeros(1, T, H, device=DEV), torch.zeros(1, T, H, device=DEV)
    b[0, 0], b[0, 1] = nearly_equal(gen, (H,))
    out, _ = gated_delta_rule(q, k, v, g, b, scale=1.0)
    want = (b[0, 1].double() - b[0, 0].double())[None, None, :, None].expand(1, T, H, V).clone()
    want[:, :2] = 0
    assert ((out.double() - want).abs() <= 2.0 ** -20).all(), float((out.double() - want).abs().max())


# ------------------------------------------------------------------ gradients of strong decays

@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("g0", [-3.0, -8.0, -20.0, -40.0])
def test_gradients_of_uniform_strong_decays(g0, dtype):
    """The gradient of log_decay scales with exp(log_decay): nothing that does not carry the decay may be left in it."""
    gen = torch.Generator(device=DEV).manual_seed(int(-g0))
    B, T, Hk, Hv, K, V = 1, 150, 1, 2, 64, 48
    args = [unit(gen, (B, T, Hk, K), dtype), unit(gen, (B, T, Hk, K), dtype), randn(gen, (B, T, Hv, V), dtype),
            torch.full((B, T, Hv), g0, device=DEV), torch.rand(B, T, Hv, generator=gen, device=DEV), randn(gen, (B, Hv, K, V))]
    cot = [randn(gen, (B, T, Hv, V), dtype), randn(gen, (B, Hv, K, V))]
    leaves = [t.requires_grad_() for t in args]
    grads = torch.autograd.grad(gated_delta_rule(*leaves), leaves, cot)
    want = ref.gdr_bwd(*[f64(t) for t in args], K ** -0.5, *[f64(c) for c in cot])
    for name, got, w in zip(("query", "key", "value", "log_decay", "beta", "initial_state"), grads, want):
        close("gradient of " + name, got, w)


@pytest.mark.parametrize("K", [24, 128])
def test_gradients_of_strong_decays_among_weak_ones(K):
    """At the tokens whose decay is strong the gradient is far below the others': it is held to its own size.  A decay of
    exactly nothing has a gradient of exactly nothing."""
    gen = torch.Generator(device=DEV).manual_seed(K)
    B, T, H, V = 2, 200, 2, 32
    args = [unit(gen, (B, T, H, K), F32), unit(gen, (B, T, H, K), F32), randn(gen, (B, T, H, V)), -0.1 * torch.rand(B, T, H, generator=gen, device=DEV),
            torch.rand(B, T, H, generator=gen, device=DEV), randn(gen, (B, H, K, V))]
    cot = [randn(gen, (B, T, H, V)), randn(gen, (B, H, K, V))]
    strong = [0, 5, 63, 64, 90, 127, 128, 191, 192, 199]
    args[3][:, strong] = -25.0
    args[3][:, [30, 150]] = -float("inf")
    leaves = [t.requires_grad_() for t in args]
    got = torch.autograd.grad(gated_delta_rule(*leaves), leaves, cot)[3]
    want = ref.gdr_bwd(*[f64(t) for t in args], K ** -0.5, *[f64(c) for c in cot])[3]
    close("all", got, want)
    # The bound is 1e-5 of the token's own largest gradient.  (exp(-25) times the largest of all tokens is no bound on it: at
    # the last token <dS, S> is 20 times that of a weak token, and 1e-5 of the smaller figure would be 5e-7 of the value,
    # below the sqrt(6 (128 + 32 + 64)) 2^-23 = 4e-6 that float32 sums of so many terms are off by.)
    for t in strong:
        close(f"token {t}", got[:, t], want[:, t])
    assert not got[:, [30, 150]].any()


# ------------------------------------------------------------------ heads far from one

@pytest.mark.parametrize("kind", ["rms", "l2"])
@pytest.mark.parametrize("D", [64, 90])
@pytest.mark.parametrize("size,eps", [(1e15, 1e-6), (1e13, 1e-6), (1e-14, 0.0), (1e-16, 1e-36)])
def test_norm_gradients_of_large_and_small_heads(size, eps, D, kind):
    """The gradient is of the order 1 / |x|, whatever |x|: no factor on the way may leave the range of float32.  Its two
    terms cancel in part, so the bound is of the largest term (see the norm's other tests)."""
    gen = torch.Generator(device=DEV).manual_seed(D)
    q, k = randn(gen, (2, 9, 3, D)) * size, randn(gen, (2, 9, 2, D)) * size
    w = 1 + 0.1 * randn(gen, (D,))
    leaves = [t.requires_grad_() for t in (q, k, w)]
    out = qk_norm_rotate(leaves[0], leaves[1], leaves[2], kind=kind, eps=eps)
    cot = [randn(gen, t.shape) for t in out]
    gq, gk, gw = torch.autograd.grad(out, leaves, cot)
    how = (None, None, None, kind, float(np.float32(eps)), False)
    close("out", out[0], ref.qkn_fwd(f64(q), f64(w), *how))
    want, want_w = ref.qkn_bwd(f64(q), f64(w), *how, f64(cot[0]))
    top = np.abs(want).max()
    assert np.isfinite(f64(gq)).all() and np.abs(f64(gq) - want).max() <= 1e-5 * 4 * top
    close("weight", gw, want_w)
    want, _ = ref.qkn_bwd(f64(k), None, *how, f64(cot[1]))
    assert np.isfinite(f64(gk)).all() and np.abs(f64(gk) - want).max() <= 1e-5 * 4 * np.abs(want).max()


# ------------------------------------------------------------------ in place

def test_a_step_on_states_that_a_graph_saved_is_noticed():
    gen = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = unit(gen, (2, 1, 1, 16), F32), unit(gen, (2, 1, 1, 16), F32), randn(gen, (2, 1, 2, 8))
    g, b = -torch.rand(2, 1, 2, generator=gen, device=DEV), torch.rand(2, 1, 2, generator=gen, device=DEV)
    pool = randn(gen, (3, 2, 2, 16, 8))
    w = torch.ones_like(pool).requires_grad_()
    loss = (w * pool).sum()
    version = pool._version
    gated_delta_step(q, k, v, g, b, pool[:, 1])                    # a view of the pool
    assert pool._version > version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        gated_delta_step(q, k, v, g, b, torch.zeros(2, 2, 16, 8, device=DEV))    # has no version


def test_given_outputs_count_as_modified():
    gen = torch.Generator(device=DEV).manual_seed(2)
    q, k, v = unit(gen, (2, 3, 1, 16), F32), unit(gen, (2, 3, 1, 16), F32), randn(gen, (2, 3, 2, 8))
    g, b = -torch.rand(2, 3, 2, generator=gen, device=DEV), torch.rand(2, 3, 2, generator=gen, device=DEV)
    out, qo, ko = torch.zeros_like(v), torch.zeros_like(q), torch.zeros_like(k)
    at = [t._version for t in (out, qo, ko)]
    capi.gdr_fwd(q, k, v, g, b, out=out)
    capi.qkn_fwd(q, k, query_out=qo, key_out=ko)
    assert all(t._version > n for t, n in zip((out, qo, ko), at))
    n = out._version
    capi.gdr_step(q, k, v, g, b, torch.zeros(2, 2, 16, 8, device=DEV), out=out)
    assert out._version > n


# ------------------------------------------------------------------ inputs that are not finite

def rule_inputs(B, T, Hk, Hv, K, V, dtype, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return [unit(gen, (B, T, Hk, K), dtype), unit(gen, (B, T, Hk, K), dtype), randn(gen, (B, T, Hv, V), dtype),
            -torch.rand(B, T, Hv, generator=gen, device=DEV), torch.rand(B, T, Hv, generator=gen, device=DEV), randn(gen, (B, Hv, K, V))]


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("dtype,K,V,Hk,Hv", [(F32, 40, 24, 1, 2), (BF16, 128, 32, 2, 4), (F16, 64, 50, 1, 3), (BF16, 20, 64, 1, 80)], ids=str)
def test_what_is_not_finite_reaches_no_earlier_token(dtype, K, V, Hk, Hv, saved):
    """out of token t depends on tokens up to t: what comes before a NaN or an infinity keeps its bits, and from there on
    its head (a value: its column; a query: its token) is not finite, the final state neither."""
    T = 150
    clean = rule_inputs(1, T, Hk, Hv, K, V, dtype, K)
    run = lambda a: capi.gdr_fwd(*a, want_saved=saved)[:2]
    want, want_state = run(clean)
    group = Hv // Hk
    for t, bad in ((0, float("nan")), (5, float("inf")), (17, float("nan")), (31, -float("inf")), (63, float("nan")), (64, float("inf")), (149, float("nan"))):
        for which in range(5):
            args = [x.clone() for x in clean]
            h, c = (t + which) % args[which].shape[2], (7 * t + which) % args[which].shape[-1]
            if which < 3:
                args[which][0, t, h, c] = bad
            else:
                args[which][0, t, h] = float("nan") if which == 3 else bad      # a decay of -inf is an input like others
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
            gone = hit[T - 1][:, None].expand(Hv, K, V) if which else torch.zeros_like(state[0], dtype=torch.bool)
            assert torch.equal(state[0][~gone], want_state[0][~gone]) and not state[0][gone].isfinite().any(), (t, which)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_a_batch_with_garbage_behind_each_end(dtype):
    """Rows of a padded batch that hold anything: the tokens before keep their bits."""
    clean = rule_inputs(3, 140, 1, 2, 64, 48, dtype, 1)
    ends = [1, 77, 130]
    args = [x.clone() for x in clean]
    for n, end in enumerate(ends):
        for x, junk in zip(args[:5], (float("nan"), float("inf"), float("nan"), float("nan"), -float("inf"))):
            x[n, end:] = junk
    out, want = gated_delta_rule(*args)[0], gated_delta_rule(*clean)[0]
    for n, end in enumerate(ends):
        assert torch.equal(out[n, :end], want[n, :end]) and not out[n, end:].isfinite().any()


def test_a_packed_sequence_that_is_not_finite_leaves_the_others_alone():
    clean = rule_inputs(1, 200, 2, 4, 40, 32, BF16, 2)
    offsets = torch.tensor([0, 70, 71, 139, 200], dtype=torch.int32, device=DEV)
    clean[5] = torch.cat([clean[5] * (n + 1) for n in range(4)])
    want, want_state = gated_delta_rule(*clean, offsets=offsets)
    args = [x.clone() for x in clean]
    for x in args[:5]:
        x[0, 71:139] = float("nan")
    out, state = gated_delta_rule(*args, offsets=offsets)
    assert torch.equal(out[:, :71], want[:, :71]) and torch.equal(out[:, 139:], want[:, 139:]) and out[:, 71:139].isnan().all()
    assert torch.equal(state[[0, 1, 3]], want_state[[0, 1, 3]]) and state[2].isnan().all()


def test_gradients_of_what_is_not_finite_are_not_finite():
    """Entering as zero is the forward pass' way alone: a loss that saw a NaN has no finite gradients of what led to it."""
    for which in (1, 2, 4):
        args = rule_inputs(1, 100, 1, 2, 32, 16, F32, which)
        with torch.no_grad():
            args[which].view(100, -1)[40, 0] = float("nan")
        leaves = [t.requires_grad_() for t in args]
        out, state = gated_delta_rule(*leaves)
        for y in (out, state):
            grads = torch.autograd.grad(y.sum(), leaves, retain_graph=True)
            for i, name in ((1, "key"), (4, "beta"), (5, "initial_state")):
                if which != 2 or i == 4:              # a value's NaN is in the gradients that it multiplies
                    assert not grads[i].isfinite().all(), (which, name)
