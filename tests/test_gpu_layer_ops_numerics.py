"""Whether linear attention with decays keeps whole significands of what it computes on the way to outputs and
gradients of 16 bits: differences of two numbers that are alike to 2^-17 of their size (needs an MI355X).

Every case has an exact value a - b with a, b in [1, 2), made of few terms: products of bfloat16 parts of a and b with
ones, where a whole number is its three parts' sum.  Three parts of a number hold its 24 bits; the six products of parts
and the float32 sums over them that are not exact are off by at most 6 * 2^-24 * 2 each side, together under 2^-20.  The
output's own rounding is at most 2^-17 * 2^-9 (or half a subnormal step of float16, 2^-25) and inside that too.  A part
left out costs up to 2^-17 on each side."""
import pytest
import torch

from quaternion_cumprod_autodiff_amd import decay_attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
BOUND = 2.0 ** -20
K_SIZES = [32, 64, 128]


def nearly_equal(shape, seed):
    """Float32 numbers in [1, 2) with random last bits, and the same moved by 2^-17: the difference is exact, and two
    bfloat16 parts, whose last step there is 2^-16, cannot tell how large it is."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    a = (1 + 0.9 * torch.rand(shape, generator=gen, device=DEV)).double()
    a = (a * 2 ** 22).round() / 2 ** 22
    return a.float(), (a + 2.0 ** -17).float()


def parts(x, dtype):
    """Numbers of `dtype`, three of them, whose sum is x: [.., 3]."""
    out, left = [], x.double()
    for _ in range(3):
        out.append(left.to(dtype))
        left = left - out[-1].double()
    assert not left.any()
    return torch.stack(out, -1)


def zeros(*shape, dtype=F32):
    return torch.zeros(*shape, device=DEV, dtype=dtype)


def near(label, got, want):
    off = float((got.double() - want.double()).abs().max())
    assert torch.isfinite(got.double()).all() and off <= BOUND, f"{label}: off by {off:.3e}, bound {BOUND:.3e}"


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("K", K_SIZES)
def test_out_of_differences_of_state_rows(K, dtype):
    """out = S_1 - S_{K-1}."""
    T, V = 70, 48
    q, k, v = zeros(1, T, 1, K, dtype=dtype), zeros(1, T, 1, K, dtype=dtype), zeros(1, T, 1, V, dtype=dtype)
    q[..., 1], q[..., K - 1] = 1, -1
    s = zeros(1, 1, K, V)
    s[0, 0, K - 1], s[0, 0, 1] = nearly_equal((V,), K)
    out, state = decay_attention(q, k, v, zeros(1, T, 1), s, scale=1.0)
    assert torch.equal(state, s)
    near("out", out, (s[0, 0, 1].double() - s[0, 0, K - 1].double()).expand(1, T, 1, V))


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("K", K_SIZES)
def test_out_of_differences_of_pairs(K, dtype):
    """P_i0 = a, P_i1 = b: keys of a's and b's parts, queries of ones, values of 1 and -1; a chunk of its tokens."""
    T, H, V = 30, 24, 16
    a, b = nearly_equal((H,), 3 + K)
    q, k, v = zeros(1, T, H, K, dtype=dtype), zeros(1, T, H, K, dtype=dtype), zeros(1, T, H, V, dtype=dtype)
    q[0, 2:, :, :3] = 1
    k[0, 0, :, :3], k[0, 1, :, :3] = parts(a, dtype), parts(b, dtype)
    v[0, 0], v[0, 1] = 1, -1
    out, _ = decay_attention(q, k, v, zeros(1, T, H), scale=1.0)
    want = (a.double() - b.double())[None, None, :, None].expand(1, T, H, V).clone()
    want[:, :2] = 0
    near("out", out, want)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("K", K_SIZES)
def test_gradient_of_value_from_differences_of_the_states_cotangent(K, dtype):
    """dV = K dS1 with keys that are 1 at one row of dS1 and -1 at another."""
    T, V = 70, 48
    q, k, v = zeros(1, T, 1, K, dtype=dtype), zeros(1, T, 1, K, dtype=dtype), zeros(1, T, 1, V, dtype=dtype)
    k[..., 1], k[..., K - 1] = 1, -1
    d = zeros(1, 1, K, V)
    d[0, 0, K - 1], d[0, 0, 1] = nearly_equal((V,), 5 + K)
    v.requires_grad_()
    _, state = decay_attention(q, k, v, zeros(1, T, 1), scale=1.0)
    dv, = torch.autograd.grad([state], [v], [d])
    near("gradient of value", dv, (d[0, 0, 1].double() - d[0, 0, K - 1].double()).expand(1, T, 1, V))


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("K", K_SIZES)
def test_gradient_of_value_from_differences_of_pairs(K, dtype):
    """dV_j = P_ij - P_hj of two later tokens, whose queries are a's and b's parts and whose cotangents are 1 and -1."""
    T, H, V = 30, 24, 16
    a, b = nearly_equal((H,), 7 + K)
    q, k, v = zeros(1, T, H, K, dtype=dtype), zeros(1, T, H, K, dtype=dtype), zeros(1, T, H, V, dtype=dtype)
    k[0, :-2, :, :3] = 1
    q[0, -2, :, :3], q[0, -1, :, :3] = parts(a, dtype), parts(b, dtype)
    do = zeros(1, T, H, V, dtype=dtype)
    do[0, -2], do[0, -1] = 1, -1
    v.requires_grad_()
    out, _ = decay_attention(q, k, v, zeros(1, T, H), scale=1.0)
    dv, = torch.autograd.grad([out], [v], [do])
    want = (a.double() - b.double())[None, None, :, None].expand(1, T, H, V).clone()
    want[:, -2:] = 0
    near("gradient of value", dv, want)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("K", K_SIZES)
def test_gradients_of_query_and_key_from_differences_of_pairs(K, dtype):
    """Phi_ij = O_i.V_j: for queries, values of a's and b's parts read by cotangents of ones, with keys of 1 and -1; for
    keys the other way round."""
    T, H, V = 30, 24, 16
    a, b = nearly_equal((H,), 11 + K)
    none = lambda w: zeros(1, T, H, w, dtype=dtype)
    want = (a.double() - b.double())[None, None, :].expand(1, T, H).clone()

    q, k, v, do = none(K), none(K), none(V), none(V)
    v[0, 0, :, :3], v[0, 1, :, :3] = parts(a, dtype), parts(b, dtype)
    k[0, 0, :, 5], k[0, 1, :, 5] = 1, -1
    do[0, 2:, :, :3] = 1
    q.requires_grad_()
    out, _ = decay_attention(q, k, v, zeros(1, T, H), scale=1.0)
    dq, = torch.autograd.grad([out], [q], [do])
    x = want.clone()
    x[:, :2] = 0
    near("gradient of query", dq[..., 5], x)
    assert not dq[..., :5].any() and not dq[..., 6:].any()

    q, k, v, do = none(K), none(K), none(V), none(V)
    do[0, -2, :, :3], do[0, -1, :, :3] = parts(a, dtype), parts(b, dtype)
    q[0, -2, :, 5], q[0, -1, :, 5] = 1, -1
    v[0, :-2, :, :3] = 1
    k.requires_grad_()
    out, _ = decay_attention(q, k, v, zeros(1, T, H), scale=1.0)
    dk, = torch.autograd.grad([out], [k], [do])
    x = want.clone()
    x[:, -2:] = 0
    near("gradient of key", dk[..., 5], x)
    assert not dk[..., :5].any() and not dk[..., 6:].any()
