"""Layer norm and linear attention with decays at the sizes that their headers allow and little reaches (needs an
MI355X)."""
import numpy as np
import pytest
import torch

from oracle import layer_ops as ref
from quaternion_cumprod_autodiff_amd import capi, decay_attention_step, layer_norm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def f64(t):
    return t.detach().double().cpu().numpy()


def near(label, got, want, size):
    """Half a step of bfloat16 for the one rounding, and 1e-5 of the terms' size for float32's sums over a row: by at most
    14 levels of pairs and 32 in a row, 46 2^-24, and four products more."""
    off = np.abs(f64(got) - want) - 2.0 ** -8 * np.abs(want) - 1e-5 * size
    assert np.isfinite(f64(got)).all() and off.max() <= 1e-30, f"{label}: {off.max():.3e} too far"


@pytest.mark.parametrize("heads,D", [(65535, 1024), (65536, 1024), (1 << 20, 2040)], ids=str)
def test_norm_of_many_weights_of_heads(heads, D):
    """Columns of weights on both sides of 2^26, and close to 2^31: their gradients' kernel takes them 16 to a block, and a
    launch holds less than 2^32 threads.  One token, so a bias' gradient is its cotangent, bit for bit."""
    print(f"[norm of {heads} heads of {D}]", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(heads)
    x, dy = (torch.empty(1, heads, D, device=DEV, dtype=BF16).normal_(generator=gen) for _ in range(2))
    w, b = (torch.empty(heads, D, device=DEV, dtype=BF16).normal_(1.0, 0.3, generator=gen) for _ in range(2))
    leaves = [t.requires_grad_() for t in (x, w, b)]
    y = layer_norm(*leaves)
    dx, dw, db = torch.autograd.grad(y, leaves, dy)
    assert torch.equal(db, dy[0])
    edge = min(heads, 65536)
    for at in (slice(0, 3), slice(edge - 2, edge + 1), slice(heads - 3, heads)):
        fx, fw, fb, fd = (f64(t) for t in (x[:, at], w[at], b[at], dy[:, at]))
        h = ref.lnm_fwd(fx, None, None, 1e-5)
        near("y", y[:, at], ref.lnm_fwd(fx, fw, fb, 1e-5), np.abs(h).max(-1, keepdims=True) * np.abs(fw).max() + np.abs(fb))
        rx, rw, _ = ref.lnm_bwd(fx, fw, 1e-5, fd, True)
        near("gradient of weight", dw[at], rw, np.abs(fd[0]) * np.abs(h[0]).max())
        big = (np.abs(fd) * np.abs(fw)).max(-1, keepdims=True) * (1 + np.abs(h).max(-1, keepdims=True))
        near("gradient of x", dx[:, at], rx, big / np.sqrt(fx.var(-1, keepdims=True)))


@pytest.mark.parametrize("form", ["one token", "dense", "tokens apart", "batch apart", "apart"])
def test_norm_of_more_rows_to_a_token_than_heads(form):
    """A third axis above 2^20, of rows that are alike: as the same rows in two axes, bit for bit, gradients too."""
    H, D = (1 << 20) + 3, 8
    gen = torch.Generator(device=DEV).manual_seed(6)
    B, T = {"one token": (1, 1), "dense": (2, 2), "tokens apart": (1, 3), "batch apart": (2, 1), "apart": (2, 2)}[form]
    x = torch.empty(B + 1, T + 1, H + 1, D, device=DEV, dtype=BF16).normal_(generator=gen)[:B, :T, :H]
    if form in ("one token", "dense"):
        x = x.contiguous()
    w, b = (torch.empty(D, device=DEV, dtype=BF16).normal_(generator=gen) for _ in range(2))
    if form == "apart":
        with pytest.raises(ValueError, match="contiguous"):
            layer_norm(x, w, b)
        x = x.contiguous()
    dy = torch.empty(B, T, H, D, device=DEV, dtype=BF16).normal_(generator=gen)
    leaves = [t.detach().requires_grad_() for t in (x, w, b)]
    y = layer_norm(*leaves)
    grads = torch.autograd.grad(y, leaves, dy)
    rows = [x.reshape(-1, D).requires_grad_(), *leaves[1:]]
    want = layer_norm(*rows)
    assert torch.equal(y, want.reshape(y.shape))
    for got, same in zip(grads, torch.autograd.grad(want, rows, dy.reshape(-1, D))):
        assert torch.equal(got, same.reshape(got.shape))
    if form == "one token":
        with pytest.raises(ValueError, match="2\\^20"):
            layer_norm(x, torch.empty(H, D, device=DEV, dtype=BF16))


def test_as_many_slots_as_a_step_looks_through():
    """2^20 rows of one head and 32 columns, the last of them named by the first row already, and by its neighbour."""
    N, K, V = 1 << 20, 2, 8
    gen = torch.Generator(device=DEV).manual_seed(4)
    q, k = (torch.randn(N, 1, 1, K, generator=gen, device=DEV) for _ in range(2))
    v, g = torch.randn(N, 1, 1, V, generator=gen, device=DEV), -torch.rand(N, 1, 1, generator=gen, device=DEV)
    state = torch.randn(N, 1, K, V, generator=gen, device=DEV)
    slots = torch.randperm(N, generator=gen, device=DEV).int()
    slots[N - 1], slots[N - 2], slots[N // 2] = slots[0], slots[N - 3], slots[1]
    before = state.clone()
    out = decay_attention_step(q, k, v, g, state, slots=slots)
    run = torch.ones(N, dtype=torch.bool, device=DEV)
    run[[N - 1, N - 2, N // 2]] = False
    rows = slots.long()[run]
    want = g[run].double().exp()[:, :, :, None] * before[rows].double() + k[run, 0, :, :, None].double() * v[run, 0, :, None, :].double()
    # Two roundings and an exponential's of terms, and float32 sums of two of them.
    assert ((state[rows].double() - want).abs() <= 2.0 ** -21 * (1 + before[rows].double().abs() + (k[run, 0, :, :, None] * v[run, 0, :, None, :]).abs())).all()
    assert not out[~run].any()
    read = (want * q[run, 0, :, :, None].double()).sum(2) * K ** -0.5
    assert ((out[run, 0].double() - read).abs() <= 2.0 ** -19 * (1 + (want.abs() * q[run, 0, :, :, None].abs()).sum(2))).all()
    left = torch.ones(N, dtype=torch.bool, device=DEV)
    left[rows] = False
    assert torch.equal(state[left], before[left])
    with pytest.raises(capi.QuatCumprodError):
        decay_attention_step(*(torch.cat([t, t[:1]]) for t in (q, k, v, g)), state, slots=torch.cat([slots, slots[:1]]))
