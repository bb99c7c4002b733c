"""Layer norm and linear attention with decays at the sizes that their headers allow and little reaches (needs an
MI355X)."""
import threading

import numpy as np
import pytest
import torch

from oracle import layer_ops as ref
from quaternion_cumprod_autodiff_amd import capi, decay_attention, decay_attention_step, layer_norm

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


def test_attention_beyond_2_to_the_31_elements():
    """Values of 4.8 GB: a decay of -inf makes what is behind it, gradients too, what the tail alone gives, bit for bit."""
    T, Hk, Hv, K, V = 131072, 16, 144, 16, 128
    cut, tail = T - 1024, 2880         # whole chunks; segments differ, but decays forget a token within a chunk or two
    assert T * Hv * V > 2 ** 31
    gen = torch.Generator(device=DEV).manual_seed(8)
    q, k = (torch.empty(1, T, Hk, K, device=DEV, dtype=BF16).normal_(0, 0.5, generator=gen) for _ in range(2))
    v = torch.empty(1, T, Hv, V, device=DEV, dtype=BF16).normal_(generator=gen)
    g = -torch.rand(1, T, Hv, generator=gen, device=DEV)
    g[:, cut] = -float("inf")
    dy = torch.zeros_like(v)
    dy[:, cut:].normal_(generator=gen)

    def run(*args):
        *leaves, cot = args
        leaves = [t.requires_grad_() for t in leaves]
        out, state = decay_attention(*leaves)
        return (out.detach(), *torch.autograd.grad(out, leaves, cot)), state.detach()

    whole, state = run(q, k, v, g, dy)
    rows, last = run(*(t.detach()[:, T - tail:].clone() for t in (q, k, v, g, dy)))
    assert torch.equal(state, last)
    for name, a, b in zip(("out", "query", "key", "value", "log_decay"), whole, rows):
        assert b[:, cut - T:].any() and torch.equal(a[:, cut:], b[:, cut - T:]), name


def test_many_packed_sequences():
    """70000 of them, of no to three tokens: as a padded batch, bit for bit."""
    N, L, H = 70000, 3, 2
    gen = torch.Generator(device=DEV).manual_seed(9)
    lengths = torch.randint(0, L + 1, (N,), generator=gen, device=DEV)
    offsets = torch.cat([torch.zeros(1, device=DEV, dtype=torch.int32), lengths.cumsum(0).int()])
    T = int(offsets[-1])
    q, k = (torch.empty(1, T, 1, 32, device=DEV, dtype=BF16).normal_(generator=gen) for _ in range(2))
    v = torch.empty(1, T, H, 32, device=DEV, dtype=BF16).normal_(generator=gen)
    g = -torch.rand(1, T, H, generator=gen, device=DEV)
    at = (offsets[:-1, None].long() + torch.arange(L, device=DEV)).clamp_max(T - 1)
    inside = torch.arange(L, device=DEV) < lengths[:, None]
    padded = lambda t: torch.where(inside.reshape(N, L, *[1] * (t.dim() - 2)), t[0][at], torch.zeros((), device=DEV, dtype=t.dtype))
    out, state = decay_attention(q, k, v, g, offsets=offsets)
    want, last = decay_attention(*(padded(t) for t in (q, k, v, g)))
    assert torch.equal(out[0], want[inside]) and torch.equal(state, last)


def test_calls_of_several_threads_and_streams():
    """Plans are shared by a process' threads: each call's bits are what it gives alone."""
    def inputs(seed):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        q = torch.randn(1, 700, 4, 64, generator=gen, device=DEV).to(BF16)
        return q, -torch.rand(1, 700, 4, generator=gen, device=DEV)

    def call(q, g):
        leaf = q.clone().requires_grad_()
        out, _ = decay_attention(leaf, q, q, g)
        return out.detach(), torch.autograd.grad(out, [leaf], q)[0], layer_norm(q)

    seeds, got = range(4), {}
    data = [inputs(s) for s in seeds]
    want = [call(*d) for d in data]
    torch.cuda.synchronize()

    def work(seed):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got[seed] = [call(*data[seed]) for _ in range(10)]
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(s,)) for s in seeds]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(a, b) for s in seeds for x in got[s] for a, b in zip(x, want[s]))
