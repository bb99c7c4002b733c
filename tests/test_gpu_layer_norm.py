"""Parity of layer norm and its VJP with the float64 oracle (needs an MI355X).

Tolerance of y, element by element: half a step of its type relative to the
value, for the one rounding, and 1e-5 of the row's largest |h w| + |b| for
float32: sums of D terms by at most 14 levels of pairs and 32 in a row are off by
46 2^-24 = 2.7e-6 at most, relative to the terms' sizes, and the products by
another 4 2^-24.  Where a row lies far from zero, its differences to the mean
are off by 2^-24 of the mean as well (the subtraction's rounding).  Gradients:
the same of their terms' sizes; a weight's is a sum of rows, in parts of parts."""
import numpy as np
import pytest
import torch

from oracle import layer_ops as ref
from quaternion_cumprod_autodiff_amd import capi, layer_norm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(gen, shape, dtype=F32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=F32).to(dtype)


def near(label, got, want, size):
    rel = torch.finfo(got.dtype).eps / 2
    low = rel * torch.finfo(got.dtype).smallest_normal      # half a step of what is below the normal numbers: 2^-25 for float16
    got = f64(got)
    assert got.shape == want.shape, label
    if want.size:
        off = np.abs(got - want) - np.maximum(rel * np.abs(want), low) - 1e-5 * size
        assert np.isfinite(got).all() and off.max() <= 1e-30, f"{label}: {off.max():.3e} too far"


def check(x, w, b, dy, eps=1e-5):
    by_head = w is not None and w.dim() == 2 or b is not None and b.dim() == 2
    y = layer_norm(x, w, b, eps=eps)
    leaves = [t.detach().requires_grad_() for t in (x, w, b) if t is not None]
    it = iter(leaves)
    lx, lw, lb = (None if t is None else next(it) for t in (x, w, b))
    y2 = layer_norm(lx, lw, lb, eps=eps)
    assert torch.equal(y, y2) and y.shape == x.shape and y.is_contiguous()
    grads = list(torch.autograd.grad(y2, leaves, dy))
    fx, fw, fb, fd = f64(x), None if w is None else f64(w), None if b is None else f64(b), f64(dy)
    want = ref.lnm_fwd(fx, fw, fb, eps)
    mean, r = fx.mean(-1, keepdims=True), 1 / np.sqrt(fx.var(-1, keepdims=True) + eps)
    far = 2.0 ** -24 / 1e-5 * np.abs(mean) * r                  # what a subtraction from the mean loses, in units of the bound
    h, ww = (fx - mean) * r, 1.0 if fw is None else np.abs(fw)
    near("y", y, want, (np.abs(h).max(-1, keepdims=True) + far) * np.max(ww) + (0.0 if fb is None else np.abs(fb)))
    dx, dw, db = ref.lnm_bwd(fx, fw, eps, fd, by_head)
    dh = np.abs(fd) * ww
    size = r * (dh.max(-1, keepdims=True) * (1 + np.abs(h).max(-1, keepdims=True)) * (1 + far))
    near("gradient of x", grads.pop(0), dx, size)
    axes = tuple(range(x.dim() - (2 if by_head else 1)))
    if w is not None:
        near("gradient of weight", grads.pop(0), dw, np.sqrt((fd * fd * (np.abs(h) + far) ** 2).sum(axes)) * 2 + np.abs(dw))
    if b is not None:
        near("gradient of bias", grads.pop(0), db, np.sqrt((fd * fd).sum(axes)) * 2 + np.abs(db))
    return y


def inputs(shape, affine, dtype, seed, heads=False):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = (randn(gen, shape) * (0.3 + randn(gen, shape[:-1] + (1,)).abs()) + randn(gen, shape[:-1] + (1,))).to(dtype)
    size = shape[-2:] if heads else shape[-1:]
    w = (1 + 0.3 * randn(gen, size)).to(dtype) if affine in ("both", "weight") else None
    b = (0.3 * randn(gen, size)).to(dtype) if affine in ("both", "bias") else None
    return x, w, b, randn(gen, shape, dtype)


SIZES = [(1, 1), (3, 2), (7, 8), (5, 31), (300, 40), (65, 64), (2, 3, 100), (33, 127), (9, 256), (4, 512), (3, 520), (2, 5, 777), (4, 1000), (6, 1024), (5, 1025),
         (3, 2048), (2, 2056), (3, 4096), (2, 4099), (1, 8192), (2, 8200), (2, 16384), (1, 16383), (2000, 16), (1200, 129)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("shape", SIZES, ids=str)
def test_norm(shape, dtype):
    print(f"[norm {shape} {dtype}]", flush=True)
    for affine in ("both", "none"):
        check(*inputs(shape, affine, dtype, sum(shape)))


@pytest.mark.parametrize("affine", ["weight", "bias"])
def test_weight_or_bias_alone(affine):
    check(*inputs((50, 72), affine, BF16, 1))
    check(*inputs((5, 9, 4, 33), affine, F32, 2, heads=True))


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("shape", [(3, 8), (1, 1, 1), (7, 3, 24), (2, 50, 5, 64), (2, 33, 4, 100), (1, 9, 2, 1024), (40, 1500, 16), (2, 3, 2, 4096), (3, 3, 3, 1100)], ids=str)
def test_weights_of_heads(shape, dtype):
    print(f"[heads {shape} {dtype}]", flush=True)
    check(*inputs(shape, "both", dtype, sum(shape), heads=True))


def test_rows_of_five_axes_and_one():
    x, w, b, dy = inputs((2, 3, 2, 4, 24), "both", F32, 3)
    check(x, w, b, dy)
    x, w, b, dy = inputs((2, 3, 2, 4, 24), "both", BF16, 4, heads=True)
    check(x, w, b, dy)
    check(*inputs((130,), "both", F32, 5))


@pytest.mark.parametrize("heads", [False, True])
def test_strides(heads):
    """Views of a fused projection, on 16 bytes and on 2, heads before tokens, a batch's first rows, broadcast rows."""
    gen = torch.Generator(device=DEV).manual_seed(6)
    for lead in (0, 8, 1):
        fused = randn(gen, (2, 30, lead + 4 * 64 + 24), BF16)
        x = fused[..., lead:lead + 256].unflatten(-1, (4, 64))
        _, w, b, dy = inputs(tuple(x.shape), "both", BF16, lead, heads)
        check(x, w, b, dy)
        check(x.transpose(1, 2), *inputs((2, 4, 30, 64), "both", BF16, lead, heads)[1:])
        if not heads:
            check(fused[..., lead:lead + 256], *inputs((2, 30, 256), "both", BF16, lead)[1:])
            check(fused[:, 3:9, lead:lead + 256], *inputs((2, 6, 256), "both", BF16, lead)[1:])
    one = randn(gen, (1, 1, 4, 40))
    check(one.expand(3, 5, 4, 40), *inputs((3, 5, 4, 40), "both", F32, 9, heads)[1:])
    check(randn(gen, (6, 5, 4, 40))[::2, 1:4], *inputs((3, 3, 4, 40), "both", F32, 9, heads)[1:])
    check(randn(gen, (5, 1, 4, 40))[::2], *inputs((3, 1, 4, 40), "both", F32, 9, heads)[1:])
    check(randn(gen, (5, 6, 1, 40))[::2, 1:4], *inputs((3, 3, 1, 40), "both", F32, 9, heads)[1:])


def test_rows_far_from_zero_constant_and_of_all_sizes():
    gen = torch.Generator(device=DEV).manual_seed(7)
    x, w, b, dy = inputs((60, 300), "both", F32, 8)
    check(x + 1000 * randn(gen, (60, 1)), w, b, dy)
    scale = 10.0 ** torch.linspace(-12, 15, 60, device=DEV)[:, None]
    check(x * scale, w, b, dy, eps=1e-30)
    flat = torch.full((3, 64), 7.25, device=DEV)
    y = layer_norm(flat, None, torch.arange(64.0, device=DEV))
    assert torch.equal(y, torch.arange(64.0, device=DEV).expand(3, 64))        # no variance: the bias alone


@pytest.mark.parametrize("D", [24, 128, 500, 1032, 4096, 9000])
def test_a_row_does_not_depend_on_the_rows_beside_it(D):
    """One row, a few, and so many that they come several to a group: the same bits, gradients of x among them."""
    x, w, b, dy = inputs((40000 if D < 512 else 3000, D), "both", BF16, D)

    def run(n):
        leaf = x[:n].clone().requires_grad_()
        y = layer_norm(leaf, w, b)
        return y.detach(), torch.autograd.grad(y, [leaf], dy[:n])[0]

    every = run(len(x))
    for n in (1, 7, 300):
        assert all(torch.equal(a[:n], c) for a, c in zip(every, run(n)))


def test_heads_that_fill_no_block():
    for H, D in ((3, 16), (5, 128), (17, 64), (33, 8), (2, 600), (70, 24)):
        check(*inputs((3, 11, H, D), "both", F32, H, heads=True))
        check(*inputs((2, 400, H, D), "both", BF16, H, heads=True))


def test_not_finite_rows_stay_their_own():
    x, w, b, dy = inputs((70, 96), "both", BF16, 9)
    want = layer_norm(x, w, b)
    for bad in (float("nan"), float("inf"), -float("inf")):
        z = x.clone()
        z[13, 5] = bad
        leaf = z.requires_grad_()
        y = layer_norm(leaf, w, b)
        dx, = torch.autograd.grad(y, [leaf], dy)
        rest = torch.arange(70, device=DEV) != 13
        assert torch.equal(y[rest], want[rest]) and y[13].isnan().all() and dx[13].isnan().all() and dx[rest].isfinite().all()


def test_no_rows():
    for shape, heads in (((0, 8), False), ((3, 0, 8), False), ((0, 4, 8), True), ((2, 0, 8), True)):
        x, w, b, dy = inputs(shape, "both", F32, 1, heads)
        leaves = [t.requires_grad_() for t in (x, w, b)]
        y = layer_norm(*leaves)
        grads = torch.autograd.grad(y, leaves, dy)
        assert y.shape == shape and all(g.shape == t.shape and not g.any() for g, t in zip(grads, leaves))


@pytest.mark.parametrize("shape", [(2, 3, 0, 4, 8), (0, 2, 3, 4, 8), (2, 2, 3, 4, 0, 8)], ids=str)
def test_no_rows_of_many_axes(shape):
    x, w, b, dy = inputs(shape, "both", F32, 1)
    leaves = [t.requires_grad_() for t in (x, w, b)]
    y = layer_norm(*leaves)
    grads = torch.autograd.grad(y, leaves, dy)
    assert y.shape == shape and all(g.shape == t.shape and not g.any() for g, t in zip(grads, leaves))


def test_some_gradients_alone():
    x, w, b, dy = inputs((40, 200), "both", F32, 10)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    every = torch.autograd.grad(layer_norm(*leaves), leaves, dy)
    for i in range(3):
        some = [t.clone().requires_grad_(j == i) for j, t in enumerate((x, w, b))]
        got, = torch.autograd.grad(layer_norm(*some), [some[i]], dy)
        assert torch.allclose(got, every[i], rtol=1e-5, atol=1e-6)


def test_gradients_against_differences():
    x, w, b, dy = inputs((11, 50), "both", F32, 11)
    gen = torch.Generator(device=DEV).manual_seed(1)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    loss = lambda *a: (layer_norm(*a, eps=0.1).double() * dy).sum()
    grads = torch.autograd.grad(loss(*leaves), leaves)
    for i, g in enumerate(grads):
        d, h = randn(gen, g.shape), 1e-2
        at = (x, w, b)
        up, down = (loss(*[t + s * h * d if j == i else t for j, t in enumerate(at)]) for s in (1, -1))
        want, got = float((up - down) / (2 * h)), float((g.double() * d.double()).sum())
        # h^2 of the third derivative, and float32 outputs' 2^-24 over h
        assert abs(got - want) <= 5e-3 * (abs(want) + float((g * d).norm())), (i, got, want)


def test_streams_graphs_and_bits():
    x, w, b, dy = inputs((2, 700, 4, 64), "both", BF16, 12, heads=True)

    def call(**kw):
        y, stats = capi.lnm_fwd(x, w, b, want_stats=True, **kw)
        return (y, *capi.lnm_bwd(x, w, b, stats, dy, **kw))

    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, here = call(stream=side), call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(here, want))
    graphs, outs = [], []
    for _ in range(2):
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


def test_beyond_2_to_the_31_elements():
    gen = torch.Generator(device=DEV).manual_seed(13)
    rows = 2 ** 31 // 4096 + 3
    x = torch.zeros(rows, 4096, device=DEV, dtype=BF16)
    tail = randn(gen, (5, 4096), BF16)
    x[-5:] = tail
    w = (1 + 0.1 * randn(gen, (4096,))).to(BF16)
    y = layer_norm(x, w)
    assert torch.equal(y[-5:], layer_norm(tail, w)) and not y[:-5].any()
    del y
    dy = torch.zeros_like(x)
    dy[-5:] = tail.flip(0)
    lx, lw = x.requires_grad_(), w.clone().requires_grad_()
    dx, dw = torch.autograd.grad(layer_norm(lx, lw), [lx, lw], dy)
    tx, tw = tail.clone().requires_grad_(), w.clone().requires_grad_()
    sx, sw = torch.autograd.grad(layer_norm(tx, tw), [tx, tw], tail.flip(0))
    assert torch.equal(dx[-5:], sx) and not dx[:-5].any()
    assert torch.allclose(dw.float(), sw.float(), rtol=2 ** -8, atol=1e-5)      # the same five rows, joined in another order


def test_refusals():
    x, w, b, dy = inputs((6, 4, 32), "both", BF16, 14)
    for args in ((x, w[:-1]), (x, w.float()), (x, None, b.to(F16)), (x, w.cpu()), (x.double(),), (x.int(),), (x, torch.zeros(3, 32, device=DEV, dtype=BF16)),
                 (x, w, torch.zeros(4, 32, device=DEV, dtype=BF16)), (x[0, 0], torch.zeros(1, 32, device=DEV, dtype=BF16)), (x, w[None, None]),
                 (torch.zeros(2, 16385, device=DEV),), (torch.zeros(2, 0, device=DEV),), (x.cpu(),)):
        with pytest.raises((ValueError, TypeError)):
            layer_norm(*args)
    for eps in (-1.0, float("nan")):
        with pytest.raises(ValueError):
            layer_norm(x, w, eps=eps)
    stats = capi.lnm_fwd(x, w, want_stats=True)[1]
    for bad in (stats[:-1], stats.half()):
        with pytest.raises(ValueError):
            capi.lnm_bwd(x, w, None, bad, dy)
    with pytest.raises(ValueError):
        capi.lnm_fwd(x, w, out=x[:3])
    with pytest.raises(capi.QuatCumprodError):
        capi.lnm_fwd(x, w, out=x)
    with pytest.raises(RuntimeError):                         # the gradient's own gradient
        leaf = x.clone().requires_grad_()
        d, = torch.autograd.grad(layer_norm(leaf, w).float().sum(), [leaf], create_graph=True)
        d.sum().backward()
    out = torch.zeros_like(x)
    version = out._version
    capi.lnm_fwd(x, w, out=out)
    assert out._version > version
