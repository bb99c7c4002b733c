"""Memory that the language-model operators may not touch, and sizes whose offsets need 64 bits (needs an MI355X)."""
import numpy as np
import pytest
import torch

from oracle import lm_ops as ref
from quaternion_cumprod_autodiff_amd import capi, gated_delta_step
from test_gpu_lm_ops import check_norm, close, f64, norm_inputs, randn, unit

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


# ------------------------------------------------------------------ nothing beside the tensors is written

class Arena:
    """Tensors inside one buffer, between bands that hold a pattern."""
    BAND = 1 << 16

    def __init__(self, nbytes):
        self.buf = torch.full((nbytes,), 0xA5, dtype=torch.uint8, device=DEV)
        self.at, self.used = self.BAND, []

    def new(self, nbytes):
        start = self.at
        self.used.append((start, start + nbytes))
        self.at = (start + nbytes + 255) // 256 * 256 + self.BAND
        assert self.at <= self.buf.numel()
        return self.buf.data_ptr() + start

    def put(self, t):
        p = self.new(t.numel() * t.element_size())
        lo, hi = self.used[-1]
        self.buf[lo:hi].copy_(t.contiguous().view(-1).view(torch.uint8))
        return p

    def bands_whole(self):
        edges = [0] + [x for lo, hi in self.used for x in (lo, hi)] + [self.buf.numel()]
        return all(bool((self.buf[a:b] == 0xA5).all()) for a, b in zip(edges[::2], edges[1::2]))


def offset_lists():
    rng = np.random.default_rng(4)
    top = 2 ** 31 - 1
    fixed = [[0, 150, 100, 50], [-5, 70, 90, 150], [0, 70, 90, 10 ** 9], [150, 100, 50, 0], [top] * 4, [-top - 1] * 4, [-top - 1, top, -top - 1, top],
             [top, -top - 1, top, 0], [0, 0, 0, 150], [149, 150, 151, 152], [0, 150, 0, 150], [64, 128, 64, 128]]
    return fixed + [rng.integers(-40, 200, 4).tolist() for _ in range(12)]


@pytest.mark.parametrize("K,V,Hk,Hv,dtype", [(32, 16, 1, 2, BF16), (128, 40, 2, 2, F32), (50, 100, 1, 3, F16)], ids=str)
def test_no_offsets_reach_beyond_the_tensors(K, V, Hk, Hv, dtype):
    """The kernels clamp offsets and take every slot of their buffers from the clamped ones: whatever they hold, only
    the outputs, the saved state and the workspace are written."""
    gen = torch.Generator(device=DEV).manual_seed(K)
    T, N = 150, 3
    lib, e = capi.load(), torch.finfo(dtype).bits // 8
    q, k, v = unit(gen, (1, T, Hk, K), dtype), unit(gen, (1, T, Hk, K), dtype), randn(gen, (1, T, Hv, V), dtype)
    g, b = -torch.rand(1, T, Hv, generator=gen, device=DEV), torch.rand(1, T, Hv, generator=gen, device=DEV)
    s, d_out, d_fin = randn(gen, (N, Hv, K, V)), randn(gen, (1, T, Hv, V), dtype), randn(gen, (N, Hv, K, V))
    d = capi.GdrDims(1, T, Hk, Hv, K, V, N)
    for st, t in ((d.q_stride, q), (d.k_stride, k), (d.v_stride, v)):
        st[:] = t.stride()[:3]
    d.dtype, d.scale, d.packed = capi._LM_DTYPES[dtype], 0.5, 1
    stream = torch.cuda.current_stream().cuda_stream
    sizes = [lib.gdr_saved_bytes(d), lib.gdr_workspace_bytes(d, 0), lib.gdr_workspace_bytes(d, 1)]
    for offsets in offset_lists():
        print(f"[offsets {offsets}]", flush=True)
        inputs = [q, k, v, g, b, torch.tensor(offsets, dtype=torch.int32, device=DEV), s, d_out, d_fin]
        arena = Arena(sum(sizes) + 64 * Arena.BAND + 4 * sum(t.numel() * 4 for t in inputs))
        p = [arena.put(t) for t in inputs]
        out, fin, saved, ws, ws2 = (arena.new(n) for n in (T * Hv * V * e, N * Hv * K * V * 4, *sizes))
        grads = [arena.new(n) for n in (T * Hk * K * e, T * Hk * K * e, T * Hv * V * e, T * Hv * 4, T * Hv * 4, N * Hv * K * V * 4)]
        assert lib.gdr_fwd(d, *p[:6], p[6], out, fin, saved, ws, sizes[1], stream) == 0
        assert lib.gdr_bwd(d, *p[:6], saved, p[7], p[8], *grads, ws2, sizes[2], stream) == 0
        torch.cuda.synchronize()
        assert arena.bands_whole(), offsets
        for t, (lo, hi) in zip(inputs, arena.used):
            assert torch.equal(arena.buf[lo:hi], t.contiguous().view(-1).view(torch.uint8)), offsets


# ------------------------------------------------------------------ repeated slots, far rows

def test_step_skips_rows_of_a_slot_named_far_before():
    """Rows are looked through 64 at a time: repeats on both sides of that, of the first row, of a padding row."""
    gen = torch.Generator(device=DEV).manual_seed(6)
    B, Hk, Hv, K, V, n_slots = 211, 1, 2, 24, 20, 190
    q, k, v = unit(gen, (B, 1, Hk, K), BF16), unit(gen, (B, 1, Hk, K), BF16), randn(gen, (B, 1, Hv, V), BF16)
    g, b = -torch.rand(B, 1, Hv, generator=gen, device=DEV), torch.rand(B, 1, Hv, generator=gen, device=DEV)
    state = randn(gen, (n_slots, Hv, K, V))
    slots = torch.randperm(n_slots, generator=gen, device=DEV).to(torch.int32).cpu()
    slots = torch.cat([slots, slots[:21]])                            # rows 190.. repeat rows 0..20
    slots[[64, 65, 128, 129, 200]] = slots[[0, 1, 63, 64, 199]]
    slots[[70, 150]] = -1
    seen, run = set(), []
    for i, x in enumerate(slots.tolist()):
        if x >= 0 and x not in seen:
            run.append(i)
        seen.add(x)
    before, at = state.clone(), slots[run].long()
    out = gated_delta_step(q, k, v, g, b, state, slots=slots.to(DEV))
    want, fin = ref.gdr_fwd(*(f64(x)[run] for x in (q, k, v, g, b)), f64(before)[at.numpy()], K ** -0.5)
    close("out", out[run], want)
    close("state", state[at.to(DEV)], fin)
    rest = sorted(set(range(B)) - set(run))
    assert len(rest) >= 26 and not out[rest].any()
    untouched = sorted(set(range(n_slots)) - set(at.tolist()))
    assert torch.equal(state[untouched], before[untouched])


# ------------------------------------------------------------------ four heads in a row

@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("kind,interleaved", [("rms", False), ("rms", True), ("l2", False), ("l2", True)])
@pytest.mark.parametrize("size", [(1, 1700, 3, 2, 90, 42, 300), (1, 9400, 5, 2, 128, 64, 300), (2, 4100, 4, 4, 128, 128, 50), (3, 3001, 1, 3, 240, 16, 9)],
                         ids=str)
def test_norm_of_many_heads(size, kind, interleaved, dtype):
    """Calls of so many heads that a group takes four of a token in a row, in every type, kind and order of pairs."""
    print(f"[norm {size} {kind} {interleaved} {dtype}]", flush=True)
    check_norm(*norm_inputs(*size, dtype, kind == "rms", seed=size[1]), kind=kind, interleaved=interleaved)


# ------------------------------------------------------------------ offsets beyond 2^31 elements

@pytest.fixture
def much_memory():
    yield
    torch.cuda.empty_cache()


def test_step_on_a_pool_of_more_than_2_to_the_31_elements(much_memory):
    gen = torch.Generator(device=DEV).manual_seed(7)
    B, Hk, Hv, K, V, n_slots = 5, 2, 32, 128, 128, 4200
    q, k, v = unit(gen, (B, 2, Hk, K), BF16), unit(gen, (B, 2, Hk, K), BF16), randn(gen, (B, 2, Hv, V), BF16)
    g, b = -torch.rand(B, 2, Hv, generator=gen, device=DEV), torch.rand(B, 2, Hv, generator=gen, device=DEV)
    pool = torch.full((n_slots, Hv, K, V), 3.0, device=DEV)
    slots = torch.tensor([4199, 0, 4096, 4095, 2048], dtype=torch.int32, device=DEV)
    near = randn(gen, (B, Hv, K, V))
    pool[slots.long()] = near
    out = gated_delta_step(q, k, v, g, b, pool, slots=slots)
    want = gated_delta_step(q, k, v, g, b, near)
    assert torch.equal(out, want) and torch.equal(pool[slots.long()], near)
    for n in (1, 2047, 2049, 4094, 4097, 4198):
        assert (pool[n] == 3.0).all()


def test_rule_of_more_than_2_to_the_31_elements(much_memory):
    """A training step of 65 sequences of 8192 tokens of 32 heads of 128, against some of its sequences alone, bit for bit."""
    gen = torch.Generator(device=DEV).manual_seed(8)
    B, T, H, K, V = 65, 8192, 32, 128, 128
    new = lambda *s: torch.empty(s, dtype=BF16, device=DEV).normal_(generator=gen)
    q, k, v, d_out = new(B, T, H, K).mul_(K ** -0.5), new(B, T, H, K).mul_(K ** -0.5), new(B, T, H, V), new(B, T, H, V)
    g, b = -torch.rand(B, T, H, generator=gen, device=DEV), torch.rand(B, T, H, generator=gen, device=DEV)
    s, d_fin = randn(gen, (B, H, K, V)), randn(gen, (B, H, K, V))
    assert v.numel() > 2 ** 31
    out, state, saved = capi.gdr_fwd(q, k, v, g, b, s, want_saved=True)
    grads = capi.gdr_bwd(q, k, v, g, b, saved, d_out, d_fin)
    del saved
    for n in (0, 31, 63, 64):
        one = [t[n:n + 1] for t in (q, k, v, g, b, s)]
        o, st, sv = capi.gdr_fwd(*one, want_saved=True)
        gr = capi.gdr_bwd(*one[:5], sv, d_out[n:n + 1], d_fin[n:n + 1])
        for name, x, y in zip(("out", "state", "query", "key", "value", "log_decay", "beta", "initial"), (out, state, *grads), (o, st, *gr)):
            assert torch.equal(x[n:n + 1], y), (n, name)


def test_norm_of_more_than_2_to_the_31_heads_and_elements(much_memory):
    """Numbers of heads beyond 31 bits (64-bit divisions) on more blocks than a launch has, and offsets beyond 2^31."""
    gen = torch.Generator(device=DEV).manual_seed(9)
    B, T, Hq, Hk, D = 2, 179_000_003, 5, 1, 2
    new = lambda *s: torch.empty(s, dtype=BF16, device=DEV).normal_(generator=gen)
    q, k = new(B, T, Hq, D), new(B, T, Hk, D)
    assert B * T * (Hq + Hk) >= 2 ** 31 and q.numel() > 2 ** 31
    angle = randn(gen, (1000, 1))
    pos = torch.randint(0, 1000, (B, T), generator=gen, device=DEV, dtype=torch.int32)
    w = randn(gen, (D,), BF16)
    cuts = [(0, 0), (0, T // 2), (0, T - 300), (1, 0), (1, 2 ** 31 // (Hq * D) - T - 150), (1, T - 300)]
    qo, ko = capi.qkn_fwd(q, k, w, None, angle.cos(), angle.sin(), pos)
    how = lambda b, c: (f64(angle.cos()), f64(angle.sin()), pos[b:b + 1, c].cpu().numpy(), "rms", 1e-6, False)
    for b, t in cuts:
        c = slice(t, t + 300)
        close(f"query {b} {t}", qo[b:b + 1, c], ref.qkn_fwd(f64(q[b:b + 1, c]), f64(w), *how(b, c)))
        close(f"key {b} {t}", ko[b:b + 1, c], ref.qkn_fwd(f64(k[b:b + 1, c]), None, *how(b, c)))
    dq, dk, _, _ = capi.qkn_bwd(q, k, w, None, angle.cos(), angle.sin(), pos, qo, ko, want=(True, True, False, False))
    for b, t in cuts:
        c = slice(t, t + 300)
        for name, got, x, wt, dy in (("query", dq, q, w, qo), ("key", dk, k, None, ko)):
            x, dy, wt = f64(x[b:b + 1, c]), f64(dy[b:b + 1, c]), None if wt is None else f64(wt)
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
            # the gradient's two terms cancel: the bound is of the largest of them (see the norm's other tests)
            top = float((2 * r * np.abs(dy).max(-1, keepdims=True) * (1 if wt is None else np.abs(wt).max())).max())
            close(f"gradient of {name} {b} {t}", got[b:b + 1, c], ref.qkn_bwd(x, wt, *how(b, c), dy)[0], top=top)
