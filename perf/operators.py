"""The gated-delta-rule operators as measured cases: inputs, plain forms, values in 64 bits, and work.

Three operators that a linear-attention language model runs next to the gated delta recurrences of this framework:

  rule   out, state = gated_delta_rule(...): a whole sequence, a padded batch or packed sequences (prefill), and its
         gradients (training).  Per value head h, with key head h // (Hv / Hk) and a state S [K, V]:
             S = exp(g_t) S;   u = b_t (v_t - S^T k_t);   S = S + k_t u^T;   out_t = scale S^T q_t
  step   the same recurrence for one or a few new tokens per sequence, on a pool of states updated in place (decoding)
  norm   the norm of every query and key head (root mean square or Euclidean) with the position rotation of its first
         `rotary` elements, and its gradients

`own` false: elementary torch operations in 32 bits (cumulated decays in 64), rounded once at the end.
`own` true: the framework's calls.
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"
CHUNK = 64  # tokens to a chunk of the plain form of `rule`


# ------------------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # One user's next token in a layer with shared key heads: latency alone counts.
        {"name": "step_single", "op": "step", "dtype": "bf16", "n": 1, "tokens": 1, "hk": 16, "hv": 32, "k": 128, "v": 128, "pool": 16},
        # A full decoding batch: every state is read and written once.
        {"name": "step_batch", "op": "step", "dtype": "bf16", "n": 192, "tokens": 1, "hk": 16, "hv": 32, "k": 128, "v": 128, "pool": 200},
        # A few drafted tokens per sequence, odd head sizes, 16-bit floats of the other kind.
        {"name": "step_draft_odd", "op": "step", "dtype": "fp16", "n": 33, "tokens": 5, "hk": 3, "hv": 6, "k": 72, "v": 100, "pool": 40},
        # One long prompt.
        {"name": "rule_prompt", "op": "rule", "dtype": "bf16", "batch": 1, "t": 8192, "seqs": 0, "hk": 16, "hv": 32, "k": 128, "v": 128, "train": False},
        # Prompts of many lengths packed one after another (an empty one and a single token among them).
        {"name": "rule_packed", "op": "rule", "dtype": "bf16", "batch": 1, "t": 12001, "seqs": 29, "hk": 8, "hv": 16, "k": 128, "v": 128, "train": False},
        # The sizes of this repository's own recurrence benchmark, in its 32 bits.
        {"name": "rule_train_fp32", "op": "rule", "dtype": "fp32", "batch": 8, "t": 2048, "seqs": 0, "hk": 16, "hv": 16, "k": 64, "v": 128, "train": True},
        # A training step's layer.
        {"name": "rule_train", "op": "rule", "dtype": "bf16", "batch": 4, "t": 4096, "seqs": 0, "hk": 16, "hv": 32, "k": 128, "v": 128, "train": True},
        # A small odd one: ragged last chunk, heads that fill no tile, packed sequences, gradients.
        {"name": "rule_train_odd", "op": "rule", "dtype": "fp16", "batch": 1, "t": 777, "seqs": 5, "hk": 2, "hv": 6, "k": 40, "v": 72, "train": True},
        # A decoding batch's queries and keys, rotated in their first half by positions of a long context.
        {"name": "norm_decode", "op": "norm", "dtype": "bf16", "batch": 64, "t": 1, "hq": 16, "hk": 2, "d": 128, "rotary": 64, "table": 131072, "kind": "rms", "interleaved": False, "weights": True, "train": False},
        # A prompt's queries and keys.
        {"name": "norm_prompt", "op": "norm", "dtype": "bf16", "batch": 1, "t": 16384, "hq": 32, "hk": 8, "d": 128, "rotary": 128, "table": 32768, "kind": "rms", "interleaved": False, "weights": True, "train": False},
        # A training step's.
        {"name": "norm_train", "op": "norm", "dtype": "bf16", "batch": 4, "t": 4096, "hq": 16, "hk": 16, "d": 128, "rotary": 128, "table": 4096, "kind": "rms", "interleaved": False, "weights": True, "train": True},
        # Unit keys and queries for the recurrence, odd sizes, neighbouring pairs, 32 bits.
        {"name": "norm_train_odd", "op": "norm", "dtype": "fp32", "batch": 3, "t": 1001, "hq": 5, "hk": 3, "d": 90, "rotary": 42, "table": 2048, "kind": "l2", "interleaved": True, "weights": False, "train": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["step", "rule", "rule", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "step":
        hk = _log(rng, 1, 16)
        n = _log(rng, 1, 128)
        return {"op": op, "dtype": dtype, "n": n, "tokens": rng.choice([1, 1, 1, 2, 4, 7]), "hk": hk, "hv": hk * rng.choice([1, 2, 4]) if hk <= 8 else hk,
                "k": rng.choice([64, 128, 128, _log(rng, 8, 128)]), "v": rng.choice([64, 128, 128, _log(rng, 8, 192)]), "pool": n + _log(rng, 1, 64)}
    if op == "rule":
        train = rng.random() < 0.5
        hk = _log(rng, 1, 16)
        hv = hk * rng.choice([1, 2, 3])
        batch = rng.choice([1, 1, 2, 5])
        seqs = rng.choice([0, _log(rng, 1, 40)]) if batch == 1 else 0
        t = _log(rng, 1, max(64, min(12000, (100000 if train else 200000) // (batch * hv))))
        return {"op": op, "dtype": dtype, "batch": batch, "t": max(t, seqs), "seqs": seqs, "hk": hk, "hv": hv,
                "k": rng.choice([64, 128, 128, _log(rng, 4, 128)]), "v": rng.choice([64, 128, 128, _log(rng, 4, 160)]), "train": train}
    d = rng.choice([64, 128, 128, 256, 2 * _log(rng, 8, 160)])
    rotary = rng.choice([0, d, d, 2 * (d // 4), 2 * rng.randint(1, d // 2)])
    batch = rng.choice([1, 1, 2, 8])
    return {"op": op, "dtype": dtype, "batch": batch, "t": _log(rng, 1, 8192 // batch), "hq": _log(rng, 1, 32), "hk": _log(rng, 1, 8), "d": d, "rotary": rotary,
            "table": _log(rng, 512, 65536), "kind": rng.choice(["rms", "rms", "l2"]), "interleaved": rng.random() < 0.3, "weights": rng.random() < 0.7, "train": rng.random() < 0.5}


def lengths(case):
    """The packed sequences' lengths: of the case alone.  Some short, some long, one empty and one single where there are four or more."""
    n, t = case["seqs"], case["t"]
    rng = random.Random(n * 100003 + t)
    share = [rng.random() ** 3 + 0.02 for _ in range(n)]
    if n >= 4:
        share[n // 2] = 0.0
    lens = [int(t * x / sum(share)) for x in share]
    if n >= 4:
        lens[1] = 1
    lens[0] += t - sum(lens)
    return lens


# ----------------------------------------------------------------------------------------------------- the inputs

def _randn(shape, gen, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _unit(shape, gen, dtype):
    x = _randn(shape, gen)
    return (x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-12)).to(dtype)


def _gates(shape, gen):
    """Decays as layers have them: a rate per head from slow to fast, times a softplus of the token; write strengths in (0, 1)."""
    rate = torch.exp(torch.linspace(-4.0, 1.0, shape[-1], device=DEV))
    x = _randn(shape, gen)
    g = -rate * torch.log1p(torch.exp(x))
    return g, torch.sigmoid(_randn(shape, gen))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 1000003 + 17)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "step":
        n, t = case["n"], case["tokens"]
        s["query"] = _unit((n, t, case["hk"], case["k"]), gen, dt)
        s["key"] = _unit((n, t, case["hk"], case["k"]), gen, dt)
        s["value"] = _randn((n, t, case["hv"], case["v"]), gen, dt)
        s["log_decay"], s["beta"] = _gates((n, t, case["hv"]), gen)
        s["state"] = _randn((case["pool"], case["hv"], case["k"], case["v"]), gen).mul_(0.3)
        s["slots"] = torch.randperm(case["pool"], generator=gen, device=DEV)[:n].to(torch.int32)
    elif case["op"] == "rule":
        b, t = case["batch"], case["t"]
        n = case["seqs"] or b
        s["query"] = _unit((b, t, case["hk"], case["k"]), gen, dt)
        s["key"] = _unit((b, t, case["hk"], case["k"]), gen, dt)
        s["value"] = _randn((b, t, case["hv"], case["v"]), gen, dt)
        s["log_decay"], s["beta"] = _gates((b, t, case["hv"]), gen)
        s["state"] = _randn((n, case["hv"], case["k"], case["v"]), gen).mul_(0.3)
        s["offsets"] = s["lens"] = None
        if case["seqs"]:
            s["lens"] = lengths(case)
            s["offsets"] = torch.tensor([sum(s["lens"][:i]) for i in range(n + 1)], dtype=torch.int32, device=DEV)
        if case["train"]:
            s["d_out"] = _randn((b, t, case["hv"], case["v"]), gen, dt)
            s["d_state"] = _randn((n, case["hv"], case["k"], case["v"]), gen).mul_(0.1)
            s["leaves"] = [s[x].requires_grad_() for x in ("query", "key", "value", "log_decay", "beta", "state")]
    else:
        b, t, d, r = case["batch"], case["t"], case["d"], case["rotary"]
        # Views of one fused projection's rows, as a layer has them.
        rows = _randn((b, t, (case["hq"] + case["hk"]) * d), gen, dt).mul_(1.7)
        s["query"] = rows[..., : case["hq"] * d].unflatten(-1, (case["hq"], d))
        s["key"] = rows[..., case["hq"] * d:].unflatten(-1, (case["hk"], d))
        s["query_weight"] = s["key_weight"] = s["cos"] = s["sin"] = s["positions"] = None
        if case["weights"]:
            s["query_weight"] = (1 + 0.1 * _randn((d,), gen)).to(dt)
            s["key_weight"] = (1 + 0.1 * _randn((d,), gen)).to(dt)
        if r:
            at = torch.arange(case["table"], device=DEV, dtype=torch.float64)
            angle = at[:, None] * 10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
            s["positions"] = torch.randint(0, case["table"], (b, t), generator=gen, device=DEV, dtype=torch.int32)
        if case["train"]:
            s["d_query"] = _randn((b, t, case["hq"], d), gen, dt)
            s["d_key"] = _randn((b, t, case["hk"], d), gen, dt)
            names = ("query", "key") + (("query_weight", "key_weight") if case["weights"] else ())
            s["query"], s["key"] = s["query"].detach(), s["key"].detach()
            s["leaves"] = [s[x].requires_grad_() for x in names]
    return s


# ------------------------------------------------------------------------------------------------ the plain forms

def _pad_packed(x, lens):
    """[1, total, ...] to [sequences, longest, ...], zeros behind each sequence's end; and the rows' places."""
    longest = max(lens)
    where = torch.tensor([sum(lens[:i]) for i in range(len(lens))], device=x.device)[:, None] + torch.arange(longest, device=x.device)
    inside = torch.arange(longest, device=x.device) < torch.tensor(lens, device=x.device)[:, None]
    rows = x[0][where.clamp_max(x.shape[1] - 1)]
    return torch.where(inside.reshape(inside.shape + (1,) * (x.dim() - 2)), rows, torch.zeros_like(rows)), inside


def _plain_rule(q, k, v, g, b, state, scale, lens):
    """The recurrence over chunks of 64 tokens: within a chunk the updates solve a unit lower triangular system, whose
    inverse is built from its blocks; only the states pass from chunk to chunk."""
    out_type = v.dtype
    q, k, v, g, b = (x.float() for x in (q, k, v, g, b))
    inside = None
    if lens is not None:
        q, k, v, g = (_pad_packed(x, lens)[0] for x in (q, k, v, g))
        b, inside = _pad_packed(b, lens)
    n, t, hv = g.shape
    group = hv // q.shape[2]
    c = CHUNK
    nc = -(-t // c)
    more = nc * c - t

    def chunks(x):  # [n, t, h, w] to [n, h, nc, c, w]
        x = torch.cat([x, x.new_zeros((n, more) + x.shape[2:])], 1)
        return x.unflatten(1, (nc, c)).permute(0, 3, 1, 2, 4)

    q, k = (chunks(x.repeat_interleave(group, 2)) for x in (q, k))
    v = chunks(v)
    g, b = chunks(g[..., None])[..., 0], chunks(b[..., None])
    cum = g.double().cumsum(-1)
    lower = torch.ones(c, c, device=q.device, dtype=torch.bool).tril()
    gap = torch.where(lower, cum[..., :, None] - cum[..., None, :], torch.zeros((), device=q.device, dtype=torch.float64)).float()
    decay = torch.where(lower, gap.exp(), torch.zeros((), device=q.device))
    head, tail = cum.float().exp()[..., None], (cum[..., -1:] - cum).float().exp()[..., None]
    whole = cum[..., -1].float().exp()[..., None, None]
    kt = k.transpose(-1, -2).contiguous()
    a = (b * decay * (k @ kt)).tril(-1)
    inv = torch.eye(c, device=q.device).expand_as(a)
    at = torch.arange(c, device=q.device)
    for level in range(6):  # blocks of 1, 2, ..., 32 rows join in pairs
        pair = ((at[:, None] >> level) == (at[None, :] >> level) + 1) & ((at[:, None] >> level) % 2 == 1)
        inv = inv - inv @ ((a * pair) @ inv)
    inv = inv * b.transpose(-1, -2)
    p = (decay * (q @ kt)) * scale
    qh, kh, ke = q * head * scale, k * head, (k * tail).transpose(-1, -2)
    s, outs = state.float(), []
    for i in range(nc):
        d = inv[:, :, i] @ (v[:, :, i] - kh[:, :, i] @ s)
        outs.append(qh[:, :, i] @ s + p[:, :, i] @ d)
        s = whole[:, :, i] * s + ke[:, :, i] @ d
    out = torch.cat(outs, 2)[:, :, :t].transpose(1, 2)
    if inside is not None:
        out = out[inside][None]
    return out.to(out_type), s


def _plain_step(q, k, v, g, b, pool, slots, scale):
    group = v.shape[2] // q.shape[2]
    rows = slots.long()
    s = pool[rows]
    outs = []
    qf, kf, vf = q.float().repeat_interleave(group, 2), k.float().repeat_interleave(group, 2), v.float()
    for t in range(q.shape[1]):
        kt, qt = kf[:, t, :, :, None], qf[:, t, :, :, None]
        s = s * g[:, t].exp()[..., None, None]
        u = b[:, t, :, None] * (vf[:, t] - (s * kt).sum(2))
        s = s + kt * u[:, :, None, :]
        outs.append((s * qt).sum(2) * scale)
    pool[rows] = s
    return torch.stack(outs, 1).to(v.dtype)


def _plain_norm(x, w, cos, sin, positions, kind, eps, interleaved):
    y = x.float()
    sq = y.square().sum(-1, keepdim=True)
    y = y * torch.rsqrt(sq / x.shape[-1] + eps if kind == "rms" else sq + eps)
    if w is not None:
        y = y * w.float()
    if cos is not None:
        r = 2 * cos.shape[-1]
        c, s = (z[positions.long()][:, :, None, :] for z in (cos, sin))
        a, b = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., : r // 2], y[..., r // 2: r])
        a, b = a * c - b * s, b * c + a * s
        turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
        y = torch.cat([turned, y[..., r:]], -1)
    return y.to(x.dtype)


EPS = 1e-6


def run(s):
    case = s["case"]
    if case["op"] == "step":
        if own:
            from quaternion_cumprod_autodiff_amd import gated_delta_step
            out = gated_delta_step(s["query"], s["key"], s["value"], s["log_decay"], s["beta"], s["state"], slots=s["slots"])
        else:
            out = _plain_step(s["query"], s["key"], s["value"], s["log_decay"], s["beta"], s["state"], s["slots"], case["k"] ** -0.5)
        return {"out": out, "state": s["state"]}
    if case["op"] == "rule":
        args = [s[x] for x in ("query", "key", "value", "log_decay", "beta", "state")]
        if own:
            from quaternion_cumprod_autodiff_amd import gated_delta_rule
            out, state = gated_delta_rule(*args, offsets=s["offsets"])
        else:
            out, state = _plain_rule(*args, case["k"] ** -0.5, s["lens"])
        got = {"out": out, "state": state}
        if case["train"]:
            got["grads"] = list(torch.autograd.grad([out, state], s["leaves"], [s["d_out"], s["d_state"]]))
        return got
    if own:
        from quaternion_cumprod_autodiff_amd import qk_norm_rotate
        q, k = qk_norm_rotate(s["query"], s["key"], s["query_weight"], s["key_weight"], s["cos"], s["sin"], s["positions"],
                              kind=case["kind"], eps=EPS, interleaved=case["interleaved"])
    else:
        how = (s["cos"], s["sin"], s["positions"], case["kind"], EPS, case["interleaved"])
        q, k = _plain_norm(s["query"], s["query_weight"], *how), _plain_norm(s["key"], s["key_weight"], *how)
    got = {"query": q, "key": k}
    if case["train"]:
        got["grads"] = list(torch.autograd.grad([q, k], s["leaves"], [s["d_query"], s["d_key"]]))
    return got


# ------------------------------------------------------------------------------------------------------- the work

def work(case):
    e = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if case["op"] == "norm":
        rows = case["batch"] * case["t"]
        x = rows * (case["hq"] + case["hk"]) * case["d"] * e
        tables = rows * (4 + 4 * case["rotary"]) if case["rotary"] else 0
        weights = 2 * case["d"] * e if case["weights"] else 0
        # Forward: rows in, rows out.  Gradients: rows and their cotangents in, rows out.
        n = rows * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": (5 if case["train"] else 2) * x + (2 if case["train"] else 1) * tables + (3 if case["train"] else 1) * weights,
                "flops": n * (24 if case["train"] else 8)}
    hk, hv, k, v = case["hk"], case["hv"], case["k"], case["v"]
    tokens = case["n"] * case["tokens"] if case["op"] == "step" else case["batch"] * case["t"]
    n = case["n"] if case["op"] == "step" else case["seqs"] or case["batch"]
    rows = tokens * (2 * hk * k + 2 * hv * v) * e + tokens * hv * 8
    states = 2 * n * hv * k * v * 4
    # A token's recurrence: decay, S^T k, the update, S^T q.  Its gradient reverses each product once for each factor.
    flops = tokens * hv * k * v * 7
    if case["op"] == "rule" and case["train"]:
        # Gradients: q, k, v, gates, initial state and both cotangents in; five gradients and the state's out.
        grads = tokens * (4 * hk * k + 3 * hv * v) * e + tokens * hv * 16 + 3 * n * hv * k * v * 4
        return {"bytes": rows + states + grads, "flops": 3 * flops}
    return {"bytes": rows + states, "flops": flops}


# ------------------------------------------------------------------------------------------------ values in 64 bits

def _exact_rule(s, scale, lens, train):
    q, k, v, g, b = (s[x].detach().double() for x in ("query", "key", "value", "log_decay", "beta"))
    d_out = s["d_out"].double() if train else None
    if lens is not None:
        place = [(i, t) for i, x in enumerate(lens) for t in range(x)]
        seq, pos = (torch.tensor(list(z), device=q.device) for z in zip(*place))

        def spread(x):
            y = x.new_zeros((len(lens), max(lens)) + x.shape[2:])
            y[seq, pos] = x[0]
            return y
        q, k, v, g, b = map(spread, (q, k, v, g, b))
        d_out = spread(d_out) if train else None
    n, T, hv = g.shape
    hk = q.shape[2]
    head = torch.arange(hv, device=q.device) // (hv // hk)
    st = s["state"].detach().double()
    a = g.exp()

    def token(st, t):
        sd = st * a[:, t, :, None, None]
        e = v[:, t] - torch.einsum("nhkv,nhk->nhv", sd, k[:, t][:, head])
        u = b[:, t, :, None] * e
        return sd, e, u, sd + k[:, t][:, head][..., None] * u[:, :, None, :]

    out = torch.zeros_like(v)
    seg = 64
    starts = []
    for t in range(T):
        if t % seg == 0:
            starts.append(st)
        st = token(st, t)[3]
        out[:, t] = scale * torch.einsum("nhkv,nhk->nhv", st, q[:, t][:, head])
    got = {"out": out[seq, pos][None] if lens is not None else out, "state": st}
    if not train:
        return got
    dst = s["d_state"].double()
    dq, dk, dv, dg, db = q.new_zeros((n, T, hv, q.shape[3])), q.new_zeros((n, T, hv, q.shape[3])), torch.zeros_like(v), torch.zeros_like(g), torch.zeros_like(b)
    for j in range(len(starts) - 1, -1, -1):
        st, kept = starts[j], []
        for t in range(j * seg, min(T, j * seg + seg)):
            kept.append(token(st, t))
            st = kept[-1][3]
        for t in range(min(T, j * seg + seg) - 1, j * seg - 1, -1):
            sd, e, u, st = kept[t - j * seg]
            do = scale * d_out[:, t]
            kh = k[:, t][:, head]
            dq[:, t] = torch.einsum("nhkv,nhv->nhk", st, do)
            dst = dst + q[:, t][:, head][..., None] * do[:, :, None, :]
            du = torch.einsum("nhkv,nhk->nhv", dst, kh)
            de = b[:, t, :, None] * du
            db[:, t] = (du * e).sum(-1)
            dv[:, t] = de
            dk[:, t] = torch.einsum("nhkv,nhv->nhk", dst, u) - torch.einsum("nhkv,nhv->nhk", sd, de)
            dst = dst - kh[..., None] * de[:, :, None, :]
            dg[:, t] = (dst * sd).sum((-1, -2))
            dst = dst * a[:, t, :, None, None]
    dq, dk = (x.unflatten(2, (hk, hv // hk)).sum(3) for x in (dq, dk))
    grads = [dq, dk, dv, dg, db]
    if lens is not None:
        grads = [x[seq, pos][None] for x in grads]
    got["grads"] = grads + [dst]
    return got


def _exact_norm(x, w, cos, sin, positions, case, dy):
    """Rotation as a product of complex numbers; the gradient from its formula."""
    x = x.detach().double()
    d = x.shape[-1]
    w = torch.ones(d, device=x.device, dtype=torch.float64) if w is None else w.detach().double()
    size = d if case["kind"] == "rms" else 1
    r = 1 / ((x * x).sum(-1, keepdim=True) / size + EPS).sqrt()

    def turn(y, sign):
        if cos is None:
            return y
        m = cos.shape[-1]
        z = torch.complex(cos.double(), sign * sin.double())[positions.long()][:, :, None, :]
        y = y.clone()
        if case["interleaved"]:
            y[..., : 2 * m] = torch.view_as_real(torch.view_as_complex(y[..., : 2 * m].reshape(y.shape[:-1] + (m, 2)).contiguous()) * z).flatten(-2)
        else:
            p = torch.complex(y[..., :m].contiguous(), y[..., m: 2 * m].contiguous()) * z
            y[..., :m], y[..., m: 2 * m] = p.real, p.imag
        return y

    y = turn(x * r * w, 1.0)
    if dy is None:
        return y, None, None
    dn = turn(dy.double(), -1.0)
    dh = dn * w
    dx = r * dh - x * r ** 3 * ((dh * x).sum(-1, keepdim=True) / size)
    return y, dx, (dn * x * r).sum((0, 1, 2))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rule":
        if case["t"] > 9000 and not case["seqs"]:
            return None
        return _exact_rule(s, case["k"] ** -0.5, s["lens"], case["train"])
    if case["op"] == "step":
        one = dict(s, state=s["state"][s["slots"].long()])
        got = _exact_rule(one, case["k"] ** -0.5, None, False)
        pool = s["state"].double()
        pool[s["slots"].long()] = got["state"]
        return {"out": got["out"], "state": pool}
    q, dq, dwq = _exact_norm(s["query"], s["query_weight"], s["cos"], s["sin"], s["positions"], case, s.get("d_query"))
    k, dk, dwk = _exact_norm(s["key"], s["key_weight"], s["cos"], s["sin"], s["positions"], case, s.get("d_key"))
    got = {"query": q, "key": k}
    if case["train"]:
        got["grads"] = [dq, dk] + ([dwq, dwk] if case["weights"] else [])
    return got
