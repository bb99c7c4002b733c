"""Float64 oracles of the language-model operators, from their definitions:
the gated delta rule token by token (include/gated_delta.h) with the VJP by
reversing it, and the norm and rotation of heads (include/qk_norm.h).  Plain
loops, independent of the chunked form the device runs."""
import numpy as np


def gdr_fwd(q, k, v, g, b, s0, scale, lengths=None):
    """(out, final states).  q, k [B, T, Hk, K], v [B, T, Hv, V]; with lengths
    B is 1 and the rows are packed sequences, one state each; rows behind the
    last are zero in out."""
    out = np.zeros(v.shape)
    fin = np.array(s0, dtype=np.float64)
    group = v.shape[2] // q.shape[2]
    for n, bi, lo, hi in _sequences(v.shape, lengths):
        for h in range(v.shape[2]):
            S = fin[n, h].copy()
            for t in range(lo, hi):
                kt, qt = k[bi, t, h // group], q[bi, t, h // group]
                S = np.exp(g[bi, t, h]) * S
                S = S + np.outer(kt, b[bi, t, h] * (v[bi, t, h] - S.T @ kt))
                out[bi, t, h] = scale * (S.T @ qt)
            fin[n, h] = S
    return out, fin


def gdr_bwd(q, k, v, g, b, s0, scale, d_out, d_fin, lengths=None):
    """Gradients (q, k, v, g, b, s0) for the cotangents of out and the final states."""
    dq, dk, dv, dg, db = (np.zeros(x.shape) for x in (q, k, v, g, b))
    ds0 = np.zeros(s0.shape)
    group = v.shape[2] // q.shape[2]
    for n, bi, lo, hi in _sequences(v.shape, lengths):
        for h in range(v.shape[2]):
            kept, S = [], np.array(s0[n, h], dtype=np.float64)
            for t in range(lo, hi):
                kt = k[bi, t, h // group]
                decayed = np.exp(g[bi, t, h]) * S
                e = v[bi, t, h] - decayed.T @ kt
                S = decayed + np.outer(kt, b[bi, t, h] * e)
                kept.append((decayed, e, S))
            dS = np.zeros(S.shape) if d_fin is None else np.array(d_fin[n, h], dtype=np.float64)
            for t in range(hi - 1, lo - 1, -1):
                decayed, e, S = kept[t - lo]
                kt, qt, do = k[bi, t, h // group], q[bi, t, h // group], scale * d_out[bi, t, h]
                dq[bi, t, h // group] += S @ do
                dS = dS + np.outer(qt, do)
                du = dS.T @ kt
                de = b[bi, t, h] * du
                db[bi, t, h] = du @ e
                dv[bi, t, h] = de
                dk[bi, t, h // group] += dS @ (b[bi, t, h] * e) - decayed @ de
                dS = dS - np.outer(kt, de)
                dg[bi, t, h] = np.sum(dS * decayed)
                dS = np.exp(g[bi, t, h]) * dS
            ds0[n, h] = dS
    return dq, dk, dv, dg, db, ds0


def _sequences(shape, lengths):
    if lengths is None:
        return [(i, i, 0, shape[1]) for i in range(shape[0])]
    ends = np.cumsum([0] + list(lengths))
    return [(i, 0, int(ends[i]), int(ends[i + 1])) for i in range(len(lengths))]


def _turn(y, cos, sin, rows, interleaved, sign):
    m = cos.shape[1]
    z = (cos + 1j * sign * sin)[rows][:, :, None, :]
    y = y.copy()
    if interleaved:
        p = (y[..., 0:2 * m:2] + 1j * y[..., 1:2 * m:2]) * z
        y[..., 0:2 * m:2], y[..., 1:2 * m:2] = p.real, p.imag
    else:
        p = (y[..., :m] + 1j * y[..., m:2 * m]) * z
        y[..., :m], y[..., m:2 * m] = p.real, p.imag
    return y


def _rows(x, positions):
    return np.broadcast_to(np.arange(x.shape[1]), x.shape[:2]) if positions is None else positions


def qkn_fwd(x, w, cos, sin, positions, kind, eps, interleaved):
    size = x.shape[-1] if kind == "rms" else 1
    y = x / np.sqrt((x * x).sum(-1, keepdims=True) / size + eps)
    if w is not None:
        y = y * w
    return y if cos is None else _turn(y, cos, sin, _rows(x, positions), interleaved, 1.0)


def qkn_bwd(x, w, cos, sin, positions, kind, eps, interleaved, dy):
    """(dx, dw)."""
    size = x.shape[-1] if kind == "rms" else 1
    r = 1 / np.sqrt((x * x).sum(-1, keepdims=True) / size + eps)
    dn = dy if cos is None else _turn(dy, cos, sin, _rows(x, positions), interleaved, -1.0)
    dh = dn if w is None else dn * w
    dx = r * dh - x * r ** 3 * ((dh * x).sum(-1, keepdims=True) / size)
    return dx, (dn * x * r).sum((0, 1, 2))
