"""Float64 oracles of a linear-attention layer's operators, from their
definitions: linear attention with decays token by token
(include/decay_attention.h) with the VJP by reversing it, and layer norm
(include/layer_norm.h).  Plain loops, independent of the chunked form the
device runs."""
import numpy as np

from .lm_ops import _sequences


def _token_decays(g, shape):
    return np.broadcast_to(g, shape[:3]) if np.ndim(g) == 1 else g


def dca_fwd(q, k, v, g, s0, scale, lengths=None):
    """(out, final states).  q, k [B, T, Hk, K], v [B, T, Hv, V], g [B, T, Hv]
    or [Hv]; with lengths B is 1 and the rows are packed sequences, one state
    each; rows behind the last are zero in out."""
    out, fin = np.zeros(v.shape), np.array(s0, dtype=np.float64)
    group, g = v.shape[2] // q.shape[2], _token_decays(g, v.shape)
    for n, bi, lo, hi in _sequences(v.shape, lengths):
        for h in range(v.shape[2]):
            S = fin[n, h].copy()
            for t in range(lo, hi):
                S = np.exp(g[bi, t, h]) * S + np.outer(k[bi, t, h // group], v[bi, t, h])
                out[bi, t, h] = scale * (S.T @ q[bi, t, h // group])
            fin[n, h] = S
    return out, fin


def dca_bwd(q, k, v, g, s0, scale, d_out, d_fin, lengths=None):
    """Gradients (q, k, v, g, s0) for the cotangents of out and the final states."""
    by_head, g = np.ndim(g) == 1, _token_decays(g, v.shape)
    dq, dk, dv, dg = (np.zeros(x.shape) for x in (q, k, v, g))
    ds0 = np.zeros(s0.shape)
    group = v.shape[2] // q.shape[2]
    for n, bi, lo, hi in _sequences(v.shape, lengths):
        for h in range(v.shape[2]):
            kept, S = [], np.array(s0[n, h], dtype=np.float64)
            for t in range(lo, hi):
                decayed = np.exp(g[bi, t, h]) * S
                S = decayed + np.outer(k[bi, t, h // group], v[bi, t, h])
                kept.append((decayed, S))
            dS = np.zeros(S.shape) if d_fin is None else np.array(d_fin[n, h], dtype=np.float64)
            for t in range(hi - 1, lo - 1, -1):
                decayed, S = kept[t - lo]
                do = scale * d_out[bi, t, h]
                dq[bi, t, h // group] += S @ do
                dS = dS + np.outer(q[bi, t, h // group], do)
                dk[bi, t, h // group] += dS @ v[bi, t, h]
                dv[bi, t, h] = dS.T @ k[bi, t, h // group]
                dg[bi, t, h] = np.sum(dS * decayed)
                dS = np.exp(g[bi, t, h]) * dS
            ds0[n, h] = dS
    return dq, dk, dv, dg.sum((0, 1)) if by_head else dg, ds0


def lnm_fwd(x, w, b, eps):
    d = x - x.mean(-1, keepdims=True)
    y = d / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    y = y if w is None else y * w
    return y if b is None else y + b


def lnm_bwd(x, w, eps, dy, by_head=False):
    """(dx, dw, db), dw and db [D], or [H, D] for an x [.., H, D]."""
    d = x - x.mean(-1, keepdims=True)
    r = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    h = d * r
    dh = dy if w is None else dy * w
    dx = r * (dh - dh.mean(-1, keepdims=True) - h * (dh * h).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - (2 if by_head else 1)))
    return dx, (dy * h).sum(axes), dy.sum(axes)
