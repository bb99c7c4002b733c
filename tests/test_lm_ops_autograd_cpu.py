"""What the language-model operators' autograd entries refuse before they reach the library."""
import pytest
import torch
from torch.autograd import forward_ad

from quaternion_cumprod_autodiff_amd import autograd


def case():
    q, v, g, s = torch.zeros(1, 2, 1, 4), torch.zeros(1, 2, 1, 4), torch.zeros(1, 2, 1), torch.zeros(1, 1, 4, 4)
    return {"query": q, "key": q.clone(), "value": v, "log_decay": g, "beta": g.clone()}, s


def dual(t):
    return forward_ad.make_dual(t, torch.ones_like(t))


@pytest.mark.parametrize("tracked", [False, True])
def test_forward_mode_is_refused_and_not_dropped(tracked):
    """A dual tensor does not require a gradient; its tangent may not be lost in silence."""
    args, state = case()
    with forward_ad.dual_level():
        for name in args:
            duals = {n: dual(t) if n == name else t.clone().requires_grad_(tracked) for n, t in args.items()}
            with pytest.raises(NotImplementedError, match="forward"):
                autograd.gated_delta_rule(**duals)
            with pytest.raises(NotImplementedError, match="forward"):
                autograd.gated_delta_step(**duals, state=state)
        with pytest.raises(NotImplementedError, match="forward"):
            autograd.gated_delta_rule(**args, initial_state=dual(state))
        with pytest.raises(NotImplementedError, match="forward"):
            autograd.gated_delta_step(**args, state=dual(state))
        q, k, w, table = args["query"], args["key"], torch.ones(4), torch.zeros(2, 2)
        for call in (dict(query=dual(q), key=k), dict(query=q, key=dual(k)), dict(query=q, key=k, query_weight=dual(w)),
                     dict(query=q, key=k, key_weight=dual(w)), dict(query=q, key=k, cos=dual(table), sin=table),
                     dict(query=q, key=k, cos=table, sin=dual(table))):
            with pytest.raises(NotImplementedError, match="forward"):
                autograd.qk_norm_rotate(**call)
        with torch.no_grad():                              # forward mode does not ask for it
            with pytest.raises(NotImplementedError, match="forward"):
                autograd.qk_norm_rotate(dual(q), k)
        with pytest.raises(ValueError, match="GPU"):       # a level without a dual tensor is no matter
            autograd.qk_norm_rotate(q, k)


def test_forward_mode_is_refused_by_the_scans_and_by_gated_deltanet2():
    q, init = torch.zeros(1, 2, 1, 1, 4), torch.zeros(1, 1, 1, 4)
    xs, start = torch.zeros(1, 2, 3, 4), torch.zeros(1, 3, 4)
    row, dense, state = torch.zeros(1, 1, 16, 8), torch.zeros(1, 1, 16, 8), torch.zeros(1, 1, 8, 8)
    with forward_ad.dual_level():
        for a, b in ((dual(q), init), (q, dual(init))):
            with pytest.raises(NotImplementedError, match="forward"):
                autograd.quat_cumprod(a, b)
            with pytest.raises(NotImplementedError, match="forward"):
                autograd.quat_cumprod_with_final(a, b)
        for a, b in ((dual(xs), start), (xs, dual(start))):
            with pytest.raises(NotImplementedError, match="forward"):
                autograd.scan("quat", a, b)
        with pytest.raises(NotImplementedError, match="forward"):
            autograd.gated_deltanet2(row, row, dual(dense), row, dense, row, state, chunk=16)
        with pytest.raises(NotImplementedError, match="forward"):
            autograd.gated_deltanet2(row, row, dense, row, dense, row, dual(state), chunk=16)
