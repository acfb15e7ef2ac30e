"""Steps that are skipped although every rank's own gradient is finite: the sum over the ranks is not. The sum
is made in the test, in the place of the ranks' all-reduce. Such a step leaves everything alone."""
import pytest
import torch

from sparse_moe_fine_gb300 import binding as B
from sparse_moe_fine_gb300 import layer as layer_module

from test_gpu_gate_step import CFG, device, make, pytestmark  # noqa: F401

INF = float("inf")


def ranks(monkeypatch, layers, sums):
    """Each layer's all-reduce is sums[i](g_act, g_router, status); counts stay as they are."""
    monkeypatch.setattr(layer_module, "allreduce_grads", lambda ga, gr, st, group: group(ga, gr, st))
    monkeypatch.setattr(layer_module, "allreduce_load", lambda load, group: None)
    for L, f in zip(layers, sums):
        L.group = f


def same(ga, gr, st):
    pass


def router_overflows(ga, gr, st):
    gr.view(-1)[5] = INF


def experts_overflow(ga, gr, st):
    ga[7] = INF


def flagged(ga, gr, st):
    st.bitwise_or_(B.DEV_TIMEOUT)


def _trained(L):
    return [t.clone() for t in (L.w_gate_up, L.w_down, L.p, L.m, L.v, L.w_router, L.r_p, L.r_m, L.r_v)]


def _equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("where", ["router", "experts"])
def test_bias_and_weights_stay_when_either_gradient_is_not_finite(where):
    dev = device()
    L, _, _, x, dy = make(dev, CFG, 6, bias_rate=0.01)
    L.train_step(x, dy)
    L.wait_optimizer()
    before, bias = _trained(L), L.gate_bias.clone()
    assert bias.any() and int(L.status.item()) == 0
    (L.g_router.view(-1) if where == "router" else L.g_act)[3] = INF
    L.optimizer_step()
    torch.cuda.synchronize()
    assert int(L.status.item()) == B.DEV_NONFINITE
    assert torch.equal(L.gate_bias, bias) and _equal(_trained(L), before)


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("total", [router_overflows, experts_overflow, flagged])
def test_a_rank_moves_all_of_a_step_or_nothing(monkeypatch, gated, total):
    dev = device()
    kw = {} if gated else dict(rule=None)
    L, _, _, x, dy = make_any(dev, 8, **kw)
    L.train_step(x, dy)
    L.wait_optimizer()
    before = _trained(L)
    ranks(monkeypatch, [L], [total])
    for _ in range(4):
        L.train_step(x, dy)
    torch.cuda.synchronize()
    assert _equal(_trained(L), before)
    ranks(monkeypatch, [L], [same])
    L.train_step(x, dy)
    torch.cuda.synchronize()
    assert not any(torch.equal(a, b) for a, b in zip(_trained(L), before))


def make_any(dev, seed, rule=dict(score="sigmoid")):
    if rule is not None:
        return make(dev, CFG, seed, rule)
    L, inp, act, x, dy = make(dev, CFG, seed)
    M = layer_module.MoELayer(CFG.T, CFG.H, CFG.E, CFG.k, CFG.I, L.w_gate_up, L.w_down, L.w_router, L.act,
                              device=dev)
    return M, inp, act, x, dy
