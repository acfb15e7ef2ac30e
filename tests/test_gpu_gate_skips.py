"""Steps that are skipped although every rank's own gradient is finite: the sum over the ranks is not, or only
the norm of all routers' gradients is not. The sum is made in the test, in the place of the ranks'
all-reduce. What such a step leaves alone, it leaves alone as a whole, and says so."""
import pytest
import torch

from sparse_moe_fine_gb300 import binding as B
from sparse_moe_fine_gb300 import layer as layer_module
from sparse_moe_fine_gb300 import synth
from sparse_moe_fine_gb300.trainer import StackTrainer

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


@pytest.mark.parametrize("opt", [dict(weight_decay=0.1), dict(state_bits=8), dict(max_norm=1.0)],
                         ids=["fp32", "8bit", "clipped"])
@pytest.mark.parametrize("total", [router_overflows, experts_overflow, flagged])
def test_all_routers_stay_when_one_layers_sum_is_not_finite(monkeypatch, opt, total):
    dev = device()
    layers = [make(dev, CFG, 50 + i, bias_rate=0.01)[0] for i in range(3)]
    tr = StackTrainer(layers, total_steps=10, router_adamw=opt)
    m = synth.moe_inputs(CFG, seed=50)
    x, dy = (torch.from_numpy(m[n]).to(dev).to(torch.bfloat16) for n in ("x", "dy"))
    tr.step([x], [dy])
    routers = lambda: [t.clone() for L in layers for t in (L.r_p, L.w_router)] + [
        t.view(torch.uint8).clone() for t in tr.router_opt.m + tr.router_opt.v]
    before, states = routers(), [_trained(L) for L in layers]
    biases = [L.gate_bias.clone() for L in layers]
    ranks(monkeypatch, layers, [same, total, same])
    tr.step([x], [dy])
    torch.cuda.synchronize()
    assert _equal(routers(), before)
    assert _equal(_trained(layers[1]), states[1]) and torch.equal(layers[1].gate_bias, biases[1])
    for i in (0, 2):                                          # their own step was sound
        assert not torch.equal(layers[i].p, states[i][2]) and not torch.equal(layers[i].gate_bias, biases[i])
    ranks(monkeypatch, layers, [same] * 3)
    tr.step([x], [dy])
    torch.cuda.synchronize()
    after = routers()
    # (the bottom router's; the others' gradients are below 1e-15 here, a step of lr g / eps less than a rounding)
    assert not torch.equal(after[0], before[0]) and not torch.equal(after[1], before[1])
    assert all(torch.isfinite(L.r_p).all() for L in layers)
    skipped = [r["skipped"] for r in tr.metrics()]
    bad = total is not flagged
    assert skipped == [[False] * 3, [False, bad, False], [False] * 3]


def test_a_skip_of_the_routers_alone_is_recorded(monkeypatch):
    """A finite gradient whose square passes fp32 is found by the norm, after the layers' own updates."""
    dev = device()
    layers = [make(dev, CFG, 60 + i)[0] for i in range(2)]
    tr = StackTrainer(layers, total_steps=10, router_adamw=dict(max_norm=1.0))
    m = synth.moe_inputs(CFG, seed=60)
    x, dy = (torch.from_numpy(m[n]).to(dev).to(torch.bfloat16) for n in ("x", "dy"))
    tr.step([x], [dy])
    before, p = [L.r_p.clone() for L in layers], layers[0].p.clone()

    def large(ga, gr, st):
        gr.view(-1)[5] = 1e30
    ranks(monkeypatch, layers, [large, same])
    tr.step([x], [dy])
    ranks(monkeypatch, layers, [same, same])
    kept = _equal([L.r_p for L in layers], before)
    tr.step([x], [dy])
    got = tr.metrics()
    assert kept and not torch.equal(layers[0].p, p)
    assert [r["router_skipped"] for r in got] == [False, True, False]
    assert [r["skipped"] for r in got] == [[False] * 2] * 3
    plain = StackTrainer([make(dev, CFG, 62)[0]], total_steps=10)
    plain.step([x], [dy])
    assert plain.metrics()[0]["router_skipped"] is None


@pytest.mark.parametrize("total", [router_overflows, flagged])
def test_one_layers_skip_is_one_of_the_routers_too(monkeypatch, total):
    dev = device()
    layers = [make(dev, CFG, 64 + i)[0] for i in range(2)]
    tr = StackTrainer(layers, total_steps=10, router_adamw=dict(weight_decay=0.1))
    m = synth.moe_inputs(CFG, seed=64)
    x, dy = (torch.from_numpy(m[n]).to(dev).to(torch.bfloat16) for n in ("x", "dy"))
    ranks(monkeypatch, layers, [total, same])
    tr.step([x], [dy])
    assert tr.metrics()[0]["router_skipped"] is True
