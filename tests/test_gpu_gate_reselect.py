"""Gated layers through a reselection: the dense expert gradient from the workspace that the experts' backward
leaves, and a stack of gated layers with AdamW routers over reselections, alone and as one of the ranks."""
import numpy as np
import pytest
import torch

import oracle
from oracle import gate_oracle as GO
from sparse_moe_fine_gb300 import binding as B
from sparse_moe_fine_gb300 import layer as layer_module
from sparse_moe_fine_gb300 import synth
from sparse_moe_fine_gb300 import trainer as trainer_module
from sparse_moe_fine_gb300.trainer import StackTrainer

from _gpu import rel_l2
from test_gpu_gate_step import CFG, CFG_F32, RULES, device, make, pytestmark  # noqa: F401


@pytest.mark.parametrize("rule", RULES, ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("cfg", [CFG, CFG_F32], ids=["bf16", "f32"])
def test_dense_gradient_behind_the_experts_backward(rule, cfg):
    dev = device()
    L, inp, act, x, dy = make(dev, cfg, 12, rule, bias_rate=0.01)
    L.train_step(x, dy)                                        # weights as they are after one step
    inp = {**inp, "w_gate_up": L.w_gate_up.float().cpu().numpy(), "w_down": L.w_down.float().cpu().numpy(),
           "w_router": L.w_router.cpu().numpy()}
    bias = L.gate_bias.cpu().numpy().copy()
    L.route(x)
    L.forward(x)
    L.backward_into(x, dy, dx=L.dx)
    g = torch.full((L.N,), float("nan"), device=dev)
    B.moe_wgrad_dense(L.s, L.rt, L.x_perm, L.wa, g, L.ws_bwd, accumulate=0, dev_status=L.status)
    B.moe_wgrad_dense(L.s, L.rt, L.x_perm, L.wa, g, L.ws_bwd, accumulate=1, dev_status=L.status)
    torch.cuda.synchronize()
    idx, w = GO.gate_topk(L.logits.cpu().numpy(), cfg.k, bias=bias, **rule)
    np.testing.assert_array_equal(L.rt.topk_idx.cpu().numpy().reshape(cfg.T, cfg.k), idx)
    ref = oracle.masked_expert_grad(np.arange(L.N), inp["x"], inp["w_gate_up"], inp["w_down"], idx, w,
                                    inp["dy"])
    tol = 1e-2 if cfg.bf16 else 1e-5
    assert rel_l2(g.cpu().numpy(), 2 * ref) <= tol
    assert rel_l2(L.g_act.cpu().numpy(), ref[act]) <= tol
    assert int(L.status.item()) == 0


@pytest.mark.parametrize("mode", ["rigl", "full"])
@pytest.mark.parametrize("rank", [False, True])
@pytest.mark.parametrize("act8", [False, True])
def test_stack_over_reselections(monkeypatch, mode, rank, act8):
    dev = device()
    layers = [make(dev, CFG, 70 + i, bias_rate=0.01)[0] for i in range(2)]
    if rank:  # one of two ranks whose partner has the same tokens: every sum is twice its own
        for L in layers:
            L.group = "ranks"
        double = lambda *ts: [t.mul_(2) for t in ts]
        monkeypatch.setattr(layer_module, "allreduce_grads", lambda ga, gr, st, group: double(ga, gr))
        monkeypatch.setattr(layer_module, "allreduce_load", lambda load, group: double(load))
        monkeypatch.setattr(trainer_module, "allreduce_dense_grad", lambda g, group: double(g))
    tr = StackTrainer(layers, total_steps=10, reselect_every=2, reselect=mode, act8=act8,
                      router_adamw=dict(weight_decay=0.1, max_norm=1.0))
    old = [L.act.clone() for L in layers]
    micro = [synth.moe_inputs(CFG, seed=71 + j) for j in range(2)]
    t = lambda v: torch.from_numpy(v).to(dev).to(torch.bfloat16)
    bias = [np.zeros(CFG.E) for _ in layers]
    for _ in range(5):
        tr.step([t(m["x"]) for m in micro], [t(m["dy"]) for m in micro])
        torch.cuda.synchronize()
        for i, L in enumerate(layers):
            load = L.gate_load.cpu().numpy()
            assert load.sum() == (2 if rank else 1) * 2 * CFG.T * CFG.k
            bias[i] = GO.gate_balance(bias[i], load, 0.01)
            # five steps of one rounding each, of sums below 2^-4
            np.testing.assert_allclose(L.gate_bias.cpu().numpy(), bias[i], rtol=0, atol=5 * 2.0 ** -28)
    got = tr.metrics()
    assert [r["turnover"] is not None for r in got] == [False, True, False, True, False]
    assert [r["skipped"] for r in got] == [[False] * 2] * 5
    for L, a in zip(layers, old):
        new = L.act.cpu().numpy()
        assert new.size == CFG.K and (np.diff(new) > 0).all() and not torch.equal(L.act, a)
        assert all(torch.isfinite(q).all() for q in (L.p, L.m, L.v, L.r_p, L.w_gate_up, L.w_down))
