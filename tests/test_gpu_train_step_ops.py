"""The auxiliary router losses and the 8-bit activations as a train step uses them: MoELayer with
balance_coef / z_coef, and StackTrainer(act8=True)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import train_oracle as TO
from sparse_moe_fine_gb300 import binding as B
from sparse_moe_fine_gb300 import synth
from sparse_moe_fine_gb300.layer import MoELayer
from sparse_moe_fine_gb300.trainer import StackTrainer

from _gpu import device, rel_l2

pytestmark = pytest.mark.gpu

CFG = synth.small_config("aux_step", T=256, H=128, E=8, k=2, I=128, bf16=True, frac=0.05)
# every token at every expert: no routing choice for a rounding to flip
CFG_ALL = synth.small_config("act8_stack", T=256, H=128, E=4, k=4, I=128, bf16=True, frac=0.05)
CFG_F32 = synth.small_config("aux_f32", T=128, H=64, E=8, k=2, I=32, bf16=False, frac=0.05)
CB, CZ = 40.0, 4.0  # of the size that moves this layer's router gradient as the experts' does


def make(dev, cfg, seed, **kw):
    inp = synth.moe_inputs(cfg, seed=seed)
    t = lambda a: torch.from_numpy(a).to(dev).to(torch.bfloat16 if cfg.bf16 else torch.float32)
    act = synth.uniform_mask(cfg.N, cfg.K, seed=seed)
    L = MoELayer(cfg.T, cfg.H, cfg.E, cfg.k, cfg.I, t(inp["w_gate_up"]), t(inp["w_down"]),
                 torch.from_numpy(inp["w_router"]).to(dev), torch.from_numpy(act).to(dev),
                 device=dev, **kw)
    return L, inp, act, t(inp["x"]), t(inp["dy"])


def reference(inp, cfg, logits, mask=None, off=None):
    idx, w = oracle.route_topk(logits, cfg.k)
    b = oracle.moe_backward(inp["x"], inp["w_router"], inp["w_gate_up"], inp["w_down"], idx, w,
                            logits, inp["dy"])
    a = TO.router_aux(logits, idx, cfg.k, CB, CZ, mask, off)
    g, dx = TO.router_grad(a["dlogit"], inp["x"], inp["w_router"])
    return a, b["g_router"], b["dx"], g, dx


@pytest.mark.parametrize("cfg", [CFG, CFG_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("graphed", [False, True])
def test_train_step_adds_the_losses_gradient(cfg, graphed):
    dev = device()
    L, inp, _, x, dy = make(dev, cfg, 3, balance_coef=CB, z_coef=CZ)
    rng = np.random.default_rng(0)
    off = np.array([0, 10, 10, 77, cfg.T], np.int32)
    mask = (rng.random(cfg.T) < 0.9).astype(np.uint8)
    L.set_sequences(torch.from_numpy(off).to(dev), torch.from_numpy(mask).to(dev))
    if graphed and not cfg.bf16:
        pytest.skip("fp32 layers run their forward stages together, outside the captured step")
    step = L.graphed_train_step if graphed else L.train_step
    step(x, dy)
    torch.cuda.synchronize()
    logits = L.logits.cpu().numpy()
    a, gr, dxr, ga, dxa = reference(inp, cfg, logits, mask, off)
    tol = 1e-2 if cfg.bf16 else 1e-5
    assert np.linalg.norm(ga) > 0.1 * np.linalg.norm(gr)  # large enough to be seen
    assert rel_l2(L.g_router.cpu().numpy(), gr + ga) <= tol
    assert rel_l2(L.dx.float().cpu().numpy(), dxr + dxa) <= tol
    np.testing.assert_allclose(L.aux_loss.cpu().numpy(), a["loss"], rtol=2.0 ** -14)
    np.testing.assert_array_equal(L.aux_count.cpu().numpy(), a["count"])
    np.testing.assert_array_equal(L.aux_n.cpu().numpy(), a["n_tok"])
    assert int(L.status.item()) == 0


def test_losses_off_leave_the_step_as_it_was_and_zero_coefficients_are_off():
    dev = device()
    L, _, _, x, dy = make(dev, CFG, 4)
    assert not L.aux and not hasattr(L, "aux_loss")
    with pytest.raises(ValueError):
        L.set_sequences(torch.tensor([0, CFG.T], dtype=torch.int32, device=dev))
    n0 = B.launch_count()
    L.train_step(x, dy)
    plain = B.launch_count() - n0
    M, _, _, x, dy = make(dev, CFG, 4, balance_coef=CB)
    n0 = B.launch_count()
    M.train_step(x, dy)
    assert B.launch_count() - n0 > plain


def test_balance_loss_evens_the_experts_out():
    """Forty steps of a skewed router under the balance loss alone (no upstream gradient): the
    balance falls toward 1."""
    dev = device()
    L, inp, _, x, _ = make(dev, CFG, 5, balance_coef=1.0, lr=3e-3)
    with torch.no_grad():
        L.w_router[0] += 0.05 * x.float().mean(0).sign()
        L.r_p.copy_(L.w_router.reshape(-1))
    x = x + 0.5 * x.float().mean(0).sign().to(x.dtype)
    dy = torch.zeros_like(x)
    seen = []
    for _ in range(40):
        L.train_step(x, dy)
        seen.append(float(L.aux_loss[1].item()))
    assert seen[0] > 1.02 and seen[-1] < seen[0] - 0.5 * (seen[0] - 1.0), seen


def test_checkpoint_keeps_the_coefficients():
    dev = device()
    L, _, _, x, dy = make(dev, CFG, 6, balance_coef=CB, z_coef=CZ)
    L.train_step(x, dy)
    M = MoELayer.from_checkpoint(L.checkpoint(), device=dev)
    assert (M.balance_coef, M.z_coef, M.aux) == (CB, CZ, True)


def test_set_sequences_and_shared_buffers_refuse_what_does_not_fit():
    dev = device()
    L, _, _, _, _ = make(dev, CFG, 7, balance_coef=CB)
    ok = torch.tensor([0, CFG.T], dtype=torch.int32, device=dev)
    for off, mask in ((ok.long(), None), (ok.cpu(), None), (ok[:1], None), (ok[None], None),
                      (ok, torch.ones(CFG.T, device=dev)),
                      (ok, torch.ones(CFG.T - 1, dtype=torch.uint8, device=dev))):
        with pytest.raises(ValueError):
            L.set_sequences(off, mask)
    M, _, _, _, _ = make(dev, CFG_ALL, 7)
    with pytest.raises(ValueError):
        L.share_activations(M)
    with pytest.raises(ValueError):
        L.save_act8(torch.zeros(3, 3, device=dev))


def _stack(dev, act8, n=4, every=0):
    layers = [make(dev, CFG_ALL, 60 + i, balance_coef=CB, z_coef=CZ)[0] for i in range(n)]
    return layers, StackTrainer(layers, total_steps=10, reselect_every=every, act8=act8)


def test_stack_with_8_bit_activations_follows_the_stack_without():
    """Two micro-batches through four layers. Below the top a layer's backward reads 8-bit x and h:
    each entry within 1/127 of its block's largest, so the gradients agree within 3e-2 in norm; the
    top layer reads its own activations and agrees as two runs do."""
    dev = device()
    a, ta = _stack(dev, False)
    b, tb = _stack(dev, True)
    micro = [synth.moe_inputs(CFG_ALL, seed=70 + j) for j in range(2)]
    t = lambda v: torch.from_numpy(v).to(dev).to(torch.bfloat16)
    for tr in (ta, tb):
        tr.step([t(m["x"]) for m in micro], [t(m["dy"]) for m in micro])
    torch.cuda.synchronize()
    assert len({L.x_perm.data_ptr() for L in b}) == 1 and len({L.y.data_ptr() for L in b}) == 2
    assert len({L.h.data_ptr() for L in a}) == 4
    for i, (p, q) in enumerate(zip(a, b)):
        bound = 1e-2 if i == 3 else 3e-2
        for n in ("g_act", "g_router"):
            u, v = getattr(p, n).cpu().numpy(), getattr(q, n).cpu().numpy()
            err = rel_l2(v, u)
            assert err <= bound, (i, n, err)
            assert i == 3 or err > 0
        assert int(q.status.item()) == 0
        np.testing.assert_allclose(q.aux_loss.cpu().numpy(), p.aux_loss.cpu().numpy(), rtol=2e-2)
    met = tb.metrics()[0]
    assert met["skipped"] == [False] * 4 and len(met["aux_loss"]) == 4
    # the stores are what the lower layers keep: 17/16 bytes a value of x and h
    s = tb._stores[0]
    assert s.nbytes() == (CFG_ALL.T * CFG_ALL.H + b[0].h.numel()) * 17 // 16


def test_stack_with_8_bit_activations_reselects():
    dev = device()
    _, tr = _stack(dev, True, n=2, every=2)
    t = lambda v: torch.from_numpy(v).to(dev).to(torch.bfloat16)
    for j in range(3):
        m = synth.moe_inputs(CFG_ALL, seed=80 + j)
        tr.step([t(m["x"])], [t(m["dy"])])
    met = tr.metrics()
    assert met[1]["turnover"] is not None and not any(any(m["skipped"]) for m in met)
