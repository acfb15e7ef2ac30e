"""Padding tokens and the balancing bias: tokens that a mask or the packed sequences leave out do not move it,
with the auxiliary losses on and off, over micro-batches and in a captured step."""
import numpy as np
import pytest
import torch

from oracle import gate_oracle as GO
from sparse_moe_fine_gb300.trainer import StackTrainer

from test_gpu_gate_step import CFG, device, make, pytestmark  # noqa: F401


def padded(x, live):
    """The batch with one row in the place of all tokens that are not live."""
    x = x.clone()
    x[~live] = x[0] * 0.5
    return x


def parts(dev, how):
    """(group_offset, token_mask, live) of a batch: a third of it is padding."""
    live = torch.ones(CFG.T, dtype=torch.bool, device=dev)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
    if how == "mask":
        live[torch.arange(CFG.T, device=dev) % 3 == 1] = False
        return None, live.to(torch.uint8), live
    live[:5], live[180:] = False, False
    if how == "packed":
        return i32([5, 5, 90, 180]), None, live
    live[60:70] = False
    return i32([5, 100, 180]), live.to(torch.uint8), live


def counts(L, live):
    idx = L.rt.topk_idx.view(CFG.T, CFG.k)[live]
    return np.bincount(idx.reshape(-1).cpu().numpy(), minlength=CFG.E)


@pytest.mark.parametrize("aux", [dict(balance_coef=1e-2), dict(z_coef=1e-3), {}], ids=["balance", "z", "off"])
@pytest.mark.parametrize("how", ["mask", "packed", "both"])
@pytest.mark.parametrize("graphed", [False, True])
def test_padding_does_not_move_the_bias(aux, how, graphed):
    dev = device()
    L, _, _, x, dy = make(dev, CFG, 11, bias_rate=0.01, **aux)
    off, mask, live = parts(dev, how)
    x = padded(x, live)
    step = L.graphed_train_step if graphed else L.train_step
    bias = np.zeros(CFG.E)
    for given in ((off, mask), (None, None), (off, mask)):
        L.set_sequences(*given)
        for _ in range(2):
            step(x, dy)
            torch.cuda.synchronize()
            seen = counts(L, live if given[0] is not None or given[1] is not None else slice(None))
            np.testing.assert_array_equal(L.gate_load.cpu().numpy(), seen)
            bias = GO.gate_balance(bias, seen, 0.01)
            # six steps of one rounding each, of sums below 2^-4
            np.testing.assert_allclose(L.gate_bias.cpu().numpy(), bias, rtol=0, atol=6 * 2.0 ** -28)
    assert int(L.status.item()) == 0


@pytest.mark.parametrize("aux", [dict(balance_coef=1e-2), {}], ids=["balance", "off"])
def test_micro_batches_of_a_stack(aux):
    dev = device()
    layers = [make(dev, CFG, 20 + i, bias_rate=0.01, **aux)[0] for i in range(2)]
    tr = StackTrainer(layers, total_steps=10)
    x, dy = make(dev, CFG, 20)[3:]
    given = [parts(dev, h) for h in ("mask", "both")]
    total = [np.zeros(CFG.E, np.int64) for _ in layers]

    def count(L, i, backward=layers[0].__class__.backward_into):
        def f(*a, **kw):
            live = given[count.at[i]][2]
            total[i] += counts(L, live)
            count.at[i] += 1
            return backward(L, *a, **kw)
        return f
    count.at = [0, 0]
    for i, L in enumerate(layers):
        L.backward_into = count(L, i)
    tr.step([padded(x, g[2]) for g in given], [dy, dy], sequences=[g[:2] for g in given])
    for L, n in zip(layers, total):
        np.testing.assert_array_equal(L.gate_load.cpu().numpy(), n)
    assert int(layers[0].gate_load.sum()) < 2 * CFG.T * CFG.k


def test_sequences_without_a_bias_or_losses_are_refused():
    dev = device()
    L, _, _, x, dy = make(dev, CFG, 24)
    mask = torch.ones(CFG.T, dtype=torch.uint8, device=dev)
    with pytest.raises(ValueError):
        L.set_sequences(None, mask)
    with pytest.raises(ValueError):
        StackTrainer([L], total_steps=10).step([x], [dy], sequences=[(None, mask)])
