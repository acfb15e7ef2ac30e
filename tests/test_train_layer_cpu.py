"""Host logic of the auxiliary losses and the 8-bit store in the layer and the stack, without a GPU."""
import pytest
import torch

from sparse_moe_fine_gb300.layer import MoELayer
from sparse_moe_fine_gb300.trainer import StackTrainer


def _bare(group=None):
    L = MoELayer.__new__(MoELayer)
    L.dev, L.group, L._shares = torch.device("cpu"), group, {}
    return L


def test_a_calls_share_of_the_step(monkeypatch):
    assert _bare().aux_share() is None and _bare().aux_share(1) is None
    assert _bare().aux_share(3).tolist() == [torch.tensor(1 / 3).item()]
    monkeypatch.setattr(torch.distributed, "get_world_size", lambda g: 4)
    L = _bare(group=object())
    assert L.aux_share().tolist() == [0.25] and L.aux_share(2).tolist() == [0.125]
    assert L.aux_share(2) is L.aux_share(2)  # captured steps and replays read one tensor


def test_live_tokens_by_mask_and_sequences():
    L = _bare()
    L.T = 10
    off = torch.tensor([2, 2, 5, 8], dtype=torch.int32)
    mask = torch.tensor([1, 1, 0, 3, 1, 0, 1, 1, 1, 1], dtype=torch.uint8)
    assert int(L.live_tokens()) == 10
    assert int(L.live_tokens(off)) == 6
    assert int(L.live_tokens(None, mask)) == 8
    assert int(L.live_tokens(off, mask)) == 4


class _Stub:
    aux, group, dev, T = True, None, torch.device("cpu"), 6
    live_tokens = MoELayer.live_tokens


def test_micro_batches_count_by_their_tokens(monkeypatch):
    tr = StackTrainer([_Stub()], total_steps=1)
    mask = lambda n: (None, torch.tensor([1] * n + [0] * (6 - n), dtype=torch.uint8))
    assert [s.tolist() for s in tr._shares([mask(6), mask(3), mask(3)])] == [[0.5], [0.25], [0.25]]
    assert [s.tolist() for s in tr._shares([mask(0), mask(0)])] == [[0.0], [0.0]]
    # another rank with as many tokens again
    tr.layers[0].group = object()
    monkeypatch.setattr(torch.distributed, "all_reduce", lambda t, group: t.mul_(2))
    assert [s.tolist() for s in tr._shares([mask(6), mask(2)])] == [[0.375], [0.125]]


def test_step_refuses_sequences_that_do_not_fit():
    tr = StackTrainer([_Stub()], total_steps=1)
    x = [torch.zeros(6, 4)] * 2
    with pytest.raises(ValueError):
        tr.step(x, x, sequences=[(None, None)])
    tr.layers[0].aux = False
    with pytest.raises(ValueError):
        tr.step(x, x, sequences=[(None, None)] * 2)
    assert tr.step_no == 0
