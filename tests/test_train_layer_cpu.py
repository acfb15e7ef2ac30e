"""Host logic of the auxiliary losses and the 8-bit store in the layer and the stack, without a GPU."""
import pytest
import torch

from sparse_moe_fine_gb300.layer import MoELayer


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
