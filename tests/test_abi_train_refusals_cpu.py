"""Refusals of the calls of include/usaf_train.h and of their binding that keep bad pointers off the
GPU, checked on the host."""
import ctypes

import pytest
import torch

from sparse_moe_fine_gb300 import binding as B

fake_addresses = pytest.mark.skipif(torch.cuda.is_available(),
                                    reason="fake device addresses; run where no GPU is visible")
FAKE = ctypes.c_void_p(4096)  # never dereferenced: the calls below fail on the host


@fake_addresses
@pytest.mark.parametrize("at", [4097, 4098, 4100, 4104])
def test_aux_workspace_has_to_be_aligned(at):
    """fp32 and int32 partial sums are stored from the workspace's start on."""
    r = B.lib().usaf_router_aux_fwd(8, 4, 2, FAKE, 4, FAKE, None, None, 1, 1.0, 1.0, FAKE, FAKE, FAKE,
                                    FAKE, None, ctypes.c_void_p(at), 1 << 30, None)
    assert r == 1


def test_routing_tables_may_be_absent_or_addresses():
    """A routing whose fields are None or bare addresses reaches the library, which refuses what it
    needs and does not have."""
    t = torch.zeros(4, dtype=torch.int32)
    r = B.Routing(t, None, 4096, t, None, 0, t).c()
    got = [getattr(r, f) for f, _ in B._Routing._fields_]
    assert got[0] == got[3] == got[6] == t.data_ptr() and got[2] == 4096
    assert got[1] is None and got[4] is None and not got[5]
    s = B.shape(4, 64, 4, 2, 64)
    with pytest.raises(B.UsafError):
        B.route_topk_noalloc(s, None, None, B.Routing(*[None] * 7), logits_in=4096, stream=0)
