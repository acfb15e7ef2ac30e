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
