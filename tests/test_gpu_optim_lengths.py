"""AdamW and the norm for lists on both sides of the lengths at which their launches change."""
import numpy as np
import pytest
import torch

from oracle import optim_oracle as OO
from sparse_moe_fine_gb300 import binding as B

from test_gpu_optim import BF16, F32, HYP, Case, device, pytestmark  # noqa: F401

K = 1024


@pytest.mark.parametrize("total", [512 * K, 4 * K * K, 8 * K * K])
@pytest.mark.parametrize("below", [True, False])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("g,offset", [(F32, 0), (BF16, 1)])
def test_step(total, below, bits, g, offset):
    n = total - below
    sizes = [n // 2 - 77, 0, 128, n - n // 2 - 51]
    assert sum(sizes) == n
    c = Case(device(), sizes, bits, g=g, offset=offset)
    B.adamw_step(c.t, HYP["lr"], HYP["beta1"], HYP["beta2"], HYP["eps"], HYP["step"], seed=7)
    c.check(seed=7)


@pytest.mark.parametrize("total", [16 * K, 4 * K * K])
@pytest.mark.parametrize("more", [0, 1])
@pytest.mark.parametrize("count", [1, 64, 65])
@pytest.mark.parametrize("g,offset", [(F32, 0), (BF16, 0), (F32, 3)])
def test_norm(total, more, count, g, offset):
    dev = device()
    cut = np.sort(np.random.default_rng(count).choice(total + more, count - 1, replace=False))
    sizes = np.diff(np.concatenate([[0], cut, [total + more]])).tolist()
    c = Case(dev, sizes, 32, g=g, offset=offset)
    out = torch.zeros(2, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    B.grad_norm(c.t, 0.25, out, dev_status=st)
    norm, scale = OO.grad_norm(c.g0, 0.25)
    # squares and sums of four in fp32 (3 half ulps of the sum, half of that of its root), the result's rounding
    np.testing.assert_allclose(out.cpu().numpy(), [norm, scale], rtol=2.0 ** -22)
    assert int(st.item()) == 0
