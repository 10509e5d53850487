"""The grouped products where each CTA pair walks many units: about 76 pairs take
40 tiles and more of y and dx and 80 of dW, which their roles find 16 and 32 at a
time."""
import pytest
import torch

import test_gpu_moe_experts as plain
import test_gpu_moe_experts8 as eight

pytestmark = pytest.mark.gpu


def _counts(most):
    return torch.randint(1, most, (1024,), generator=torch.Generator().manual_seed(most)).tolist()


def test_bf16():
    plain._check(_counts(12), 648, 520, seed=4)


@pytest.mark.parametrize("most", [4, 140])
def test_8_bits(most):
    eight._check(_counts(most), 648, 144, seed=5)
