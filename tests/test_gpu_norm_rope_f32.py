"""The fp32 q/k norm divides by the root that fp32 arithmetic gives: rows of one
magnitude c, a multiple of 1/64 whose square and its sums are exact, so that
without eps the mean is c^2, its reciprocal root 1/c rounded once, and y the
product of the two rounded once."""
import numpy as np
import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Dh", [64, 128])
def test_reciprocal_root_is_rounded_once(Dh):
    c = torch.arange(1, 1025, dtype=torch.float32) / 64          # squares of at most 20 bits, 2 more for their sums
    gen = torch.Generator().manual_seed(Dh)
    sign = torch.randint(0, 2, (1, 1024, 1, Dh), generator=gen) * 2 - 1
    x = (c.view(1, -1, 1, 1) * sign).cuda()
    y, _ = ratp.qk_norm_rope(x, None, None, None, None, eps=0.0)
    ratp.last_error()
    r = np.float32(1) / c.numpy()
    want = (c.numpy() * r)[None, :, None, None] * sign.numpy().astype(np.float32)
    assert np.array_equal(y.cpu().numpy(), want)
