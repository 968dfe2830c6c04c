"""4-bit cache: keys whose scores are NaN wherever they lie, and the quantiser at
quotients next to a tie."""
import numpy as np
import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("Dh", [128, 64])
@pytest.mark.parametrize("T,D,W,nan_from,nan_to,whole", [
    (1, 1, 0, 0, 1, True),          # the only cached key
    (40, 1, 0, 32, 40, True),       # all of one warp's keys, the other warp's are finite
    (1, 64, 8, 0, 1, True),         # the only ring key
    (30, 64, 40, 8, 16, True),      # all of one warp's first ring rows
    (1056, 1, 0, 512, 768, False),  # all keys of one split
])
def test_keys_of_nan_reach_the_output(T, D, W, nan_from, nan_to, whole, Dh):
    gen = torch.Generator().manual_seed(T + Dh)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).to(DEV)
    hk, hv = rnd(1, T, 2, Dh), rnd(1, T, 2, Dh)
    args = [rnd(1, 2, Dh) for _ in range(3)] + [rnd(1, 2, Dh).sigmoid()]
    outs = []
    for bad in (False, True):
        k = hk.clone()
        if bad:
            k[0, nan_from:nan_to, 1] = float("nan")
        cache = ratp.KVCache(1, 2, Dh, T + 1, D, W, kv_bits=4)
        if not whole:
            assert cache.c.split_keys <= nan_to - nan_from and nan_from % cache.c.split_keys == 0
        cache.pack(k, hv)
        outs.append(cache.decode_step(*args, torch.zeros(2, 1, 2, Dh, device=DEV)))
    ratp.last_error()
    assert bool(torch.isfinite(outs[0]).all())
    assert torch.equal(outs[1][0, 0], outs[0][0, 0])
    assert bool(torch.isnan(outs[1][0, 1]).all())
