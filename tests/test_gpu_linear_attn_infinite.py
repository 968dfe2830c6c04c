"""Linear attention with infinite entries in its state: they stay infinite, token by
token, in chunks and over segments, and reach their own columns of o alone."""
import math

import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp
from parity import bits_equal

pytestmark = pytest.mark.gpu
DEV = "cuda"
# exp of these is above, below and exactly an fp32 number: the rest is negative, positive and zero
DECAYS = [-0.25, -0.01, 0.0, -2.0 ** -9]


@pytest.mark.parametrize("Dh", [128, 64])
@pytest.mark.parametrize("T", [0, 1, 9, 40, 300, 128 * 40 + 5])
def test_infinite_entries_stay(T, Dh):
    """T 0: a single-token step."""
    H, n = len(DECAYS), max(T, 1)
    gen = torch.Generator().manual_seed(T + Dh)
    q, k, v = (torch.randn(1, n, H, Dh, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(3))
    s0 = torch.randn(1, H, Dh, Dh, generator=gen).to(DEV)
    ld = torch.tensor(DECAYS, device=DEV)
    hit = torch.zeros_like(s0, dtype=torch.bool)
    hit[:, :, 3, 5] = hit[:, :, Dh - 1, 6] = True
    bad = s0.clone()
    bad[:, :, 3, 5], bad[:, :, Dh - 1, 6] = math.inf, -math.inf
    got = []
    for s in (s0, bad):
        fin = s.clone()
        if T == 0:
            o = ratp.linear_attn_step(*[x[:, 0].contiguous() for x in (q, k, v)], ld, fin)[:, None]
        else:
            o = ratp.linear_attn_prefill(q, k, v, ld, fin, fin)
        got.append((o, fin))
    ratp.last_error()
    (o0, f0), (o1, f1) = got
    assert bits_equal(f1[~hit], f0[~hit])
    # a power that fp32 holds as 0 leaves nothing of it to be infinite
    kept = [h for h, d in enumerate(DECAYS) if math.exp(d * n) > 0 and d * min(n, 128) > -80 and d * n > -80]
    assert len(kept) >= 2
    for h in kept:
        assert float(f1[0, h, 3, 5]) == math.inf and float(f1[0, h, Dh - 1, 6]) == -math.inf, DECAYS[h]
    col = torch.ones(Dh, dtype=torch.bool, device=DEV)
    col[5] = col[6] = False
    assert bits_equal(o1[..., col], o0[..., col])
    assert not bool(torch.isfinite(o1[:, :, kept][..., ~col].float()).any())
