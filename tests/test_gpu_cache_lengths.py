"""A length that a caller wrote into a cache and that is none (negative, or past
T_max) stops its sequence's step, and nothing of it moves."""
import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp
from parity import bits_equal

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("D,W", [(1, 0), (2, 4)])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 41, 2 ** 31 - 1])
def test_bad_lengths(bits, D, W, bad):
    B, H, Dh, T = 3, 2, 64, 40
    gen = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).to(DEV)
    hk, hv = rnd(B, T - 2, H, Dh), rnd(B, T - 2, H, Dh)
    args = [rnd(B, H, Dh) for _ in range(3)] + [rnd(B, H, Dh).sigmoid()]
    st0 = torch.randn(2, B, H, Dh, generator=gen).to(DEV)
    runs = []
    for length in (T - 2, bad):
        cache = ratp.KVCache(B, H, Dh, T, D, W, kv_bits=bits)
        cache.buffer[:cache.c.len - cache.buffer.data_ptr()].zero_()
        cache.pack(hk, hv)
        cache.lengths()[1] = length
        rows = [cache.dil_rows(w).clone() for w in "kv"] + [r.clone() for r in (cache.ring("k"), cache.ring("v")) if r is not None]
        st, out = st0.clone(), torch.full((B, H, Dh), 7.0, dtype=torch.bfloat16, device=DEV)
        cache.decode_step(*args, st, out=out)
        after = [cache.dil_rows(w) for w in "kv"] + [r for r in (cache.ring("k"), cache.ring("v")) if r is not None]
        if length == bad:
            with pytest.raises(ratp.RatpError, match="CAPACITY"):
                ratp.last_error()
            assert cache.lengths().tolist() == [T - 1, bad, T - 1]
            assert bits_equal(st[:, 1], st0[:, 1]) and bool((out[1] == 7.0).all())
            assert all(bits_equal(a[1], b[1]) for a, b in zip(after, rows))
        else:
            ratp.last_error()
        runs.append([out, st.transpose(0, 1)] + after)
    for a, b in zip(*runs):
        assert bits_equal(a[0], b[0]) and bits_equal(a[2], b[2])
