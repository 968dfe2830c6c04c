"""Hand-offs of a prompt's first tokens: a cache packed from longer tensors holds
what it holds when those tokens alone are given."""
import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp
from parity import bits_equal

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("n", [2, 3])
def test_the_first_tokens_of_longer_tensors(bits, n):
    B, H, Dh, T = 2, 2, 64, 37
    gen = torch.Generator().manual_seed(1)
    xk, xv, g = (torch.randn(n, 50, H, Dh, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(3))
    got = []
    for cut in (False, True):
        cache = ratp.KVCache(B, H, Dh, T, 1, 8, kv_bits=bits)
        cache.attach_window(16)
        cache.in_ring.zero_()
        x = [t[:B, :T].contiguous() if cut else t for t in (xk, xv, g)]
        cache.pack(x[0], x[1], T)
        cache.pack_inputs(*x, T)
        assert cache.lengths().tolist() == [T] * B
        got.append([cache.dil_rows(w) for w in "kv"] + [cache.ring(w) for w in "kv"] + [cache.in_ring])
    assert all(bits_equal(a, b) for a, b in zip(*got))
    with pytest.raises(ValueError):
        cache.pack_inputs(x[0], x[1][:1].contiguous(), x[2])
    ratp.last_error()
