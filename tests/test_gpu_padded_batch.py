"""A decode step that is handed a batch padded at its end uses the front."""
import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp
from parity import bits_equal

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("bits", [4, 16])
def test_the_front_of_larger_tensors_is_used(bits):
    B, pad, H, Dh, T = 2, 5, 2, 64, 40
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).to(DEV)
    hk, hv = rnd(B, T, H, Dh), rnd(B, T, H, Dh)
    q, xk, xv, g = (rnd(pad, H, Dh) for _ in range(4))
    st0 = torch.randn(2, B, H, Dh, generator=gen).to(DEV)
    flat = torch.full((2 * pad * H * Dh,), 9.0, device=DEV)
    flat[:st0.numel()] = st0.flatten()
    want, state = None, st0.clone()
    for padded in (False, True):
        for call in ("step", "layers"):
            cache = ratp.KVCache(B, H, Dh, T + 1, 2, 4, kv_bits=bits)
            cache.pack(hk, hv)
            st = flat.clone() if padded else st0.clone()
            args = [x if padded else x[:B].contiguous() for x in (q, xk, xv, g)]
            out = torch.full_like(args[0], 7.0)
            if call == "step":
                cache.decode_step(*args, st, out=out)
            else:
                ratp.decode_step_layers([(cache, *args, st, out)])
            if want is None:
                want, state = out, st
            assert bits_equal(out[:B], want) and bool((out[B:] == 7.0).all())
            assert bits_equal(st.flatten()[:state.numel()], state.flatten()) and bool((st.flatten()[state.numel():] == 9.0).all())
    # without an output: one of q's shape
    cache = ratp.KVCache(B, H, Dh, T + 1, 2, 4, kv_bits=bits)
    cache.pack(hk, hv)
    assert bits_equal(cache.decode_step(q, xk, xv, g, flat.clone())[:B], want)
    # the state of a larger batch holds this one's value stream elsewhere
    with pytest.raises(ValueError):
        cache.decode_step(q, xk, xv, g, torch.zeros(2, pad, H, Dh, device=DEV))
    ratp.last_error()
