"""The 4-bit decode step over long heads whose keys weigh alike: the output is the
small rest of values that cancel, so it shows what the value sums lose.

Reference: attention in fp64 over the values that the cache holds.  Tolerance in
the norm: the rounding of o is at most 2^-8 / sqrt(3) of it (uniform in half a
bf16 step, values at the low end of their binade); the value sums lose at most
one last place, 2^-23, of 23.5 p s a key at each of the 16 products between two
takings out of the offset, 2^-23 * 23.5 * 136 / 16 < 2^-15.3 of the mean step s in
all, the same for every output and whatever the number of keys; weights of 16
bits and scores move key by key (2^-16 each, of |v| / sqrt(N) in the mean square,
which is |o| itself): 2^-14 of the norm."""
import math

import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp

pytestmark = pytest.mark.gpu
DEV = "cuda"


def reference(cache, q, state):
    """o in fp64 [B, H, Dh] and the mean step of the held rows; no window, D == 1."""
    k, v = (cache.dil_rows(w).double() for w in "kv")
    B, H, Dh = q.shape
    o = torch.empty(B, H, Dh, dtype=torch.float64, device=q.device)
    own = state.to(torch.bfloat16).double()
    n, steps = int(cache.lengths()[0]) - 1, []
    for h in range(H):
        off, _ = cache.head_rows(h)
        kk = torch.cat([k[:, off:off + n], own[0][:, h:h + 1]], 1)
        vv = torch.cat([v[:, off:off + n], own[1][:, h:h + 1]], 1)
        p = torch.softmax(torch.einsum("bd,bnd->bn", q[:, h].double(), kk) / math.sqrt(Dh), 1)
        o[:, h] = torch.einsum("bn,bnd->bd", p, vv)
        g = v[:, off:off + n].unflatten(-1, (-1, 32))
        steps.append((g.amax(-1) - g.amin(-1)).mean() / 15)
    return o, float(sum(steps)) / H


@pytest.mark.parametrize("Dh", [128, 64])
@pytest.mark.parametrize("B,H,T,whole", [
    (1, 2, 8192, True),
    (1, 2, 65536, True),       # one split: 32768 keys a warp
    (1, 1, 65536, False),      # as the cache splits it
    (4, 16, 32768, False),
    (1, 1, 1 << 20, False),    # as many splits as a head can have
])
def test_alike_keys(B, H, T, whole, Dh):
    gen = torch.Generator(device=DEV).manual_seed(T + Dh)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(torch.bfloat16)
    cache = ratp.KVCache(B, H, Dh, T + 32, 1, kv_bits=4)
    cache.pack(rnd(B, T, H, Dh), rnd(B, T, H, Dh))
    if whole:
        cache.c.split_keys = 1 << 20
    q = rnd(B, H, Dh) * 0.05
    state = torch.randn(2, B, H, Dh, generator=gen, device=DEV)
    out = cache.decode_step(q, rnd(B, H, Dh), rnd(B, H, Dh), rnd(B, H, Dh).sigmoid(), state)
    ratp.last_error()
    ref, step = reference(cache, q, state)
    err, norm = float((out.double() - ref).norm()), float(ref.norm())
    tol = (2.0 ** -8 / math.sqrt(3) + 2.0 ** -14) * norm + 2.0 ** -15.3 * step * math.sqrt(ref.numel())
    assert err <= tol, (err / norm, tol / norm)
