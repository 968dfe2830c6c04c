"""4-bit cache: keys whose scores are NaN wherever they lie, and the quantiser at
quotients next to a tie."""
import numpy as np
import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("Dh", [128, 64])
@pytest.mark.parametrize("T,D,W,nan_from,nan_to", [
    (1, 1, 0, 0, 1),                # the only cached key
    (40, 1, 0, 32, 40),             # all of one warp's keys, the other warp's are finite
    (1, 64, 8, 0, 1),               # the only ring key
    (30, 64, 40, 8, 16),            # all of one warp's first ring rows
    (1056, 1, 0, None, None),       # all keys of the second split
])
def test_keys_of_nan_reach_the_output(T, D, W, nan_from, nan_to, Dh):
    gen = torch.Generator().manual_seed(T + Dh)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).to(DEV)
    hk, hv = rnd(1, T, 2, Dh), rnd(1, T, 2, Dh)
    args = [rnd(1, 2, Dh) for _ in range(3)] + [rnd(1, 2, Dh).sigmoid()]
    outs = []
    for bad in (False, True):
        k = hk.clone()
        cache = ratp.KVCache(1, 2, Dh, T + 1, D, W, kv_bits=4)
        if nan_from is None:
            nan_from, nan_to = cache.c.split_keys, 2 * cache.c.split_keys
            assert nan_to < T
        if bad:
            k[0, nan_from:nan_to, 1] = float("nan")
        cache.pack(k, hv)
        outs.append(cache.decode_step(*args, torch.zeros(2, 1, 2, Dh, device=DEV)))
    ratp.last_error()
    assert bool(torch.isfinite(outs[0]).all())
    assert torch.equal(outs[1][0, 0], outs[0][0, 0])
    assert bool(torch.isnan(outs[1][0, 1]).all())


def near_ties(Dh, seed):
    """Rows whose groups have small values beside a minimum of (k + 1/2) steps: the
    quotient lies next to a tie, on it where the difference rounds to it.  Returns
    (rows bf16 [n, Dh], the values they stand for in fp32, codes that one rounding
    of the quotient to 2^-19 would have got wrong)."""
    r = np.random.default_rng(seed)
    n, groups = 240, Dh // 32
    x = np.zeros((n, groups, 32))
    for i in range(n):
        for j in range(groups):
            s, k, scale = r.choice([2.0, 3.0, 5.0]), int(r.integers(0, 15)), 2.0 ** int(r.integers(-40, 41))
            lo = -(k + 0.5) * s
            small = (1 + r.integers(0, 128, 32) / 128) * 2.0 ** r.integers(-30, -12, 32).astype(float) * r.choice([-1, 1], 32)
            small[0], small[1] = lo, lo + 15 * s
            x[i, j] = small * scale
    x = torch.from_numpy(x).to(torch.bfloat16)
    f = x.float().numpy()
    lo = f.min(-1, keepdims=True)
    d = f - lo                                               # rounds as the definition's difference in fp32
    step = torch.from_numpy((f.max(-1, keepdims=True) - lo) / np.float32(15)).to(torch.bfloat16).float().numpy()
    q = d.astype(np.float64) / step                          # 53 bits: a tie is one, and what is none stays off it
    code = np.rint(q)
    snapped = np.rint((q + 24).astype(np.float32).astype(np.float64) - 24)
    held = (lo.astype(np.float64) + code * step).astype(np.float32)
    return x.view(n, Dh), held.reshape(n, Dh), int((snapped != code).sum())


@pytest.mark.parametrize("Dh", [128, 64])
def test_codes_next_to_a_tie(Dh):
    """The hand-off (16 channels a thread) and the appended row (8): both take the
    codes over where the quick quotient was a tie that the quotient is not."""
    x, held, missed = near_ties(Dh, Dh)
    assert missed > 100
    n = x.shape[0]
    rows = x.to(DEV).view(1, n, 1, Dh)
    cache = ratp.KVCache(1, 1, Dh, n, 1, kv_bits=4)
    cache.pack(rows, rows.flip(1).contiguous())
    assert np.array_equal(cache.dil_rows("k")[0].cpu().numpy(), held)
    assert np.array_equal(cache.dil_rows("v")[0].cpu().numpy(), held[::-1])
    # gate 0: the new row is the input
    B = 60
    tok = x.to(DEV).view(B, n // B, Dh)
    cache = ratp.KVCache(B, n // B, Dh, 1, 1, kv_bits=4)
    zero = torch.zeros_like(tok)
    cache.decode_step(zero, tok, tok.flip(0).contiguous(), zero, torch.zeros(2, B, n // B, Dh, device=DEV))
    ratp.last_error()
    want = held.reshape(B, n // B, Dh)
    assert np.array_equal(cache.dil_rows("k").cpu().numpy(), want)
    assert np.array_equal(cache.dil_rows("v").cpu().numpy(), want[::-1])
