"""Precision of the state that a chunked prefill hands on, against fp64.

a^{n-1-j} k_j enters the products with the 24 bits of an fp32 product (three bf16
terms).  In the mean square over the state: a chunk's 24 products of 16 tokens
each are cut off to fp32, at most a last place 2^-23 of a sum that grows as
sqrt(i), 16 * 2^-23 = 2^-19 of it, as much again for their terms' alignment:
2^-18; the state takes one rounding of at most 2^-24 a chunk, sqrt(N) 2^-24 in N
chunks, and the powers of the decay together at most 2^-22 (one rounding of their
product, one of each weight a^{n-1-j}).  Two terms (16 bits of the decayed keys)
leave about 2^-16.7, a power that is rounded anew each chunk up to N 2^-25."""
import math

import numpy as np
import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp

pytestmark = pytest.mark.gpu
DEV = "cuda"
CHUNK = 128


def exact_state(k, v, ld, s0, cut=None):
    """Sum of a^{T-1-j} k_j v_j^T + a^T s0 in fp64 [B, H, Dh, Dh]; cut: bits that the
    decayed keys of a chunk keep (as a planted loss)."""
    B, T, H, Dh = k.shape
    out = torch.empty(B, H, Dh, Dh, dtype=torch.float64, device=k.device)
    j = torch.arange(T, dtype=torch.float64, device=k.device)
    for b in range(B):
        for h in range(H):
            l = float(ld[h])
            if cut is None:
                kk = torch.exp(l * (T - 1 - j))[:, None] * k[b, :, h].double()
            else:
                last = torch.clamp((j // CHUNK + 1) * CHUNK, max=T) - 1
                w = (torch.exp(l * (last - j))[:, None] * k[b, :, h].double()).float().view(torch.int32)
                kk = (w & ~((1 << (24 - cut)) - 1)).view(torch.float32).double() * torch.exp(l * (T - 1 - last))[:, None]
            out[b, h] = kk.T @ v[b, :, h].double()
            if s0 is not None:
                out[b, h] += math.exp(l * T) * s0[b, h].double()
    return out


def off(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("Dh", [128, 64])
@pytest.mark.parametrize("B,T,H,decays", [
    (2, 300, 3, [-0.3, -0.01, 0.0]),
    (1, 2049, 2, [-2.0 ** -9, -2.0 ** -12]),
    (1, 128 * 150 + 7, 1, [-2.0 ** -16]),           # segments
    (2, 16384, 4, [-2.0 ** -16, -2.0 ** -14, -2.0 ** -10, -2.0 ** -16 * 1.37]),
])
def test_handed_on_state(B, T, H, decays, Dh):
    gen = torch.Generator(device=DEV).manual_seed(T + Dh)
    q, k, v = (torch.randn(B, T, H, Dh, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(3))
    s0 = torch.randn(B, H, Dh, Dh, generator=gen, device=DEV) * 3
    ld = torch.tensor(decays, device=DEV)
    fin = torch.empty_like(s0)
    ratp.linear_attn_prefill(q, k, v, ld, s0, fin)
    ratp.last_error()
    ref = exact_state(k, v, ld, s0)
    tol = 2.0 ** -18 + 2.0 ** -22 + math.sqrt(-(-T // CHUNK)) * 2.0 ** -24
    assert off(fin, ref) <= tol, (off(fin, ref), tol)
    assert off(exact_state(k, v, ld, s0, cut=16), ref) > tol      # two terms would not do


def far_from_fp32(n_tokens, near):
    """The log decay about `near` whose power over n_tokens lies furthest from fp32."""
    c = np.float32(near) * (1 + np.arange(512, dtype=np.float32) / 4096)
    x = np.exp(c.astype(np.float64) * n_tokens)
    return float(c[np.argmax(np.abs(x.astype(np.float32) / x - 1))])


@pytest.mark.parametrize("B,H", [(4, 32), (1, 1)])
def test_an_old_state_decays_by_the_exact_power(B, H):
    """Nothing but an initial state, 1024 chunks: the chunks' powers together are a^T."""
    T, Dh, N = 1 << 17, 64, 1024
    ld = far_from_fp32(CHUNK, -2.0 ** -17)
    x = math.exp(ld * CHUNK)
    drift = N * abs(float(np.float32(x)) / x - 1)
    assert (ratp.linear_attn_workspace_bytes(B, T, H, Dh) == 0) == (B * H == 128)       # one chain, or segments
    zero = torch.zeros(B, T, H, Dh, dtype=torch.bfloat16, device=DEV)
    s0 = torch.randn(B, H, Dh, Dh, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    fin = torch.empty_like(s0)
    ratp.linear_attn_prefill(zero, zero, zero, torch.full((H,), ld, device=DEV), s0, fin)
    ratp.last_error()
    ref = s0.double() * math.exp(ld * T)
    tol = 2.0 ** -22 + math.sqrt(N) * 2.0 ** -24
    assert off(fin, ref) <= tol < drift / 4, (off(fin, ref), tol, drift)
