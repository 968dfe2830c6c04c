"""GPU parity of the q/k norm with rotary position against the formula in fp64.

Tolerances: fp32 arithmetic before the last rounding: the mean of squares and
its reciprocal root are within 2^-20 relative (128 products and additions at
2^-24 each, summed in a tree of depth 12, and rsqrt.approx within 2^-22), two
products and the sine's 2^-22 add below 2^-21; so a channel pair of length
|y| = sqrt(u^2 + v^2) is off by at most 2^-19 |y|; the rounding to bf16 adds
at most eps/2 = 2^-8 of the value, to fp32 2^-24."""
import numpy as np
import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp
from parity import bits_equal, to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()


def formula(x, w, inv_freq, pos, interleaved, eps):
    """(y, pair length) in fp64; x [B, T, H, Dh], pos [B, T]."""
    x = to64(x)
    y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * to64(w)
    size = np.abs(y)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    if rot:
        a = pos[:, :, None, None].astype(np.float64) * to64(inv_freq)
        c, s = np.cos(a), np.sin(a)
        lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        u, v = y[..., lo].copy(), y[..., hi].copy()
        y[..., lo], y[..., hi] = u * c - v * s, v * c + u * s
        size[..., lo] = size[..., hi] = np.hypot(u, v)
    return y, size


def check(got, x, w, inv_freq, pos, interleaved, eps, what):
    ref, size = formula(x, w, inv_freq, pos, interleaved, eps)
    g = to64(got)
    assert np.all(np.isfinite(g)), what
    err = np.abs(g - ref) - (HALF[got.dtype] * np.abs(ref) + 2.0 ** -19 * size * (1 + HALF[got.dtype]))
    assert err.max() <= 0, (what, float(err.max()))


def inputs(shape, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * scale).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,Hq,Hk,Dh,rot,interleaved", [
    (2, 37, 4, 4, 128, 128, False),
    (2, 37, 4, 4, 128, 128, True),
    (1, 5, 7, 3, 128, 64, False),
    (3, 1, 5, 1, 64, 64, True),
    (1, 130, 1, 2, 64, 16, False),
    (2, 9, 33, 2, 128, 96, True),
    (2, 9, 3, 3, 64, 48, False),
    (1, 3, 2, 2, 128, 0, False),
])
def test_against_the_formula(B, T, Hq, Hk, Dh, rot, interleaved, dtype):
    q, k = inputs((B, T, Hq, Dh), dtype, 1), inputs((B, T, Hk, Dh), dtype, 2, 30.0)
    qw, kw = 1 + 0.3 * inputs((Dh,), torch.float32, 3), 1 + 0.3 * inputs((Dh,), torch.float32, 4)
    f = freqs(rot).to(DEV) if rot else None
    start = torch.tensor([100000 * b + 17 for b in range(B)], dtype=torch.int32, device=DEV)
    t = np.arange(T)
    per_token = torch.randint(-5, 2 ** 20, (B, T), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    for pos, table in ((None, np.broadcast_to(t, (B, T))), (start, start.cpu().numpy()[:, None] + t),
                       (per_token.to(DEV), per_token.numpy())):
        for w in ((qw, kw), (None, kw)):
            qo, ko = ratp.qk_norm_rope(q, k, w[0], w[1], f, positions=pos, eps=1e-5, interleaved=interleaved)
            assert qo.shape == q.shape and qo.is_contiguous()
            check(qo, q, w[0], f, table, interleaved, 1e-5, "q")
            check(ko, k, w[1], f, table, interleaved, 1e-5, "k")
    ratp.last_error()


def test_positions_at_the_ends_of_int32():
    q = inputs((2, 2, 2, 128), torch.float32, 1)
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31], [0, 2 ** 24 + 1]], dtype=torch.int32, device=DEV)
    f = freqs(128, 500000.0).to(DEV)
    qo, none = ratp.qk_norm_rope(q, None, None, None, f, positions=pos)
    assert none is None
    check(qo, q, None, f, pos.cpu().numpy(), False, 1e-6, "q")
    # an offset whose sum with t passes int32
    start = torch.tensor([2 ** 31 - 1, 5], dtype=torch.int32, device=DEV)
    qo, _ = ratp.qk_norm_rope(q, None, None, None, f, positions=start)
    check(qo, q, None, f, start.cpu().numpy().astype(np.int64)[:, None] + np.arange(2), False, 1e-6, "q")


@pytest.mark.parametrize("scale", [0.0, 1e-12, 1e12])
def test_zero_small_and_large_rows(scale):
    q = inputs((1, 3, 2, 64), torch.float32, 1, scale)
    f = freqs(64).to(DEV)
    qo, ko = ratp.qk_norm_rope(q, q.to(torch.float32), None, None, f)
    check(qo, q, None, f, np.arange(3)[None], False, 1e-6, "q")
    assert bits_equal(qo, ko)


def test_views_of_a_fused_projection_strided_outputs_and_in_place():
    B, T, H, Dh = 2, 11, 3, 128
    f = freqs(Dh).to(DEV)
    qkv = inputs((B, T, 3, H, Dh), torch.bfloat16, 1)
    q, k, v = qkv.unbind(2)
    w = 1 + 0.2 * inputs((Dh,), torch.float32, 2)
    ref = ratp.qk_norm_rope(q.contiguous(), k.contiguous(), w, w, f)
    got = ratp.qk_norm_rope(q, k, w, w, f)
    assert all(bits_equal(a, b) for a, b in zip(ref, got))
    # head-major tensors: [B, H, T, Dh] seen as [B, T, H, Dh], in and out
    hm = [x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (q, k)]
    ho = [torch.full_like(x, 7.0) for x in hm]
    ratp.qk_norm_rope(*hm, w, w, f, q_out=ho[0], k_out=ho[1])
    assert all(bits_equal(a, b) for a, b in zip(ref, ho))
    # every second token of a longer buffer; the tokens between stay as they were
    wide = torch.full((B, 2 * T, H, Dh), 3.0, dtype=torch.bfloat16, device=DEV)
    ratp.qk_norm_rope(q, None, w, None, f, q_out=wide[:, ::2])
    assert bits_equal(wide[:, ::2], ref[0]) and bool((wide[:, 1::2] == 3.0).all())
    # a broadcast input: one batch row for all
    one = q[:1].expand(B, T, H, Dh)
    assert bits_equal(ratp.qk_norm_rope(one, None, w, None, f)[0][1], ref[0][0])
    # in place on the projection: v untouched
    before = v.clone()
    ratp.qk_norm_rope(q, k, w, w, f, q_out=q, k_out=k)
    assert bits_equal(q, ref[0]) and bits_equal(k, ref[1]) and bits_equal(v, before)


def test_a_token_at_the_cache_lengths_equals_prefill():
    """[B, H, Dh] with KVCache.lengths() is the prefill's row at that position,
    however many heads and tokens a launch has."""
    B, T, H, Dh = 3, 40, 5, 128
    q, k = inputs((B, T, H, Dh), torch.bfloat16, 1), inputs((B, T, H, Dh), torch.bfloat16, 2)
    f = freqs(Dh).to(DEV)
    qo, ko = ratp.qk_norm_rope(q, k, None, None, f)
    cache = ratp.KVCache(B, H, Dh, T, 4, kv_bits=4)
    lens = [0, 7, 39]
    cache.lengths().copy_(torch.tensor(lens, dtype=torch.int32, device=DEV))
    at = torch.tensor(lens, device=DEV)
    b = torch.arange(B, device=DEV)
    q1, k1 = ratp.qk_norm_rope(q[b, at], k[b, at], None, None, f, positions=cache.lengths())
    assert bits_equal(q1, qo[b, at]) and bits_equal(k1, ko[b, at])


def test_beyond_2_pow_31_elements_offset():
    """Rows whose offsets pass 32 bits, by strides alone."""
    H, Dh = 1, 64
    big = torch.empty(2 ** 31 + 4096, dtype=torch.bfloat16, device=DEV)
    x = big.as_strided((2, 2, H, Dh), (2 ** 31, 128, 64, 1))
    x.copy_(inputs((2, 2, H, Dh), torch.bfloat16, 1))
    f = freqs(64).to(DEV)
    got, _ = ratp.qk_norm_rope(x, None, None, None, f)
    check(got, x.contiguous(), None, f, np.broadcast_to(np.arange(2), (2, 2)), False, 1e-6, "far rows")
    ratp.last_error()


def test_graph_replay_and_another_stream():
    q, k = inputs((2, 16, 4, 128), torch.bfloat16, 1), inputs((2, 16, 4, 128), torch.bfloat16, 2)
    f = freqs(128).to(DEV)
    ref = ratp.qk_norm_rope(q, k, None, None, f)
    torch.cuda.synchronize()
    outs = [torch.zeros_like(q), torch.zeros_like(k)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ratp.qk_norm_rope(q, k, None, None, f, q_out=outs[0], k_out=outs[1])
    g.replay()
    assert all(bits_equal(a, b) for a, b in zip(ref, outs))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ratp.qk_norm_rope(q, k, None, None, f)
    s.synchronize()
    assert all(bits_equal(a, b) for a, b in zip(ref, got))


def test_refusals_on_the_device_side_of_the_binding():
    q = inputs((1, 4, 2, 128), torch.bfloat16, 1)
    f = freqs(128).to(DEV)
    bad = [
        lambda: ratp.qk_norm_rope(None, None, None, None, f),
        lambda: ratp.qk_norm_rope(q, q.float(), None, None, f),
        lambda: ratp.qk_norm_rope(q, q[:, :2], None, None, f),
        lambda: ratp.qk_norm_rope(q.half(), None, None, None, f),
        lambda: ratp.qk_norm_rope(q.transpose(2, 3), None, None, None, f),
        lambda: ratp.qk_norm_rope(q, None, torch.ones(64, device=DEV), None, f),
        lambda: ratp.qk_norm_rope(q, None, torch.ones(128, device=DEV, dtype=torch.bfloat16), None, f),
        lambda: ratp.qk_norm_rope(q, None, None, None, f.double()),
        lambda: ratp.qk_norm_rope(q, None, None, None, f, positions=torch.zeros(1, dtype=torch.int64, device=DEV)),
        lambda: ratp.qk_norm_rope(q, None, None, None, f, positions=torch.zeros(2, dtype=torch.int32, device=DEV)),
        lambda: ratp.qk_norm_rope(q, None, None, None, f, q_out=torch.empty_like(q[:, :2])),
        lambda: ratp.qk_norm_rope(q.cpu(), None, None, None, f),
        lambda: ratp.qk_norm_rope(q[0, 0], None, None, None, f),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ratp.qk_norm_rope(q, None, None, None, freqs(24).to(DEV)),
                 lambda: ratp.qk_norm_rope(q, None, None, None, freqs(144).to(DEV)),
                 lambda: ratp.qk_norm_rope(q[..., :32], None, None, None, None),
                 lambda: ratp.qk_norm_rope(q, None, None, None, f, eps=-1.0),
                 lambda: ratp.qk_norm_rope(q, None, None, None, f, eps=float("nan")),
                 lambda: ratp.qk_norm_rope(q[..., 4:68], None, None, None, None)):   # rows off 16 bytes
        with pytest.raises(ratp.RatpError):
            call()
    empty = q[:, :0]
    qo, _ = ratp.qk_norm_rope(empty, None, None, None, f)
    assert qo.shape == empty.shape
