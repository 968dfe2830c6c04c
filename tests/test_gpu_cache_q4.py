"""GPU parity of the 4-bit D-compressed cache: the hand-off and the appended
rows hold exactly the definition's values (fp64, numpy), and every decode step
is the fp64 attention over those held values.

Tolerance of a decode output o (bf16): the kernel forms each weight p s from a
bf16 part and the bf16 rest (relative error <= 2^-16, half a step of the rest
is 2^-17), the scores, sums and rescales are fp32 (a score of magnitude <= 16
in log2 units is off by < 2^-16: exp2.approx 2^-22, 128 products at 2^-24 of a
sum that the offset 128 raises up to 2^4 times, 2^-16 in all), so before the
last rounding |o - o64| <= (2^-15 + 2^-15) sum_j p_j |v_j|; the rounding adds
2^-8 |o64| (half a bf16 step is 2^-9 relative to the power of two below, 2^-8
covers it).  The test takes 2^-8 |o64| + 2^-13 max|v|.
"""
import numpy as np
import pytest
import torch

import oracle
import recurrence_augmented_dilated_chunked_b200 as ratp
from recurrence_augmented_dilated_chunked_b200 import prefill_inputs
from recurrence_augmented_dilated_chunked_b200._binding import RatpError
from parity import bits_equal, to64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64)).to(torch.bfloat16).double().numpy()


def held(x):
    """Values that 4 bits a channel stand for (x: [..., Dh] float64 of bf16 values)."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    s = bf16((hi - lo) / 15)
    n = np.clip(np.rint((g - lo) / np.where(s > 0, s, 1)), 0, 15)
    return (lo + np.where(s > 0, n * s, 0)).reshape(x.shape)


class Shadow:
    """fp64 decode over the held values; recurrent rows are the GPU's own."""

    def __init__(self, B, H, Dh, D, W, mask):
        self.B, self.H, self.Dh, self.D, self.W, self.mask = B, H, Dh, D, W, mask
        self.k, self.v = [], []                      # every position's bf16 recurrent row [B, H, Dh]

    def prefill(self, hk, hv):
        self.k += list(to64(hk).transpose(1, 0, 2, 3))
        self.v += list(to64(hv).transpose(1, 0, 2, 3))

    def rows(self, h, n):
        d = 1 if self.mask[h] else self.D
        at = list(range(d - 1, n, d))
        return at, (held(np.stack([self.k[p][:, h] for p in at], 1)) if at else None,
                    held(np.stack([self.v[p][:, h] for p in at], 1)) if at else None)

    def check_rows(self, cache, T_max):
        n = len(self.k)
        got = [cache.dil_rows(w).cpu().double().numpy() for w in "kv"]
        for h in range(self.H):
            off, cap = cache.head_rows(h)
            at, ref = self.rows(h, n)
            for g, r in zip(got, ref):
                if at:
                    # m + n s: n s is exact in fp32 (12 bits), the sum rounds once
                    np.testing.assert_allclose(g[:, off:off + len(at)], r, rtol=2.0 ** -24, atol=0)

    def step(self, q, k_new, v_new):
        """o and sum p |v| bound of the token whose recurrent rows are k_new, v_new."""
        t, o, vmax = len(self.k), np.empty((self.B, self.H, self.Dh)), 0.0
        for h in range(self.H):
            lo = t if self.mask[h] or self.W == 0 else max(0, t - self.W + 1)
            at, (ks, vs) = self.rows(h, lo)
            parts_k = [ks] if at else []
            parts_v = [vs] if at else []
            for p in range(lo, t):
                parts_k.append(self.k[p][:, h][:, None])
                parts_v.append(self.v[p][:, h][:, None])
            parts_k.append(k_new[:, h][:, None])
            parts_v.append(v_new[:, h][:, None])
            K, V = np.concatenate(parts_k, 1), np.concatenate(parts_v, 1)
            s = np.einsum("bd,bkd->bk", q[:, h], K) / np.sqrt(self.Dh)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o[:, h] = np.einsum("bk,bkd->bd", p, V)
            vmax = max(vmax, np.abs(V).max())
        self.k.append(k_new)
        self.v.append(v_new)
        return o, vmax


def assert_token(got, ref, vmax, what):
    g = to64(got)
    assert np.all(np.isfinite(g)), what
    err = np.abs(g - ref) - (2.0 ** -8 * np.abs(ref) + 2.0 ** -13 * vmax)
    assert err.max() <= 0, (what, float(err.max()))


def build(B, H, Dh, T, n, D, W, mask, L=0, window=0, scale=1.0, seed=0, cache_T=None):
    q, xk, xv, g = prefill_inputs(B, T + n, H, Dh, "bf16", gate_mean=1.0, gate_std=2.0, seed=seed)
    xk, xv = xk * scale, xv * scale
    state = torch.zeros(2, B, H, Dh, dtype=torch.float32, device=DEV)
    pre = [x[:, :T].contiguous().to(DEV) for x in (xk, xv, g)]
    cache = ratp.KVCache(B, H, Dh, cache_T or T + n, D, W, head_mask=mask, L=L, kv_bits=4)
    shadow = Shadow(B, H, Dh, D, W, mask)
    if T:
        if window:
            hk, hv = ratp.scan_prefill_kv_window(*pre, window)
        else:
            hk, hv = ratp.scan_prefill_kv(*pre, final_state=state, L=L)
        if window:
            cache.attach_window(window)
        cache.pack(hk, hv)
        if window:
            cache.pack_inputs(*pre)
        shadow.prefill(hk, hv)
    steps = [x[:, T:].contiguous().to(DEV) for x in (q, xk, xv, g)]
    return cache, shadow, state, steps


@pytest.mark.parametrize("B,H,Dh,T,n,D,W,dense", [
    (2, 4, 128, 200, 9, 4, 0, (0,)),
    (2, 2, 128, 131, 18, 16, 16, ()),
    (1, 2, 128, 5, 12, 3, 8, (1,)),
    (3, 2, 64, 300, 5, 64, 128, ()),
    (1, 1, 128, 1, 6, 1, 0, ()),
    (2, 3, 64, 100, 9, 4, 8, (1,)),
    (1, 1, 64, 17, 3, 1, 5, ()),
    (2, 2, 128, 0, 5, 2, 3, (0,)),        # from an empty cache
    (1, 2, 128, 3, 4, 64, 0, ()),         # fewer tokens than one stride: only the token's own key
    (1, 2, 64, 40, 3, 8, 64, ()),         # the window covers everything
    (1, 1, 128, 2500, 2, 1, 0, ()),       # several splits of one head
    (1, 2, 128, 1400, 3, 1, 600, (0,)),   # splits that end inside the ring
])
def test_pack_and_decode_against_held_values(B, H, Dh, T, n, D, W, dense):
    mask = [1 if h in dense else 0 for h in range(H)]
    cache, shadow, state, steps = build(B, H, Dh, T, n, D, W, mask, seed=T + n)
    shadow.check_rows(cache, T + n)
    for i in range(n):
        args = [x[:, i].contiguous() for x in steps]
        out = cache.decode_step(*args, state)
        new = state.to(torch.bfloat16)
        ref, vmax = shadow.step(to64(args[0]), to64(new[0]), to64(new[1]))
        assert_token(out, ref, vmax, "token %d" % i)
        assert cache.lengths().tolist() == [T + i + 1] * B
    ratp.last_error()
    shadow.check_rows(cache, T + n)
    if W:
        for p in range(max(0, T + n - W), T + n):
            assert np.array_equal(to64(cache.ring("k"))[:, :, p % W], shadow.k[p])
            assert np.array_equal(to64(cache.ring("v"))[:, :, p % W], shadow.v[p])
    # full: the next token is refused, and nothing moves
    before = [x.clone() for x in (state, cache.buffer)]
    cache.decode_step(*args, state)
    with pytest.raises(RatpError):
        ratp.last_error()
    assert bits_equal(before[0], state) and bits_equal(before[1], cache.buffer)


@pytest.mark.parametrize("L,window", [(8, 0), (0, 32)])
def test_other_recurrences_continue(L, window):
    cache, shadow, state, steps = build(2, 2, 128, 70, 20, 4, 8, [1, 0], L=L, window=window, seed=7)
    for i in range(20):
        args = [x[:, i].contiguous() for x in steps]
        out = cache.decode_step(*args, state)
        new = state.to(torch.bfloat16)
        ref, vmax = shadow.step(to64(args[0]), to64(new[0]), to64(new[1]))
        assert_token(out, ref, vmax, "token %d" % i)
    ratp.last_error()
    shadow.check_rows(cache, 90)


@pytest.mark.parametrize("scale", [2.0 ** -60, 16.0])
def test_small_and_large_values(scale):
    cache, shadow, state, steps = build(1, 2, 128, 90, 4, 2, 4, [0, 1], scale=scale, seed=11)
    shadow.check_rows(cache, 94)
    for i in range(4):
        args = [x[:, i].contiguous() for x in steps]
        out = cache.decode_step(*args, state)
        new = state.to(torch.bfloat16)
        ref, vmax = shadow.step(to64(args[0]), to64(new[0]), to64(new[1]))
        assert_token(out, ref, vmax, "token %d" % i)
    ratp.last_error()


def test_constant_groups_and_signed_zero_are_held_exactly():
    hk = torch.full((1, 8, 1, 64), -3.5, dtype=torch.bfloat16, device=DEV)
    hv = torch.zeros(1, 8, 1, 64, dtype=torch.bfloat16, device=DEV)
    hv[0, 3, 0, 5] = -1.0
    cache = ratp.KVCache(1, 1, 64, 8, 1, kv_bits=4)
    cache.pack(hk, hv)
    assert torch.equal(cache.dil_rows("k")[0], hk[0, :, 0].float())
    assert torch.equal(cache.dil_rows("v")[0, :, 32:], hv[0, :, 0, 32:].float())
    assert np.array_equal(cache.dil_rows("v").cpu().double().numpy(), held(to64(hv)[:, :, 0]))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), None])
def test_a_group_that_is_not_finite_stands_for_nan(bad):
    """None: finite values further apart than fp32 holds.  The rest of the cache,
    and the heads and channels that do not read the group, are what they are
    without it."""
    B, H, Dh, T = 2, 2, 128, 70
    g = torch.Generator().manual_seed(5)
    hk, hv, q, xk, xv, gate = (torch.randn(B, n, H, Dh, generator=g).to(torch.bfloat16).to(DEV) for n in (T, T, 1, 1, 1, 1))
    args = [x[:, 0].contiguous() for x in (q, xk, xv, gate.sigmoid())]

    def run(k, v):
        cache = ratp.KVCache(B, H, Dh, T + 1, 2, kv_bits=4)
        cache.pack(k, v)
        rows = [cache.dil_rows(w).clone() for w in "kv"]
        return rows, cache.decode_step(*args, torch.zeros(2, B, H, Dh, device=DEV))

    rows0, o0 = run(hk, hv)
    for which in (0, 1):
        x = [hk.clone(), hv.clone()]
        x[which][1, 41, 0, 70] = 3.0e38 if bad is None else bad          # slot 20 of head 0, channels 64 .. 95
        if bad is None:
            x[which][1, 41, 0, 71] = -3.0e38
        rows, o = run(*x)
        hit = [torch.zeros_like(r, dtype=torch.bool) for r in rows]
        hit[which][1, 20, 64:96] = True
        for r, r0, m in zip(rows, rows0, hit):
            assert torch.equal(r[~m], r0[~m])
        assert bool(torch.isnan(rows[which][hit[which]]).all())
        m = torch.zeros_like(o, dtype=torch.bool)
        if which == 0:
            m[1, 0] = True                          # a key's score: the whole head
        else:
            m[1, 0, 64:96] = True                   # a value: its channels
        assert torch.equal(o[~m], o0[~m])
        assert bool(torch.isnan(o[m]).all())
    ratp.last_error()


def test_tensors_of_another_shape_are_refused():
    cache = ratp.KVCache(2, 2, 64, 16, 2, kv_bits=4)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    state = torch.zeros(2, 2, 2, 64, device=DEV)
    prompt = torch.zeros(2, 8, 2, 64, dtype=torch.bfloat16, device=DEV)
    short = x[:1].contiguous()
    for call in (lambda: cache.decode_step(short, x, x, x, state), lambda: cache.decode_step(x, x, x, short, state),
                 lambda: cache.decode_step(x, x, x, x, state[:1].contiguous()),
                 lambda: cache.decode_step(x, x, x, x, state, out=short),
                 lambda: ratp.decode_step_layers([(cache, x, x, short, x, state, x.clone())]),
                 lambda: cache.pack(prompt[:1].contiguous(), prompt), lambda: cache.pack(prompt, prompt, T=9)):
        with pytest.raises(ValueError):
            call()


def test_unequal_lengths_and_repacking():
    """Sequences of a batch at their own lengths, and a cache packed again."""
    B, H, Dh, T, D = 3, 2, 128, 64, 4
    cache, shadow, state, steps = build(B, H, Dh, T, 1, D, 0, [0, 0], seed=3)
    lens = [64, 17, 0]
    cache.lengths().copy_(torch.tensor(lens, dtype=torch.int32, device=DEV))
    args = [x[:, 0].contiguous() for x in steps]
    st = state.clone()
    out = to64(cache.decode_step(*args, st))
    new = [to64(x) for x in st.to(torch.bfloat16)]
    for b, n in enumerate(lens):
        one = Shadow(1, H, Dh, D, 0, [0, 0])
        one.k, one.v = [x[b:b + 1] for x in shadow.k[:n]], [x[b:b + 1] for x in shadow.v[:n]]
        ref, vmax = one.step(to64(args[0])[b:b + 1], new[0][b:b + 1], new[1][b:b + 1])
        assert_token(torch.from_numpy(out[b:b + 1]), ref, vmax, "sequence %d" % b)
    assert cache.lengths().tolist() == [65, 18, 1]
    hk = torch.randn(B, 20, H, Dh, device=DEV).to(torch.bfloat16)
    cache.pack(hk, hk)
    again = Shadow(B, H, Dh, D, 0, [0, 0])
    again.prefill(hk, hk)
    again.check_rows(cache, T + 1)
    assert cache.lengths().tolist() == [20] * B
    ratp.last_error()


def test_layer_stack_of_both_kinds_in_a_replayed_graph():
    """bf16 and 4-bit layers in one token step, captured and replayed; two
    graphs over the same caches in turn."""
    B, H, Dh, T, n = 2, 2, 128, 50, 8
    q, xk, xv, g = prefill_inputs(B, T + n, H, Dh, "bf16", gate_mean=1.0, gate_std=2.0, seed=21)
    st0 = torch.zeros(2, B, H, Dh, dtype=torch.float32, device=DEV)
    hk, hv = ratp.scan_prefill_kv(*[x[:, :T].contiguous().to(DEV) for x in (xk, xv, g)], final_state=st0)
    kinds = [(4, 4, 8), (16, 1, 0), (4, 1, 0)]
    steps = [x[:, T:].contiguous().to(DEV) for x in (q, xk, xv, g)]

    def make():
        caches = [ratp.KVCache(B, H, Dh, T + n, D, W, kv_bits=bits) for bits, D, W in kinds]
        for c in caches:
            c.pack(hk, hv)
        return caches, [st0.clone() for _ in kinds], [torch.empty(B, H, Dh, dtype=torch.bfloat16, device=DEV) for _ in kinds]

    caches, states, outs = make()
    plain = []
    for i in range(n):
        args = [x[:, i].contiguous() for x in steps]
        ratp.decode_step_layers([(c, *args, s, o) for c, s, o in zip(caches, states, outs)])
        plain.append([o.clone() for o in outs])
    c2, s2, o2 = make()
    buf = [torch.empty(B, H, Dh, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            ratp.decode_step_layers([(c, *buf, s, o) for c, s, o in zip(c2, s2, o2)])
        graphs.append(gr)
    for i in range(n):
        for d, x in zip(buf, steps):
            d.copy_(x[:, i])
        graphs[i % 2].replay()
        for o, ref in zip(o2, plain[i]):
            assert bits_equal(o, ref), "token %d" % i
    ratp.last_error()


def test_another_stream():
    cache, shadow, state, steps = build(1, 2, 64, 33, 1, 2, 4, [0, 1], seed=5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    args = [x[:, 0].contiguous() for x in steps]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out = cache.decode_step(*args, state)
        rows = cache.dil_rows("k")
    s.synchronize()
    new = state.to(torch.bfloat16)
    ref, vmax = shadow.step(to64(args[0]), to64(new[0]), to64(new[1]))
    assert_token(out, ref, vmax, "token")
    assert rows.shape == (1, cache.c.rows_per_b, 64)


def test_close_to_the_bf16_cache():
    """Four bits move the output by about their own step, no more: the mean
    difference stays below the mean step of the held rows."""
    B, H, Dh, T = 2, 4, 128, 600
    q, xk, xv, g = (x.to(DEV) for x in prefill_inputs(B, T + 1, H, Dh, "bf16", gate_mean=1.0, gate_std=2.0, seed=9))
    st = torch.zeros(2, B, H, Dh, dtype=torch.float32, device=DEV)
    hk, hv = ratp.scan_prefill_kv(*[x[:, :T].contiguous() for x in (xk, xv, g)], final_state=st)
    outs = []
    for bits in (16, 4):
        cache = ratp.KVCache(B, H, Dh, T + 1, 4, 16, kv_bits=bits)
        cache.pack(hk, hv)
        outs.append(cache.decode_step(*[x[:, T].contiguous() for x in (q, xk, xv, g)], st.clone()).float())
    step = float((hv.float().unflatten(-1, (-1, 32)).amax(-1) - hv.float().unflatten(-1, (-1, 32)).amin(-1)).mean()) / 15
    assert float((outs[0] - outs[1]).abs().mean()) < step
