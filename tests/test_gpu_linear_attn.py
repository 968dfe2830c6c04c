"""GPU parity of linear attention with a decay per head against the definition
in fp64 (every token against every earlier one; numpy / torch fp64).

Tolerances, per element.  bf16 rounds by at most 2^-8 of the value (half a
step).  Output of a chunked prefill: P = a^{i-j} q_i.k_j and the state enter
their products rounded to bf16, so |o - o64| <= 2^-8 A + 2^-8 |o64| and 2^-20 A
for the fp32 sums and powers, A = scale (sum_{j in chunk} a^{i-j} |q_i.k_j|
|v_j| + a^{i+1} sum_d |q_d| |S_d|).  In the mean square the two roundings are
independent and uniform, at most 2^-8 sqrt(2/3) < 2^-8 of the norm.
State: a^{n-1-j} k_j keeps two bf16 terms (2^-16), 256 products are summed per
chunk (2^-15 if every addition truncates), and a fused multiply-add and a power
of a round once per chunk (2^-23 each chunk): (2^-16 + 2^-15 + (N + 4) 2^-23) of
sum_j a^{T-1-j} |k_j| |v_j| + a^T |S_0|, and 2^-16 of the norm in the mean
square.  Token by token: fp32 throughout, (T + Dh) 2^-23 of the same sums, and
one rounding of o."""
import numpy as np
import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp
from parity import bits_equal, to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
CHUNK = 128
RECURRENT = 16      # sequences up to this long run token by token


def make(B, T, H, Dh, seed, init=True, decays=None):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(B, T, H, Dh, generator=g).to(torch.bfloat16) for _ in range(3))
    if decays is None:
        decays = [-2.0 ** -x for x in np.linspace(1.0, 14.0, H)]
    ld = torch.tensor(decays, dtype=torch.float32)
    s0 = torch.randn(B, H, Dh, Dh, generator=g) * 3 if init else None
    return q, k, v, ld, s0


def power(ld, n):
    """exp(ld * n) for n >= 0 with 0 * -inf = 0."""
    n = np.asarray(n, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        return np.where(n == 0, 1.0, np.exp(np.where(n == 0, 0.0, ld * n)))


def definition(q, k, v, ld, s0, scale):
    """(o, A, final, F): fp64 outputs and the absolute sums of the docstring."""
    q, k, v, ld = to64(q), to64(k), to64(v), to64(ld)
    B, T, H, Dh = q.shape
    o, A = np.zeros(q.shape), np.zeros(q.shape)
    fin, F = np.zeros((B, H, Dh, Dh)), np.zeros((B, H, Dh, Dh))
    at = np.arange(T)
    for b in range(B):
        for h in range(H):
            S = np.zeros((Dh, Dh)) if s0 is None else to64(s0)[b, h]
            F0 = np.abs(S)
            for t0 in range(0, T, CHUNK):
                t1 = min(T, t0 + CHUNK)
                n = t1 - t0
                i = np.arange(n)
                Q, K, V = q[b, t0:t1, h], k[b, t0:t1, h], v[b, t0:t1, h]
                gap = i[:, None] - i[None, :]
                P = (Q @ K.T) * np.where(gap >= 0, power(ld[h], np.maximum(gap, 0)), 0.0)
                ai = power(ld[h], i + 1)[:, None]
                o[b, t0:t1, h] = scale * (P @ V + ai * (Q @ S))
                A[b, t0:t1, h] = abs(scale) * (np.abs(P) @ np.abs(V) + ai * (np.abs(Q) @ np.abs(S)))
                w = power(ld[h], n - 1 - i)[:, None]
                S = power(ld[h], n) * S + (K * w).T @ V
                F0 = power(ld[h], n) * F0 + (np.abs(K) * w).T @ np.abs(V)
            fin[b, h], F[b, h] = S, F0
    # the chunked fp64 form is itself checked against the quadratic definition
    if T <= 300 and B * H <= 8:
        for b in range(B):
            for h in range(H):
                gap = at[:, None] - at[None, :]
                P = (q[b, :, h] @ k[b, :, h].T) * np.where(gap >= 0, power(ld[h], np.maximum(gap, 0)), 0.0)
                ref = P @ v[b, :, h]
                if s0 is not None:
                    ref = ref + power(ld[h], at + 1)[:, None] * (q[b, :, h] @ to64(s0)[b, h])
                np.testing.assert_allclose(o[b, :, h], scale * ref, rtol=1e-9, atol=1e-9)
    return o, A, fin, F


def check(o, fin, ref, T, Dh, what):
    ro, A, rf, F = ref
    go = to64(o)
    assert np.all(np.isfinite(go)), what
    mid = (2.0 ** -8 + 2.0 ** -20) if T > RECURRENT else (T + Dh) * 2.0 ** -23
    err = np.abs(go - ro)
    worst = (err - (mid * A * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ro))).max()
    assert worst <= 1e-30, (what, "o", float(worst))
    assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(ro), (what, "o norm", np.linalg.norm(err) / np.linalg.norm(ro))
    if fin is not None:
        gf = to64(fin)
        N = -(-T // CHUNK)
        tol = 2.0 ** -16 + 2.0 ** -15 + (N + 4) * 2.0 ** -23 if T > RECURRENT else (T + 2) * 2.0 ** -23
        assert (np.abs(gf - rf) - tol * F).max() <= 1e-30, (what, "state", float((np.abs(gf - rf) - tol * F).max()))
        assert np.linalg.norm(gf - rf) <= 2.0 ** -16 * np.linalg.norm(rf), (
            what, "state norm", np.linalg.norm(gf - rf) / np.linalg.norm(rf))


@pytest.mark.parametrize("Dh", [128, 64])
@pytest.mark.parametrize("B,T,H,init", [
    (1, 128, 1, False),
    (2, 128, 2, True),
    (1, 17, 3, True),
    (2, 130, 2, False),
    (1, 300, 3, True),
    (1, 1, 1, False),
    (3, 1, 2, True),
    (2, 16, 2, True),
    (1, 127, 2, True),
    (1, 129, 1, True),
    (1, 1000, 2, True),
    (2, 2049, 1, False),
])
def test_prefill_against_the_definition(B, T, H, Dh, init):
    q, k, v, ld, s0 = make(B, T, H, Dh, seed=B * T + H, init=init)
    fin = torch.full((B, H, Dh, Dh), float("nan"), device=DEV)
    o = ratp.linear_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), ld.to(DEV),
                                 initial_state=s0.to(DEV) if init else None, final_state=fin)
    ratp.last_error()
    check(o, fin, definition(q, k, v, ld, s0, Dh ** -0.5), T, Dh, "prefill")


@pytest.mark.parametrize("Dh", [128, 64])
def test_decays_from_none_to_all(Dh):
    """No decay, a slow one, a fast one, one whose powers underflow inside a
    chunk, and none kept at all."""
    decays = [0.0, -1e-4, -0.7, -40.0, float("-inf")]
    q, k, v, ld, s0 = make(1, 400, 5, Dh, seed=3, decays=decays)
    fin = torch.empty(1, 5, Dh, Dh, device=DEV)
    o = ratp.linear_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), ld.to(DEV), s0.to(DEV), fin, scale=0.25)
    ratp.last_error()
    check(o, fin, definition(q, k, v, ld, s0, 0.25), 400, Dh, "decays")
    st = s0.to(DEV)
    for t in range(3):
        o1 = ratp.linear_attn_step(*[x[:, t].contiguous().to(DEV) for x in (q, k, v)], ld.to(DEV), st, scale=0.25)
    check(o1[:, None], None, [r[:, 2:3] for r in definition(q[:, :3], k[:, :3], v[:, :3], ld, s0, 0.25)[:2]] + [None] * 2,
          3, Dh, "steps")


def test_no_state_in_or_out():
    q, k, v, ld, _ = make(2, 260, 2, 128, seed=4, init=False)
    dev = [x.to(DEV) for x in (q, k, v, ld)]
    fin = torch.empty(2, 2, 128, 128, device=DEV)
    a = ratp.linear_attn_prefill(*dev)
    b = ratp.linear_attn_prefill(*dev, final_state=fin)
    assert bits_equal(a, b)
    zero = torch.zeros_like(fin)
    c = ratp.linear_attn_prefill(*dev, initial_state=zero, final_state=zero)      # in place
    assert bits_equal(a, c) and bits_equal(zero, fin)


def test_steps_and_pieces_continue_a_prefill():
    """A prompt in pieces, then single tokens: each piece starts from the last
    one's state (in place), and every output is the whole sequence's."""
    B, H, Dh = 2, 2, 128
    cuts = [0, 256, 300, 309, 310, 311, 700]
    q, k, v, ld, s0 = make(B, cuts[-1], H, Dh, seed=6)
    whole = definition(q, k, v, ld, s0, Dh ** -0.5)
    st = s0.to(DEV)
    exact, F = s0.double(), np.abs(to64(s0))         # fp64 state at the cut and its absolute sums
    for t0, t1 in zip(cuts, cuts[1:]):
        x = [y[:, t0:t1].contiguous() for y in (q, k, v)]
        d = [y.to(DEV) for y in x]
        if t1 - t0 == 1:
            o = ratp.linear_attn_step(*[y[:, 0].contiguous() for y in d], ld.to(DEV), st)[:, None]
        else:
            o = ratp.linear_attn_prefill(*d, ld.to(DEV), initial_state=st, final_state=st)
        # the piece's own chunks start at t0: its absolute sums are those of the
        # definition started there (not of chunks counted from token 0)
        ro, A, exact_end, F_end = definition(*x, ld, exact, Dh ** -0.5)
        np.testing.assert_allclose(ro, whole[0][:, t0:t1], rtol=1e-9, atol=1e-9)
        # the state handed on is off by at most 2^-14 F (2^-16 + 2^-15 and less than
        # 2^-16 for its additions, decayed since): through q and a^{i+1}
        i = np.arange(t1 - t0)
        ai = np.stack([power(float(l), i + 1) for l in ld], 1)[None, :, :, None]
        handed = 2.0 ** -14 * Dh ** -0.5 * ai * np.einsum("bthd,bhde->bthe", np.abs(to64(x[0])), F)
        mid = (2.0 ** -8 + 2.0 ** -20) if t1 - t0 > RECURRENT else (t1 - t0 + Dh) * 2.0 ** -23
        tol = (mid * A + handed) * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(ro)
        assert (np.abs(to64(o) - ro) - tol).max() <= 0, (t0, t1)
        w = np.stack([power(float(l), t1 - t0) for l in ld])[None, :, None, None]
        kw = np.abs(to64(x[1])) * np.stack([power(float(l), t1 - t0 - 1 - i) for l in ld], 1)[None, :, :, None]
        F = w * F + np.einsum("bthd,bthe->bhde", kw, np.abs(to64(x[2])))
        exact = torch.from_numpy(exact_end)
    gf = to64(st)
    assert np.linalg.norm(gf - whole[2]) <= 2.0 ** -15 * np.linalg.norm(whole[2])
    ratp.last_error()


@pytest.mark.parametrize("B,T,H,Dh", [(1, 128 * 40 + 5, 1, 128), (1, 128 * 150, 1, 64), (3, 128 * 24, 7, 128)])
def test_segments(B, T, H, Dh):
    """Few (b, h) and many chunks: the sequence is cut into segments."""
    assert ratp.linear_attn_workspace_bytes(B, T, H, Dh) > 0
    q, k, v, ld, s0 = make(B, T, H, Dh, seed=T, decays=[-2.0 ** -9] * H)
    fin = torch.empty(B, H, Dh, Dh, device=DEV)
    o = ratp.linear_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), ld.to(DEV), s0.to(DEV), fin)
    ratp.last_error()
    check(o, fin, definition(q, k, v, ld, s0, Dh ** -0.5), T, Dh, "segments")


def test_many_pairs_and_unaligned_output():
    B, T, H, Dh = 40, 40, 8, 64
    q, k, v, ld, s0 = make(B, T, H, Dh, seed=8)
    buf = torch.full((q.numel() + 8,), 5.0, dtype=torch.bfloat16, device=DEV)
    out = buf[8:].view(q.shape)                     # 16-byte, not 32-byte aligned
    fin = torch.empty(B, H, Dh, Dh, device=DEV)
    ratp.linear_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), ld.to(DEV), s0.to(DEV), fin, out=out)
    check(out, fin, definition(q, k, v, ld, s0, Dh ** -0.5), T, Dh, "pairs")
    assert bool((buf[:8] == 5.0).all())


def test_two_graphs_and_streams_do_not_share_a_workspace():
    """Two captured calls of one shape, replayed on two streams at once."""
    B, T, H, Dh = 1, 128 * 32, 1, 128
    ins = [make(B, T, H, Dh, seed=s) for s in (1, 2)]
    dev = [[x.to(DEV) for x in i] for i in ins]
    want = [ratp.linear_attn_prefill(*d[:4], initial_state=d[4]) for d in dev]
    torch.cuda.synchronize()
    graphs, outs = [], [torch.zeros_like(w) for w in want]
    for d, o in zip(dev, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ratp.linear_attn_prefill(*d[:4], initial_state=d[4], out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert bits_equal(o, w)
    ratp.last_error()


def test_step_of_a_full_batch():
    B, H, Dh = 9, 3, 128
    q, k, v, ld, s0 = make(B, 1, H, Dh, seed=11)
    st = s0.to(DEV)
    o = ratp.linear_attn_step(*[x[:, 0].contiguous().to(DEV) for x in (q, k, v)], ld.to(DEV), st)
    check(o[:, None], st, definition(q, k, v, ld, s0, Dh ** -0.5), 1, Dh, "step")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("B,T,H,Dh,at,seen", [
    (1, 128 * 9 + 30, 2, 128, 128 * 4 + 77, True),      # inside a segment's chunk
    (1, 128 * 9 + 30, 2, 64, 128 * 9 + 20, True),       # in the last, ragged chunk
    (2, 200, 1, 128, 127, True),
    (2, 200, 1, 128, 199, False),                       # the last token, its state not asked for
    (1, 11, 1, 64, 5, True),                            # token by token
])
def test_values_that_are_not_finite_leave_the_tokens_before_alone(B, T, H, Dh, at, seen, bad):
    """One channel of v (then of k) at one token, as right padding may hold.
    What it does not reach is bit for bit what it is without it: the products
    with it were with zeros."""
    q, k, v, ld, s0 = (x.to(DEV) for x in make(B, T, H, Dh, seed=12, decays=[-0.01, -0.5][:H]))
    fin0 = torch.zeros(B, H, Dh, Dh, device=DEV)
    o0 = ratp.linear_attn_prefill(q, k, v, ld, s0, fin0)
    b, h, c = B - 1, H - 1, 37
    for which in "vk":
        x = {"v": v, "k": k}[which].clone()
        x[b, at, h, c] = bad
        fin = torch.zeros(B, H, Dh, Dh, device=DEV) if seen else None
        o = ratp.linear_attn_prefill(q, x if which == "k" else k, x if which == "v" else v, ld, s0, fin)
        hit = torch.zeros_like(o, dtype=torch.bool)
        hit[b, at:, h, c if which == "v" else slice(None)] = True
        assert bits_equal(o[~hit], o0[~hit]), which
        assert not bool(torch.isfinite(o[hit].float()).any()), which
        if seen:
            hit = torch.zeros_like(fin, dtype=torch.bool)
            if which == "v":
                hit[b, h, :, c] = True
            else:
                hit[b, h, c, :] = True
            assert bits_equal(fin[~hit], fin0[~hit]), which
            assert not bool(torch.isfinite(fin[hit]).any()), which
    ratp.last_error()


@pytest.mark.parametrize("decay", [0.25, float("nan"), float("inf")])
@pytest.mark.parametrize("T", [1, 300])
def test_a_decay_that_grows_is_reported(T, decay):
    q, k, v, ld, _ = (x.to(DEV) for x in make(1, T, 2, 64, seed=2, decays=[-0.1, decay], init=True))
    ratp.linear_attn_prefill(q, k, v, ld)
    with pytest.raises(ratp.RatpError):
        ratp.last_error()
    ratp.last_error()                               # reported once
    if T == 1:
        ratp.linear_attn_step(q[:, 0], k[:, 0], v[:, 0], ld, torch.zeros(1, 2, 64, 64, device=DEV))
        with pytest.raises(ratp.RatpError):
            ratp.last_error()


def test_no_token_hands_the_state_on():
    q, _, _, ld, s0 = (x.to(DEV) for x in make(2, 20, 2, 64, seed=1))
    none = q[:, :0].contiguous()
    fin = torch.full_like(s0, 3.0)
    ratp.linear_attn_prefill(none, none, none, ld, s0, fin)
    assert bits_equal(fin, s0)
    ratp.linear_attn_prefill(none, none, none, ld, None, fin)
    assert not bool(fin.any())


def test_refusals():
    q, k, v, ld, s0 = (x.to(DEV) for x in make(1, 20, 2, 64, seed=1))
    flat = torch.zeros(4 * q.numel(), dtype=torch.bfloat16, device=DEV)      # an out that begins inside v
    both = [flat[i * q.numel() - (64 if i == 3 else 0):][:q.numel()].view(q.shape) for i in range(4)]
    bad = [
        lambda: ratp.linear_attn_prefill(q.float(), k, v, ld),
        lambda: ratp.linear_attn_prefill(q, k[:, :10], v, ld),
        lambda: ratp.linear_attn_prefill(q.transpose(1, 2), k, v, ld),
        lambda: ratp.linear_attn_prefill(q, k, v, ld.double()),
        lambda: ratp.linear_attn_prefill(q, k, v, ld[:1]),
        lambda: ratp.linear_attn_prefill(q, k, v, ld, initial_state=s0[:, :1]),
        lambda: ratp.linear_attn_prefill(q, k, v, ld, final_state=s0.to(torch.bfloat16)),
        lambda: ratp.linear_attn_prefill(q[0], k[0], v[0], ld),
        lambda: ratp.linear_attn_prefill(q.cpu(), k.cpu(), v.cpu(), ld.cpu()),
        lambda: ratp.linear_attn_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), ld, None),
        lambda: ratp.linear_attn_step(q, k, v, ld, s0),
        lambda: ratp.linear_attn_prefill(q, k, v, ld, out=v),
        lambda: ratp.linear_attn_prefill(*both[:3], ld, out=both[3]),
        lambda: ratp.linear_attn_prefill(q, k, v, ld, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
        lambda: ratp.linear_attn_prefill(q, k, v, ld, workspace=torch.empty(1 << 20, device=DEV)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ratp.linear_attn_prefill(q[..., :32].contiguous(), k[..., :32].contiguous(), v[..., :32].contiguous(), ld),
                 lambda: ratp.linear_attn_prefill(q, k, v, ld, scale=float("inf"))):
        with pytest.raises(ratp.RatpError):
            call()
    empty = q[:, :0].contiguous()
    fin = s0.clone()
    assert ratp.linear_attn_prefill(empty, empty, empty, ld, s0, fin).shape == empty.shape
    assert bits_equal(fin, s0)
