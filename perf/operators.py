"""Cases, plain forms and calls of the serving operators around the dilated mixer.

Three operators of one layer stack:

* ``norm_rope``: RMS norm of every head of q and k with the rotary position in the same pass;
* ``cache4``: the D-compressed key/value cache held in 4 bits: the prefill hand-off and the decode step
  (recurrence, append, attention) that reads it;
* ``linear``: linear attention with a decay for each head: chunked prefill and the single-token step.

``run`` computes a pass in plain torch (``own = False``) or through the library (``own = True``).
"""
import math

import torch

own = False
DEV = "cuda"
GROUP = 32        # channels that share one minimum and one scale in the 4-bit cache
CHUNK = 128       # tokens a chunk of the plain linear attention
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the queries and keys of one prefill of the 7.6B-like layer
        dict(name="norm_rope_7p6b_t8192", op="norm_rope", B=4, T=8192, H=32, Dh=128, rot=128, dtype="bf16",
             interleaved=False, fused=False, start=0),
        # a later piece of a prompt, read straight out of the fused projection, half the channels rotated in pairs
        dict(name="norm_rope_fused_odd", op="norm_rope", B=3, T=1021, H=16, Dh=128, rot=64, dtype="bf16",
             interleaved=True, fused=True, start=131072),
        # the new token of every sequence of a decode batch, at the length of its context
        dict(name="norm_rope_token", op="norm_rope", B=64, T=0, H=16, Dh=128, rot=128, dtype="bf16",
             interleaved=False, fused=True, start=32768),
        # the fp32 layer
        dict(name="norm_rope_f32", op="norm_rope", B=2, T=3001, H=8, Dh=64, rot=64, dtype="f32",
             interleaved=False, fused=False, start=0),
        # one token of 64 sequences with 32K-token contexts at D = 64 and a window
        dict(name="cache4_step_ctx32k", op="cache4_step", B=64, H=16, Dh=128, t=32768, room=256, D=64, W=128, dense=0),
        # one token of few sequences with many cached rows each (D = 4): the rows are split over CTAs
        dict(name="cache4_step_few_long", op="cache4_step", B=4, H=32, Dh=128, t=32768, room=128, D=4, W=0, dense=0),
        # one token of a small head-wise hybrid: dense heads append a row every step
        dict(name="cache4_step_small_hybrid", op="cache4_step", B=2, H=4, Dh=64, t=1001, room=1, D=4, W=16, dense=1),
        # the hand-off of a finished prefill of the head-wise hybrid layer (2 dense heads, the rest D = 4)
        dict(name="cache4_pack_hybrid", op="cache4_pack", B=4, H=32, Dh=128, t=8192, D=4, W=0, dense=2),
        # a long prompt through a linear-attention layer: few heads, so the sequence is split
        dict(name="linear_prefill_t16k", op="linear", B=2, T=16384, H=16, Dh=128, init=False),
        # the 7.6B-like layer
        dict(name="linear_prefill_7p6b", op="linear", B=4, T=8192, H=32, Dh=128, init=False),
        # a ragged continuation of a prompt from its saved state, small heads
        dict(name="linear_prefill_odd_d64", op="linear", B=3, T=1013, H=5, Dh=64, init=True),
        # the new token of every sequence of a decode batch: the state is read and written
        dict(name="linear_step", op="linear_step", B=64, H=16, Dh=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope", "cache4_step", "cache4_step", "cache4_pack", "linear", "linear",
                     "linear_step"])
    Dh = rng.choice([64, 128, 128])
    H = _log_int(rng, 1, 32)
    B = _log_int(rng, 1, 64)
    if op == "norm_rope":
        T = rng.choice([0, 1]) if rng.random() < 0.25 else _log_int(rng, 2, max(2, 1048576 // (B * H)))
        return dict(op=op, B=B, T=T, H=H, Dh=Dh, rot=rng.choice([Dh, Dh, Dh // 2, 16]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), interleaved=rng.random() < 0.4,
                    fused=rng.random() < 0.5, start=rng.choice([0, rng.randrange(1, 1000000)]))
    if op == "linear":
        T = _log_int(rng, 1, max(1, min(16384, 1048576 // (B * H))))
        return dict(op=op, B=B, T=T, H=H, Dh=Dh, init=rng.random() < 0.5)
    if op == "linear_step":
        return dict(op=op, B=B, H=H, Dh=Dh)
    D = rng.choice([1, 2, 3, 4, 16, 64])
    W = rng.choice([0, 0, 1, 16, 128])
    dense = min(rng.choice([0, 0, 1, 2]), H)
    # a hand-off, and a step that appends a row, return every cached row: up to 400K rows, out of 4M at most
    most = min(4194304, 400000 * (1 if dense else D)) // (B * H)
    t = max(W, D, _log_int(rng, 1, max(1, min(32768, most))))
    if op == "cache4_pack":
        return dict(op=op, B=B, H=H, Dh=Dh, t=t, D=D, W=W, dense=dense)
    return dict(op=op, B=B, H=H, Dh=Dh, t=t, room=1, D=D, W=W, dense=dense)


# ---- inputs -------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _mask(case):
    return [1 if h < case["dense"] else 0 for h in range(case["H"])]


def _quantise(x):
    """bf16 rows [..., Dh] -> (codes uint8 [..., Dh/32, 32], scale, minimum), one scale and minimum a group."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo = g.amin(-1, keepdim=True)
    scale = ((g.amax(-1, keepdim=True) - lo) / 15.0).to(torch.bfloat16).float()
    code = torch.where(scale > 0, ((g - lo) / scale).round().clamp(0, 15), torch.zeros_like(g))
    return code.to(torch.uint8), scale.to(torch.bfloat16), lo.to(torch.bfloat16)


def _values(code, scale, lo):
    return (lo.float() + code.float() * scale.float()).flatten(-2)


def _row_positions(case, n):
    """Positions that the cache keeps of the first n, flattened over heads: (head index, position)."""
    hs, ps = [], []
    for h in range(case["H"]):
        d = 1 if h < case["dense"] else case["D"]
        p = torch.arange(n // d, device=DEV) * d + d - 1
        hs.append(torch.full_like(p, h))
        ps.append(p)
    return torch.cat(hs), torch.cat(ps)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    B, H, Dh = case["B"], case["H"], case["Dh"]
    s = {"case": case}
    if op == "norm_rope":
        dt, T = DT[case["dtype"]], case["T"]
        mid = (B,) if T == 0 else (B, T)
        if case["fused"]:                       # one projection holds q, k and v of a token side by side
            qkv = _randn(g, mid + (3, H, Dh), dt)
            s["q"], s["k"] = qkv[..., 0, :, :], qkv[..., 1, :, :]
        else:
            s["q"], s["k"] = _randn(g, mid + (H, Dh), dt), _randn(g, mid + (H, Dh), dt)
        s["qw"], s["kw"] = (1.0 + _randn(g, (Dh,), torch.float32, 0.1) for _ in range(2))
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])).float()
        s["pos"] = (torch.randint(0, 64, (B,), generator=g, device=DEV) + case["start"]).to(torch.int32)
        return s
    if op in ("linear", "linear_step"):
        mid = (B,) if op == "linear_step" else (B, case["T"])
        s["q"], s["k"], s["v"] = (_randn(g, mid + (H, Dh), torch.bfloat16) for _ in range(3))
        # horizons from 16 tokens (first head) to 64K tokens (last head)
        s["log_decay"] = -torch.exp2(-torch.linspace(4.0, 16.0, H, device=DEV)).float()
        if op == "linear_step" or case["init"]:
            s["state"] = _randn(g, (B, H, Dh, Dh), torch.float32, 4.0)
        return s
    # the recurrent keys and values of a finished prefill
    t = case["t"]
    hk, hv = (_randn(g, (B, t, H, Dh), torch.bfloat16, 0.5) for _ in range(2))
    if op == "cache4_pack":
        s["hk"], s["hv"] = hk, hv
        if own:
            import recurrence_augmented_dilated_chunked_b200 as ratp
            s["cache"] = ratp.KVCache(B, H, Dh, t, case["D"], case["W"], head_mask=_mask(case), kv_bits=4)
        return s
    s["q"], s["xk"], s["xv"] = (_randn(g, (B, H, Dh), torch.bfloat16) for _ in range(3))
    s["g"] = torch.sigmoid(2.0 + _randn(g, (B, H, Dh), torch.float32, 1.5)).to(torch.bfloat16)
    s["state"] = torch.stack([hk[:, -1].float(), hv[:, -1].float()])
    s["len0"] = torch.full((B,), t, dtype=torch.int32, device=DEV)
    T_max = t + case["room"]
    if own:
        import recurrence_augmented_dilated_chunked_b200 as ratp
        s["cache"] = ratp.KVCache(B, H, Dh, T_max, case["D"], case["W"], head_mask=_mask(case), kv_bits=4)
        s["cache"].pack(hk, hv)
        return s
    W = case["W"]
    hs, ps = _row_positions(case, T_max)
    old = torch.where(ps < t, ps, torch.zeros_like(ps))
    s["rows"] = [list(_quantise(x[:, old, hs])) for x in (hk, hv)]
    s["row_head"], s["row_pos"] = hs, ps
    # row of (head, slot), padded with row 0, and which of them there are
    cap = max(1, max(int((hs == h).sum()) for h in range(H)))
    table = torch.zeros(H, cap, dtype=torch.int64, device=DEV)
    there = torch.zeros(H, cap, dtype=torch.bool, device=DEV)
    for h in range(H):
        r = (hs == h).nonzero().flatten()
        table[h, :r.numel()] = r
        there[h, :r.numel()] = True
    s["table"], s["there"] = table, there
    # the last W positions, position p in slot p mod W
    ring_pos = torch.arange(max(0, t - W), t, device=DEV)
    s["ring"] = []
    for x in (hk, hv):
        r = torch.zeros(B, H, W, Dh, dtype=torch.bfloat16, device=DEV)
        if W:
            r[:, :, ring_pos % W] = x[:, ring_pos].transpose(1, 2)
        s["ring"].append(r)
    s["len"] = s["len0"].clone()
    return s


# ---- plain forms --------------------------------------------------------------
def _norm_rope(x, w, cos, sin, rot, interleaved, eps=1e-6):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * w
    r, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1).to(x.dtype)


def _plain_norm_rope(s):
    c = s["case"]
    pos = s["pos"].double()
    if c["T"]:
        pos = pos[:, None] + torch.arange(c["T"], device=DEV, dtype=torch.float64)
    ang = (pos[..., None] * s["inv_freq"].double())[..., None, :]     # far positions: angles in 64 bits
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    return [_norm_rope(x, w, cos, sin, c["rot"], c["interleaved"]) for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"]))]


def _plain_linear(s):
    c = s["case"]
    B, T, H, Dh = c["B"], c["T"], c["H"], c["Dh"]
    scale = Dh ** -0.5
    N = -(-T // CHUNK)
    pad = N * CHUNK - T
    q, k, v = (torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, pad)).view(B, N, CHUNK, H, Dh).permute(0, 3, 1, 2, 4)
               for x in (s["q"], s["k"], s["v"]))                       # [B, H, N, C, Dh]
    ld = s["log_decay"].double()[:, None, None]
    i = torch.arange(CHUNK, device=DEV, dtype=torch.float64)
    diff = i[:, None] - i[None, :]
    near = torch.where(diff >= 0, torch.exp(ld * diff.clamp(min=0)), torch.zeros((), device=DEV, dtype=torch.float64)).float()
    intra = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * near[:, None], v)
    # state that each chunk adds, brought to the chunk's end; then the state before each chunk and after the last
    tail = torch.exp(ld * (CHUNK - 1 - i)[:, None]).float()             # [H, C, 1]
    add = torch.matmul((k * tail[:, None]).transpose(-1, -2), v)        # [B, H, N, Dh, Dh]
    n = torch.arange(N, device=DEV, dtype=torch.float64)
    gap = (n[:, None] - n[None, :] - 1) * CHUNK                         # tokens from the end of chunk m to the start of chunk n
    far = torch.where(gap >= 0, torch.exp(ld * gap.clamp(min=0)), torch.zeros_like(gap)).float()
    states = torch.matmul(far, add.flatten(-2)).unflatten(-1, (Dh, Dh))
    # the last chunk of a ragged sequence ends pad tokens early
    early = torch.exp(ld * (CHUNK - pad - 1 - i).clamp(min=0)[:, None]).float()
    last = torch.matmul((k[:, :, -1] * early).transpose(-1, -2), v[:, :, -1])
    if "state" in s:
        states = states + torch.exp(ld * (n * CHUNK)[:, None]).float()[..., None] * s["state"][:, :, None]
    final = torch.exp(ld * (CHUNK - pad)).float() * states[:, :, -1] + last
    inter = torch.matmul(q, states) * torch.exp(ld * (i[:, None] + 1)).float()[:, None]
    o = ((intra + inter) * scale).permute(0, 2, 3, 1, 4).reshape(B, N * CHUNK, H, Dh)[:, :T]
    return [o.to(torch.bfloat16), final]


def _plain_linear_step(s):
    c = s["case"]
    lam = torch.exp(s["log_decay"].double()).float()[:, None, None]
    s["state"].mul_(lam).add_(s["k"].float()[..., :, None] * s["v"].float()[..., None, :])
    o = (s["q"].float()[..., :, None] * s["state"]).sum(-2) * c["Dh"] ** -0.5
    return [o.to(torch.bfloat16), s["state"]]


def _appends(c):
    return c["dense"] > 0 or c["t"] % c["D"] == c["D"] - 1


def _plain_cache4_step(s):
    c = s["case"]
    B, H, Dh, W, t, D = c["B"], c["H"], c["Dh"], c["W"], c["t"], c["D"]
    s["len"].copy_(s["len0"])
    g = s["g"].float()
    x = torch.stack([s["xk"].float(), s["xv"].float()])
    s["state"].copy_(x + g * (s["state"] - x))
    new = s["state"].to(torch.bfloat16)                                 # [2, B, H, Dh]
    q = s["q"].float() * Dh ** -0.5
    lo = max(0, t - W + 1) if W else t
    wide = torch.arange(H, device=DEV) >= c["dense"]                    # the dilated heads: theirs is the window
    before = torch.where(wide, lo // D, t)                              # cached slots that are attended
    slot = torch.arange(s["table"].shape[1], device=DEV)
    use = s["there"] & (slot[None] < before[:, None])          # [H, cap]
    ks, vs = (_values(*r)[:, s["table"]] for r in s["rows"])            # [B, H, cap, Dh]
    logit = torch.where(use, (q[:, :, None] * ks).sum(-1), torch.full((), -math.inf, device=DEV))
    parts, vals = [logit, (q * new[0].float()).sum(-1, keepdim=True)], [vs, new[1].float()[:, :, None]]
    if W and lo < t:
        at = torch.arange(lo, t, device=DEV) % W
        kr, vr = (r[:, :, at].float() for r in s["ring"])
        parts.append(torch.where(wide[:, None], (q[:, :, None] * kr).sum(-1), torch.full((), -math.inf, device=DEV)))
        vals.append(vr)
    p = torch.cat(parts, -1)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = (p[..., None] * torch.cat(vals, 2)).sum(2).to(torch.bfloat16)
    for r, n in zip(s["ring"], new):
        if W:
            r[:, :, t % W] = n
    out = [o, s["state"], s["len"].add_(1)]
    if W:
        out += s["ring"]
    if _appends(c):                                                     # the new row of every head that keeps position t
        at = (s["row_pos"] == t).nonzero().flatten()
        for r, n in zip(s["rows"], new):
            for held, fresh in zip(r, _quantise(n[:, s["row_head"][at]])):
                held[:, at] = fresh
        out += [_values(*r) for r in s["rows"]]
    return out


def _plain_cache4_pack(s):
    c = s["case"]
    hs, ps = _row_positions(c, c["t"])
    out = [_values(*_quantise(x[:, ps, hs])) for x in (s["hk"], s["hv"])]
    W = c["W"]
    if W:
        at = torch.arange(c["t"] - W, c["t"], device=DEV)
        for x in (s["hk"], s["hv"]):
            r = torch.empty(c["B"], c["H"], W, c["Dh"], dtype=torch.bfloat16, device=DEV)
            r[:, :, at % W] = x[:, at].transpose(1, 2)
            out.append(r)
    return out


# ---- a pass -------------------------------------------------------------------
def _own(s):
    import recurrence_augmented_dilated_chunked_b200 as ratp
    c = s["case"]
    op = c["op"]
    if op == "norm_rope":
        return list(ratp.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["inv_freq"], positions=s["pos"],
                                      interleaved=c["interleaved"]))
    if op == "linear":
        final = torch.empty(c["B"], c["H"], c["Dh"], c["Dh"], dtype=torch.float32, device=DEV)
        o = ratp.linear_attn_prefill(s["q"], s["k"], s["v"], s["log_decay"], initial_state=s.get("state"),
                                     final_state=final)
        return [o, final]
    if op == "linear_step":
        return [ratp.linear_attn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"]), s["state"]]
    cache = s["cache"]
    if op == "cache4_pack":
        cache.pack(s["hk"], s["hv"])
        out = [cache.dil_rows("k"), cache.dil_rows("v")]
        return out + [cache.ring("k"), cache.ring("v")] if c["W"] else out
    cache.lengths().copy_(s["len0"])                                    # the same token again: the cache back at its prompt
    o = cache.decode_step(s["q"], s["xk"], s["xv"], s["g"], s["state"])
    out = [o, s["state"], cache.lengths()]
    if c["W"]:
        out += [cache.ring("k"), cache.ring("v")]
    if _appends(c):
        out += [cache.dil_rows("k"), cache.dil_rows("v")]
    return out


_PLAIN = {"norm_rope": _plain_norm_rope, "linear": _plain_linear, "linear_step": _plain_linear_step,
          "cache4_step": _plain_cache4_step, "cache4_pack": _plain_cache4_pack}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    B, H, Dh = case["B"], case["H"], case["Dh"]
    if op == "norm_rope":
        n = 2 * B * max(1, case["T"]) * H * Dh                          # elements of q and k
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4), "flops": 8 * n}
    if op == "linear":
        T = case["T"]
        n = B * T * H * Dh
        state = B * H * Dh * Dh * 4
        # the recurrence itself: k v^T added to the decayed state, q read against it
        return {"bytes": 4 * n * 2 + state * (2 if case["init"] else 1), "flops": 4 * n * Dh}
    if op == "linear_step":
        return {"bytes": 2 * B * H * Dh * Dh * 4 + 4 * B * H * Dh * 2, "flops": 5 * B * H * Dh * Dh}
    row4 = Dh // 2 + 4 * Dh // GROUP
    t, D, W, dense = case["t"], case["D"], case["W"], case["dense"]
    kept = lambda n: B * (dense * n + (H - dense) * (n // D))           # noqa: E731
    if op == "cache4_pack":
        ring = 2 * 2 * B * H * W * Dh * 2
        return {"bytes": 2 * kept(t) * (2 * Dh + row4 + 4 * Dh) + ring, "flops": 2 * kept(t) * Dh * 4}
    lo = max(0, t - W + 1) if W else t
    rows = B * (dense * t + (H - dense) * (lo // D))
    ring = B * (H - dense) * (t - lo)
    token = B * H * Dh
    size = 2 * rows * row4 + 2 * ring * Dh * 2 + token * (5 * 2 + 2 * 2 * 4) + (2 * token * 2 if W else 0)
    if _appends(case):
        size += 2 * kept(t + 1) * Dh * 4
    return {"bytes": size, "flops": 4 * (rows + ring) * Dh}


# ---- 64 bits ------------------------------------------------------------------
def _exact_norm_rope(s):
    c = s["case"]
    out = []
    pos = s["pos"].to(torch.float64)
    pos = pos if c["T"] == 0 else pos.view(-1, 1) + torch.arange(c["T"], device=DEV).to(torch.float64)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.unsqueeze(-1) * s["inv_freq"].to(torch.float64))
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.to(torch.float64)
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["Dh"] + 1e-6) * w.to(torch.float64)
        r = c["rot"]
        pairs = y[..., :r].reshape(*y.shape[:-1], r // 2, 2) if c["interleaved"] else \
            y[..., :r].reshape(*y.shape[:-1], 2, r // 2).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn.unsqueeze(-2))
        y[..., :r] = (z if c["interleaved"] else z.transpose(-1, -2)).reshape(*y.shape[:-1], r)
        out.append(y)
    return out


def _exact_linear(s):
    c = s["case"]
    B, T, H, Dh = c["B"], c["T"], c["H"], c["Dh"]
    o = torch.empty(B, T, H, Dh, dtype=torch.float64, device=DEV)
    final = torch.empty(B, H, Dh, Dh, dtype=torch.float64, device=DEV)
    at = torch.arange(T, device=DEV, dtype=torch.float64)
    for h in range(H):
        ld = s["log_decay"][h].to(torch.float64)
        w_end = torch.exp(ld * (T - 1 - at))
        for b in range(B):
            q, k, v = (s[n][b, :, h].to(torch.float64) for n in "qkv")
            f = k.t() @ (w_end[:, None] * v)
            if "state" in s:
                f = f + torch.exp(ld * T) * s["state"][b, h].to(torch.float64)
            final[b, h] = f
            for t0 in range(0, T, 4096):                                # every earlier token of 4096 queries at a time
                t1 = min(T, t0 + 4096)
                gap = at[t0:t1, None] - at[None, :t1]
                p = (q[t0:t1] @ k[:t1].t()) * torch.where(gap < 0, 0.0, torch.exp(ld * gap.clamp_(min=0)))
                r = p @ v[:t1]
                if "state" in s:
                    r = r + torch.exp(ld * (at[t0:t1] + 1))[:, None] * (q[t0:t1] @ s["state"][b, h].to(torch.float64))
                o[b, t0:t1, h] = r / math.sqrt(Dh)
    return [o, final]


def _exact_linear_step(s):
    c = s["case"]
    q, k, v = (s[n].to(torch.float64) for n in "qkv")
    S = torch.exp(s["log_decay"].to(torch.float64)).view(-1, 1, 1) * s["state"].to(torch.float64) + torch.einsum("bhi,bhj->bhij", k, v)
    return [torch.einsum("bhi,bhij->bhj", q, S) / math.sqrt(c["Dh"]), S]


def _held(x):
    """The values that 4 bits a channel stand for, from the definition."""
    g = x.to(torch.float64).reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
    s = ((hi - lo) / 15).to(torch.bfloat16).to(torch.float64)
    n = torch.round((g - lo) / torch.where(s > 0, s, torch.ones_like(s))).clamp(0, 15)
    return (lo + n * s).reshape(x.shape)


def _exact_cache4_pack(s):
    c = s["case"]
    out = []
    for x in (s["hk"], s["hv"]):
        rows = []
        for h in range(c["H"]):
            d = 1 if h < c["dense"] else c["D"]
            rows.append(_held(x[:, d - 1::d, h][:, : c["t"] // d]))
        out.append(torch.cat(rows, 1))
    if c["W"]:
        t, W = c["t"], c["W"]
        for x in (s["hk"], s["hv"]):
            r = torch.zeros(c["B"], c["H"], W, c["Dh"], dtype=torch.float64, device=DEV)
            for p in range(t - W, t):
                r[:, :, p % W] = x[:, p].to(torch.float64)
            out.append(r)
    return out


def _exact_cache4_step(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)                                         # the held codes, as plain tensors
    finally:
        own = was
    c = case
    t, W, D, H = c["t"], c["W"], c["D"], c["H"]
    f = lambda x: x.to(torch.float64)                                   # noqa: E731
    g = f(s["g"])
    state = torch.stack([g * f(s["state"][i]) + (1 - g) * f(s[n]) for i, n in enumerate(("xk", "xv"))])
    # the row that joins the cache is the recurrence rounded to bf16; its rounding is that of the 32-bit state
    x = torch.stack([s["xk"].float(), s["xv"].float()])
    new = (x + s["g"].float() * (s["state"] - x)).to(torch.bfloat16)
    kv = [(f(r[2]) + f(r[0]) * f(r[1])).flatten(-2) for r in s["rows"]]
    o = torch.empty(c["B"], H, c["Dh"], dtype=torch.float64, device=DEV)
    for h in range(H):
        dense = h < c["dense"]
        lo = max(0, t - W + 1) if W and not dense else t
        r = ((s["row_head"] == h) & (s["row_pos"] < lo)).nonzero().flatten()
        ks, vs = [kv[0][:, r], f(new[0][:, h:h + 1])], [kv[1][:, r], f(new[1][:, h:h + 1])]
        if lo < t:
            at = torch.arange(lo, t, device=DEV) % W
            ks.append(f(s["ring"][0][:, h, at]))
            vs.append(f(s["ring"][1][:, h, at]))
        p = torch.softmax(torch.einsum("bd,bkd->bk", f(s["q"][:, h]), torch.cat(ks, 1)) / math.sqrt(c["Dh"]), -1)
        o[:, h] = torch.einsum("bk,bkd->bd", p, torch.cat(vs, 1))
    out = [o, state, None]
    if W:
        for r, n in zip(s["ring"], new):
            r = f(r)
            r[:, :, t % W] = f(n)
            out.append(r)
    if _appends(c):
        at = (s["row_pos"] == t).nonzero().flatten()
        for r, n in zip(kv, new):
            r[:, at] = _held(n[:, s["row_head"][at]])
            out.append(r)
    return out


def exact(case, seed):
    if case["op"] == "cache4_step":
        return _exact_cache4_step(case, seed)
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "linear": _exact_linear, "linear_step": _exact_linear_step,
            "cache4_pack": _exact_cache4_pack}[case["op"]](s)
