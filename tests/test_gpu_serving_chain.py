"""The serving operators as they are used together: norm and rotary position,
scan and dilated attention, the 4-bit cache, and a linear-attention layer beside
them -- prefill, then tokens, eager and as one captured graph -- and the new GPU
tests again under the guarded build.

Every stage is held to its own operator's tolerance on what the stage before it
gave (see the operators' own tests)."""
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp
from recurrence_augmented_dilated_chunked_b200 import build as B_
from recurrence_augmented_dilated_chunked_b200 import prefill_inputs
from conftest import ROOT
from parity import assert_close, bits_equal, to64
from test_gpu_cache_q4 import Shadow, assert_token
from test_gpu_linear_attn import check, definition
from test_gpu_norm_rope import check as check_norm
from test_gpu_norm_rope import freqs
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, H, DH, T, N = 2, 4, 128, 150, 6
D, W, MASK = 4, 8, [1, 0, 0, 0]


def _layer():
    q, xk, xv, g = (x.to(DEV) for x in prefill_inputs(B, T + N, H, DH, "bf16", gate_mean=1.0, gate_std=2.0, seed=77))
    gen = torch.Generator().manual_seed(78)
    w = [(1 + 0.2 * torch.randn(DH, generator=gen)).to(DEV) for _ in range(2)]
    ld = torch.tensor([-0.5, -0.05, -0.005, 0.0], device=DEV)
    return q, xk, xv, g, w, freqs(DH).to(DEV), ld


def _prefill(q, xk, xv, g, w, f, ld):
    qn, kn = ratp.qk_norm_rope(q[:, :T], xk[:, :T], w[0], w[1], f)
    state = torch.zeros(2, B, H, DH, device=DEV)
    v = xv[:, :T].contiguous()
    hk, hv = ratp.scan_prefill_kv(kn, v, g[:, :T].contiguous(), final_state=state)
    o = ratp.dilated_attn_prefill(qn, hk, hv, D, W, head_mask=MASK)
    cache = ratp.KVCache(B, H, DH, T + N, D, W, head_mask=MASK, kv_bits=4)
    cache.pack(hk, hv)
    S = torch.empty(B, H, DH, DH, device=DEV)
    lo = ratp.linear_attn_prefill(qn, kn, v, ld, final_state=S)
    return qn, kn, hk, hv, o, lo, state, cache, S


def test_prefill_then_tokens():
    q, xk, xv, g, w, f, ld = _layer()
    qn, kn, hk, hv, o, lo, state, cache, S = _prefill(q, xk, xv, g, w, f, ld)
    ratp.last_error()
    pos = np.broadcast_to(np.arange(T), (B, T))
    check_norm(qn, q[:, :T], w[0], f, pos, False, 1e-6, "q")
    check_norm(kn, xk[:, :T], w[1], f, pos, False, 1e-6, "k")
    assert_close(hk, oracle.scan(to64(kn), to64(g[:, :T])), "bf16", "hk")
    assert_close(o, oracle.attention(to64(qn), to64(hk), to64(hv), D, W, dense_mask=MASK), "bf16", "attention")
    # the whole sequence's normed rows, for the tokens and the linear layer
    qa, ka = ratp.qk_norm_rope(q, xk, w[0], w[1], f)
    check(lo, S, definition(qn, kn, xv[:, :T], ld, None, DH ** -0.5), T, DH, "linear prefill")
    shadow = Shadow(B, H, DH, D, W, MASK)
    shadow.prefill(hk, hv)
    shadow.check_rows(cache, T + N)
    s_ref = S.cpu().double()
    for i in range(N):
        t = T + i
        q1, k1 = ratp.qk_norm_rope(q[:, t], xk[:, t], w[0], w[1], f, positions=cache.lengths())
        assert bits_equal(q1, qa[:, t]) and bits_equal(k1, ka[:, t]), "token %d" % t
        v1, g1 = xv[:, t].contiguous(), g[:, t].contiguous()
        o1 = cache.decode_step(q1, k1, v1, g1, state)
        new = state.to(torch.bfloat16)
        ref, vmax = shadow.step(to64(q1), to64(new[0]), to64(new[1]))
        assert_token(o1, ref, vmax, "token %d" % t)
        l1 = ratp.linear_attn_step(q1, k1, v1, ld, S)
        want = definition(q1[:, None], k1[:, None], v1[:, None], ld, s_ref, DH ** -0.5)
        check(l1[:, None], S, want, 1, DH, "linear token %d" % t)
        s_ref = S.cpu().double()
    shadow.check_rows(cache, T + N)
    ratp.last_error()


def test_a_captured_token_step_equals_the_eager_one():
    """norm -> decode step -> linear step, positions read from the cache's own
    lengths, captured once and replayed for every token."""
    q, xk, xv, g, w, f, ld = _layer()
    runs = []
    for graph in (False, True):
        *_, state, cache, S = _prefill(q, xk, xv, g, w, f, ld)
        buf = [torch.empty(B, H, DH, dtype=torch.bfloat16, device=DEV) for _ in range(6)]     # q, k, v, g, o, lo
        qk = [torch.empty_like(buf[0]) for _ in range(2)]

        def token():
            ratp.qk_norm_rope(buf[0], buf[1], w[0], w[1], f, positions=cache.lengths(), q_out=qk[0], k_out=qk[1])
            cache.decode_step(qk[0], qk[1], buf[2], buf[3], state, out=buf[4])
            ratp.linear_attn_step(qk[0], qk[1], buf[2], ld, S, out=buf[5])

        if graph:
            torch.cuda.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                token()
        outs = []
        for i in range(N):
            for d, x in zip(buf, (q, xk, xv, g)):
                d.copy_(x[:, T + i])
            gr.replay() if graph else token()
            outs += [buf[4].clone(), buf[5].clone()]
        # by now every row of the cache has been written
        runs.append(outs + [state.clone(), S.clone(), cache.dil_rows("k"), cache.dil_rows("v"), cache.ring("k").clone()])
        ratp.last_error()
    for a, b in zip(*runs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_batches_on_two_streams_at_once():
    """Two callers with their own caches and states, interleaved on two streams."""
    q, xk, xv, g, w, f, ld = _layer()
    want, made = [], []
    for _ in range(2):
        *_, state, cache, S = _prefill(q, xk, xv, g, w, f, ld)
        made.append((state, cache, S))
    tok = [x[:, T].contiguous() for x in (q, xk, xv, g)]

    def step(state, cache, S):
        q1, k1 = ratp.qk_norm_rope(tok[0], tok[1], w[0], w[1], f, positions=cache.lengths())
        return cache.decode_step(q1, k1, tok[2], tok[3], state), ratp.linear_attn_step(q1, k1, tok[2], ld, S)

    *_, s0, c0, S0 = _prefill(q, xk, xv, g, w, f, ld)
    want = step(s0, c0, S0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, m in zip(streams, made):
        with torch.cuda.stream(s):
            got.append(step(*m))
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert bits_equal(a, b)
    ratp.last_error()


def test_serving_suite_under_the_guarded_build():
    env = dict(os.environ, RATP_LIBRARY=B_.build_library(guarded=True))
    env["PYTHONPATH"] = ROOT + os.pathsep + env.get("PYTHONPATH", "")
    files = ["tests/test_gpu_norm_rope.py", "tests/test_gpu_cache_q4.py", "tests/test_gpu_linear_attn.py",
             "tests/test_gpu_serving_chain.py"]
    res = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider", "-k",
                          "not guarded_build"] + files, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert res.returncode == 0, "\n".join((res.stdout + res.stderr).splitlines()[-30:])
    m = re.search(r"(\d+) passed", res.stdout)
    assert m and int(m.group(1)) >= 80, res.stdout[-500:]
