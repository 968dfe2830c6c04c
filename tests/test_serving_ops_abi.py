"""CPU checks of the q/k norm, 4-bit cache and linear attention entry points:
refusals happen on the host before any launch, sizes follow the documented
layouts, and the binding refuses host tensors."""
import ctypes
import os
import subprocess

import pytest
import torch

from conftest import ROOT
import recurrence_augmented_dilated_chunked_b200 as ratp
from recurrence_augmented_dilated_chunked_b200 import _binding, build

ARG, SHAPE, ALIGN, CAPACITY, UNSUPPORTED = 1, 2, 3, 4, 7


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return ratp.load_library()


def view(data=4096, sb=1024, st=512, sh=128, heads=2):
    return _binding._VIEW.pack(data, sb, st, sh, heads, 0)


def norm(lib, q=None, k=None, qo=None, ko=None, w=None, f=4096, pos=None, per_token=0, B=1, T=4, Dh=128, rot=128,
         inter=0, eps=1e-6, dtype=1):
    v = view()
    p = lambda x: None if x is None else ctypes.c_void_p(x)
    return lib.ratp_qk_norm_rope(q or v, k or v, qo or v, ko or v, p(w), p(w), p(f), p(pos), per_token, B, T, Dh, rot,
                                 inter, eps, dtype, None)


def test_norm_rope_refusals(lib):
    assert norm(lib, B=-1) == ARG
    assert norm(lib, dtype=2) == ARG
    assert norm(lib, eps=-1.0) == ARG
    assert norm(lib, eps=float("nan")) == ARG
    assert norm(lib, eps=float("inf")) == ARG
    assert norm(lib, f=None) == ARG                       # a rotation without frequencies
    assert norm(lib, q=view(data=0)) == ARG
    assert norm(lib, qo=view(heads=3)) == ARG             # in and out differ in heads
    assert norm(lib, k=view(st=-512)) == ARG
    assert norm(lib, q=view(heads=-1)) == ARG
    assert norm(lib, Dh=96) == SHAPE
    assert norm(lib, rot=24) == SHAPE
    assert norm(lib, rot=144) == SHAPE
    assert norm(lib, rot=-16) == SHAPE
    assert norm(lib, Dh=64, rot=80) == SHAPE
    assert norm(lib, q=view(data=4104)) == ALIGN
    assert norm(lib, ko=view(sh=132)) == ALIGN            # rows off 16 bytes
    assert norm(lib, q=view(sh=66), qo=view(sh=66), k=view(heads=0), ko=view(heads=0), dtype=0) == ALIGN
    assert norm(lib, w=4100) == ALIGN
    assert norm(lib, f=4100) == ALIGN
    assert norm(lib, pos=4098) == ALIGN
    # outputs whose own rows overlap: broadcast tokens, heads closer than a row
    assert norm(lib, qo=view(st=0)) == ARG and norm(lib, ko=view(sh=64)) == ARG and norm(lib, ko=view(st=128)) == ARG
    assert norm(lib, B=2, ko=view(sb=1024)) == ARG        # 4 tokens of 512
    # nothing to do, nothing launched
    assert norm(lib, B=0) == 0 and norm(lib, T=0) == 0
    none = view(data=0, heads=0)
    assert norm(lib, q=none, k=none, qo=none, ko=none) == 0


def test_cache_q4_bytes_and_refusals(lib):
    n, m = ctypes.c_size_t(), ctypes.c_size_t()
    B, H, Dh, T, D, W = 64, 16, 128, 33024, 64, 128
    assert lib.ratp_cache_bytes_q4(B, H, Dh, T, D, W, None, ctypes.byref(n)) == 0
    assert lib.ratp_cache_bytes(B, H, Dh, T, D, W, None, ctypes.byref(m)) == 0
    rows, ring = B * H * (T // D), B * H * W
    held = B * H * (-(-(T // D) // 32) * 32)              # whole blocks of 32 slots
    assert n.value >= 2 * (held * 80 + ring * 256)        # 64 bytes of codes + 16 of parameters; a bf16 ring
    assert n.value < 2 * (held * 80 + ring * 256) + m.value - 2 * (rows + ring) * 256 + (1 << 20)
    assert lib.ratp_cache_bytes_q4(1, 4, 96, 64, 4, 0, None, ctypes.byref(n)) == SHAPE
    assert lib.ratp_cache_bytes_q4(1, 4, 128, 64, 0, 0, None, ctypes.byref(n)) == ARG
    assert lib.ratp_cache_bytes_q4(1, 4, 128, 64, 4, -1, None, ctypes.byref(n)) == ARG
    assert lib.ratp_cache_bytes_q4(1, 4, 128, 64, 4, 0, None, None) == ARG
    c = _binding.CacheStruct()
    p = ctypes.c_void_p(4096)
    assert lib.ratp_cache_init_q4(None, p, 1 << 30, 1, 1, 64, 8, 1, 0, None, None) == ARG
    assert lib.ratp_cache_init_q4(ctypes.byref(c), ctypes.c_void_p(4104), 1 << 30, 1, 1, 64, 8, 1, 0, None, None) == ALIGN
    assert lib.ratp_cache_init_q4(ctypes.byref(c), p, 16, 1, 1, 64, 8, 1, 0, None, None) == CAPACITY
    # reading back is for 4-bit caches
    assert lib.ratp_cache_read_q4(None, p, p, None) == ARG
    assert lib.ratp_cache_read_q4(ctypes.byref(c), p, p, None) == ARG
    c.kv_bits, c.B, c.Dh, c.rows_per_b = 4, 1, 64, 0
    assert lib.ratp_cache_read_q4(ctypes.byref(c), ctypes.c_void_p(4104), None, None) == ALIGN
    assert lib.ratp_cache_read_q4(ctypes.byref(c), p, p, None) == 0          # no rows
    with pytest.raises(ValueError, match="kv_bits"):
        ratp.KVCache(1, 1, 64, 8, 1, kv_bits=8)


def prefill(lib, q=4096, k=4096, v=4096, ld=4096, init=None, fin=None, o=4096, B=1, T=40, H=1, Dh=128, scale=0.1, dtype=1,
            ws=None, n=0):
    p = lambda x: None if x is None else ctypes.c_void_p(x)
    return lib.ratp_linear_attn_prefill(p(q), p(k), p(v), p(ld), p(init), p(fin), p(o), B, T, H, Dh, scale, dtype, p(ws), n,
                                        None)


def test_linear_attention_refusals(lib):
    assert prefill(lib, B=-1) == ARG and prefill(lib, T=-1) == ARG and prefill(lib, H=-1) == ARG
    assert prefill(lib, Dh=96) == SHAPE
    assert prefill(lib, dtype=0) == UNSUPPORTED and prefill(lib, dtype=5) == ARG
    assert prefill(lib, scale=float("inf")) == ARG and prefill(lib, scale=float("nan")) == ARG
    for name in ("q", "k", "v", "ld", "o"):
        assert prefill(lib, **{name: None}) == ARG
    for name in ("q", "k", "v", "o", "init", "fin"):
        assert prefill(lib, **{name: 4104}) == ALIGN
    assert prefill(lib, ld=4098) == ALIGN
    assert prefill(lib, B=1 << 11, H=1 << 10) == SHAPE
    assert prefill(lib, T=0, q=None) == 0 and prefill(lib, B=0) == 0
    n = ctypes.c_size_t()
    assert lib.ratp_linear_attn_workspace_bytes(1, 16384, 1, 128, ctypes.byref(n)) == 0 and n.value > 0
    assert prefill(lib, T=16384) == ARG                                      # needs its workspace
    assert prefill(lib, T=16384, ws=4104, n=n.value) == ALIGN
    assert prefill(lib, T=16384, ws=4096, n=n.value - 1) == CAPACITY
    assert lib.ratp_linear_attn_workspace_bytes(64, 100, 16, 128, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.ratp_linear_attn_workspace_bytes(1, 16, 1, 64, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.ratp_linear_attn_workspace_bytes(1, 16, 1, 32, ctypes.byref(n)) == SHAPE
    assert lib.ratp_linear_attn_workspace_bytes(1, 16, 1, 64, None) == ARG
    p = ctypes.c_void_p(4096)
    step = lambda *a: lib.ratp_linear_attn_step(*a, None)
    assert step(p, p, p, p, None, p, 1, 1, 64, 0.1, 1) == ARG
    assert step(p, p, p, p, ctypes.c_void_p(4100), p, 1, 1, 64, 0.1, 1) == ALIGN
    assert step(p, p, p, p, p, p, 1, 1, 72, 0.1, 1) == SHAPE
    assert step(p, p, p, p, p, p, 1, 1, 64, 0.1, 0) == UNSUPPORTED
    assert step(None, None, None, None, None, None, 0, 1, 64, 0.1, 1) == 0


def test_segment_plans_stay_in_bounds(lib):
    """Every plan's workspace is whole segments of whole states, at most 256 a sequence."""
    n = ctypes.c_size_t()
    for B, T, H, Dh in [(1, 17, 1, 64), (1, 129, 1, 128), (1, 10 ** 6, 1, 128), (2, 16384, 16, 128), (3, 5000, 7, 64),
                        (1, 2 ** 31 - 1, 1, 64), (512, 4096, 2, 128)]:
        assert lib.ratp_linear_attn_workspace_bytes(B, T, H, Dh, ctypes.byref(n)) == 0
        state = B * H * Dh * Dh * 4
        assert n.value % state == 0 and n.value // state != 1
        assert n.value // state <= min(256, -(-T // 128))


def test_host_tensors_are_refused():
    x4, x3 = torch.zeros(1, 8, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    f, ld, s = torch.ones(32), torch.zeros(1), torch.zeros(1, 1, 64, 64)
    for call in (lambda: ratp.qk_norm_rope(x4, x4, None, None, f), lambda: ratp.qk_norm_rope(None, None, None, None, f),
                 lambda: ratp.linear_attn_prefill(x4, x4, x4, ld), lambda: ratp.linear_attn_step(x3, x3, x3, ld, s)):
        with pytest.raises(ValueError):
            call()


def test_view_and_cache_structs_have_the_c_sizes(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ratp.h"\n'
                   'int main(void) { printf("%zu %zu %zu %zu\\n", sizeof(ratp_view), offsetof(ratp_view, heads), '
                   'sizeof(ratp_cache), offsetof(ratp_cache, kv_bits)); return 0; }\n')
    exe = tmp_path / "sizes"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert got == [_binding._VIEW.size, 32, ctypes.sizeof(_binding.CacheStruct), _binding.CacheStruct.kv_bits.offset]
