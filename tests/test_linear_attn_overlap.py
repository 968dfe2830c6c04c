"""Linear attention refuses tensors that overlap what it writes, on the host."""
import ctypes

import pytest
import torch

import recurrence_augmented_dilated_chunked_b200 as ratp
from test_serving_ops_abi import ARG, lib, prefill  # noqa: F401 (lib: fixture)

AT = {name: (i + 1) << 24 for i, name in enumerate(("q", "k", "v", "ld", "init", "fin", "o", "ws"))}
STATE, TOKEN = 128 * 128 * 4, 128 * 2


@pytest.mark.parametrize("T", [3, 40, 16384])
def test_refusals(lib, T):  # noqa: F811
    n = ctypes.c_size_t()
    assert lib.ratp_linear_attn_workspace_bytes(1, T, 1, 128, ctypes.byref(n)) == 0
    ws = dict(ws=AT["ws"], n=n.value) if n.value else {}
    at = {k: v for k, v in AT.items() if k != "ws"}
    for name, where in [("fin", at["init"] + STATE - 16), ("fin", at["init"] - 16), ("fin", at["q"]), ("fin", at["v"] + T * TOKEN - 16),
                        ("fin", at["o"] + 16), ("o", at["k"] + T * TOKEN - 16), ("o", at["init"] + 16), ("o", at["q"])]:
        assert prefill(lib, **dict(at, T=T, **dict(ws, **{name: where}))) == ARG, (name, where)
    if ws:
        for where in (at["init"] + 16, at["fin"] + 16, at["o"] + 16, at["k"]):
            assert prefill(lib, **dict(at, T=T, ws=where, n=n.value)) == ARG


def test_step_refusals(lib):  # noqa: F811
    p = ctypes.c_void_p
    for state, o in ((AT["q"], AT["o"]), (AT["o"] - STATE + 16, AT["o"]), (AT["init"], AT["v"]), (AT["init"], AT["init"] + 64)):
        assert lib.ratp_linear_attn_step(p(AT["q"]), p(AT["k"]), p(AT["v"]), p(AT["ld"]), p(state), p(o), 1, 1, 128, 0.1, 1,
                                         None) == ARG


def test_no_token(lib):  # noqa: F811
    assert prefill(lib, T=0, init=AT["init"], fin=AT["init"] + 16) == ARG


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 2000])
def test_states_that_overlap_in_part(T):
    q = torch.randn(1, T, 1, 64, device="cuda").to(torch.bfloat16)
    ld = torch.full((1,), -0.1, device="cuda")
    flat = torch.zeros(64 * 64 + 4, device="cuda")
    a, b = flat[:-4].view(1, 1, 64, 64), flat[4:].view(1, 1, 64, 64)
    with pytest.raises(ratp.RatpError):
        ratp.linear_attn_prefill(q, q, q, ld, a, b)
    want = ratp.linear_attn_prefill(q, q, q, ld, torch.zeros_like(a))
    assert torch.equal(ratp.linear_attn_prefill(q, q, q, ld, a, a), want)
    ratp.last_error()
