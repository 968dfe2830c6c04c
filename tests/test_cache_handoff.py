"""What the hand-offs of a cache read of their tensors, on the CPU: the library is
replaced by one that copies the elements its pointers lead to."""
import ctypes

import pytest
import torch

from recurrence_augmented_dilated_chunked_b200 import _binding

B, H, DH = 2, 3, 64


class Reader:
    """ratp_cache_pack / ratp_cache_pack_inputs, as dense [B, T, H, Dh] reads."""

    def __init__(self):
        self.seen = None

    def read(self, ptrs, T):
        n = B * T * H * DH
        self.seen = [torch.frombuffer((ctypes.c_char * (2 * n)).from_address(p.value or 0), dtype=torch.bfloat16).clone()
                     .view(B, T, H, DH) for p in ptrs]
        return 0

    def ratp_cache_pack(self, c, hk, hv, T, stream):
        return self.read((hk, hv), T)

    def ratp_cache_pack_inputs(self, c, xk, xv, g, T, stream):
        return self.read((xk, xv, g), T)


@pytest.fixture
def cache(monkeypatch):
    lib = Reader()
    monkeypatch.setattr(_binding, "load_library", lambda: lib)
    monkeypatch.setattr(_binding, "_stream", lambda t: None)
    monkeypatch.setattr(_binding, "_on", lambda index: _binding._HERE)

    def need(t, name, dtype=None):
        if not isinstance(t, torch.Tensor) or not t.is_contiguous() or t.dtype != dtype:
            raise ValueError(name)

    monkeypatch.setattr(_binding, "_need", need)
    c = object.__new__(_binding.KVCache)
    c.B, c.H, c.Dh, c._dev, c.buffer, c.c = B, H, DH, -1, torch.empty(0), _binding.CacheStruct()
    c._ref = ctypes.byref(c.c)
    return c, lib


def prompt(n, T, seed, shape=(H, DH)):
    return torch.randn(n, T, H * DH, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).view(n, T, *shape)


@pytest.mark.parametrize("n,length,T", [(2, 9, 9), (2, 9, None), (2, 9, 5), (2, 9, 1), (4, 9, 9), (4, 9, 5)])
@pytest.mark.parametrize("shape", [(H, DH), (H * DH,)])
def test_the_first_tokens_of_each_sequence_are_read(cache, n, length, T, shape):
    c, lib = cache
    x = [prompt(n, length, s, shape) for s in range(3)]
    want = [t[:B, :T].reshape(B, -1, H, DH) for t in x]
    c.pack(x[0], x[1], T)
    assert all(torch.equal(a, b) for a, b in zip(lib.seen, want[:2]))
    c.pack_inputs(*x, T)
    assert all(torch.equal(a, b) for a, b in zip(lib.seen, want))
    # the tensors of a call may differ in length
    c.pack(prompt(n, length, 0, shape), prompt(n, length + 3, 7, shape), length if T is None else T)
    assert torch.equal(lib.seen[1], prompt(n, length + 3, 7, shape)[:B, :length if T is None else T].reshape(B, -1, H, DH))


def test_flat_buffers_are_read_from_their_front(cache):
    c, lib = cache
    x = prompt(B, 6, 3).flatten()
    c.pack(x, x.clone(), 4)
    assert torch.equal(lib.seen[0].flatten(), x[:B * 4 * H * DH])


def test_short_tensors_are_refused(cache):
    c, lib = cache
    full, short, one = prompt(B, 8, 1), prompt(B, 7, 2), prompt(1, 8, 3)
    for bad in (short, one, full.float(), full[:, ::2], None):
        calls = [lambda: c.pack(full, bad), lambda: c.pack_inputs(full, bad, full), lambda: c.pack_inputs(full, full, bad)]
        if bad is not short:                    # it would set T
            calls += [lambda: c.pack(bad, full), lambda: c.pack_inputs(bad, full, full)]
        for call in calls:
            with pytest.raises(ValueError):
                call()
    for call in (lambda: c.pack(full, full, 9), lambda: c.pack_inputs(full, full, full, 9)):
        with pytest.raises(ValueError):
            call()
    assert lib.seen is None
