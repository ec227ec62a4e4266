"""The Python layer of the paged cache compares the devices of caches and tensors: the C side sees addresses only, and a
kernel that is given another device's, or the host's, would fault.  Nothing here reaches a GPU: tensors are stand-ins
that say where they are, and the library's functions record whether they were called."""
import types

import pytest
import torch

import sparse_dimension_attention_b200 as aq
from sparse_dimension_attention_b200 import abi


class OnDevice:
    """As much of a tensor as the wrappers look at."""

    def __init__(self, t, device):
        self.t, self.is_cuda, self.device = t, device >= 0, f"cuda:{device}"
        self.index, self.dtype, self.shape, self.nbytes = device, t.dtype, t.shape, t.nbytes

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.t.is_contiguous()

    def stride(self):
        return self.t.stride()

    def data_ptr(self):
        return self.t.data_ptr()


@pytest.fixture
def calls(monkeypatch):
    seen = []
    names = ("aqua_paged_append", "aqua_paged_decode_attn", "aqua_paged_gather", "aqua_paged_status")
    lib = types.SimpleNamespace(**{n: (lambda *a, n=n: seen.append(n) or abi.AQUA_OK) for n in names})
    abi._torch()
    monkeypatch.setattr(abi, "_lib", lib)
    monkeypatch.setattr(abi, "load_library", lambda path=None: lib)
    monkeypatch.setattr(abi, "_call", lambda fn, dev, stream, *a: fn(*a))
    return seen


def _run(op, cache, dst, dev):
    t = lambda *s, dt=torch.float32: OnDevice(torch.zeros(s, dtype=dt), dev)
    ints = t(2, dt=torch.int32)
    if op == "append":
        aq.aqua_paged_append(cache.desc, t(2, 2, 128), t(2, 2, 128), ints, t(2, 128, 128))
    elif op == "decode":
        aq.aqua_paged_decode_attn(cache.desc, t(2, 4, 128), ints, t(2, 128, 128), 4, 8, t(2, 4, 128), t(64, dt=torch.uint8))
    else:
        aq.aqua_paged_gather(cache.desc, ints, dst.desc, 16)


@pytest.mark.parametrize("op", ["append", "decode", "gather"])
@pytest.mark.parametrize("cache_on,dst_on,tensors_on,fine", [(0, 0, 0, True), (1, 1, 1, True), (1, 0, 0, False),
                                                             (-1, 0, 0, False), (0, 1, 0, False), (0, -1, 0, False),
                                                             (None, None, 0, True)])
def test_devices_are_compared(calls, op, cache_on, dst_on, tensors_on, fine):
    cache, dst = aq.AquaPagedCache(2, 2, 4, 2, device="cpu"), aq.AquaCache(2, 2, 16, device="cpu")
    assert cache.desc.device == -1 and dst.desc.device == -1
    cache.desc.device, dst.desc.device = cache_on, dst_on
    if op != "gather":
        fine = cache_on in (None, tensors_on)
    if fine:
        _run(op, cache, dst, tensors_on)
        assert len(calls) == 1
    else:
        with pytest.raises(aq.AquaError):
            _run(op, cache, dst, tensors_on)
        assert calls == []


def test_status_of_a_cache_on_the_host_is_refused(calls):
    cache = aq.AquaPagedCache(2, 2, 4, 2, device="cpu")
    with pytest.raises(aq.AquaError):
        aq.aqua_paged_status(cache.desc)
    assert calls == []
    cache.desc.device = 1                      # asked of the cache's own device, not of the current one
    assert aq.aqua_paged_status(cache.desc) == 0 and calls == ["aqua_paged_status"]
