"""A stand-in for CUDA tensors and streams, so that what the bindings do before a launch can be looked at without a GPU: which
tensors a call makes, on which stream, and which arguments it hands to the library. Nothing is computed."""
import contextlib
import itertools
import math

import torch

_address = itertools.count(1 << 20, 1 << 20)


class Device:
    def __init__(self, index):
        self.type, self.index = ("cuda", index) if index >= 0 else ("cpu", None)


class Stream:
    def __init__(self, name, index=0):
        self.name, self.device, self.cuda_stream, self.waited_for = name, Device(index), next(_address), []

    def wait_stream(self, stream):
        self.waited_for.append(stream)


class Tensor:
    """Shape, strides, type and place of a tensor; `made_on` is the stream that was current when a call made it."""
    requires_grad = False

    def __init__(self, shape, dtype, index=0, strides=None, made_on=None, clear=False):
        self.shape, self.dtype, self.index, self.made_on, self.clear = torch.Size(shape), dtype, index, made_on, clear
        dense = [math.prod(self.shape[i + 1:]) for i in range(len(self.shape))]
        self.strides, self.dense = tuple(dense if strides is None else strides), tuple(dense)
        self.address, self.used_on = next(_address), []

    is_cuda = property(lambda self: self.index >= 0)
    device = property(lambda self: Device(self.index))

    def get_device(self):
        return self.index

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def is_contiguous(self):
        return all(n == 1 or s == d for n, s, d in zip(self.shape, self.strides, self.dense))

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def data_ptr(self):
        return self.address if self.numel() else 0

    def record_stream(self, stream):
        self.used_on.append(stream)


class Cuda:
    """torch.cuda, with a current stream and device of its own."""

    def __init__(self, device=0):
        self.device_index, self.now = device, Stream("current", device)

    def current_stream(self, device=None):
        return self.now

    def current_device(self):
        return self.device_index

    @contextlib.contextmanager
    def stream(self, s):
        before, self.now = self.now, s if s is not None else self.now
        yield
        self.now = before


class Torch:
    """torch, of which tensors are made here; `made` lists them."""

    def __init__(self, device=0):
        self.cuda, self.made = Cuda(device), []

    def __getattr__(self, name):
        return getattr(torch, name)

    def _make(self, shape, dtype, device, strides=None, clear=False):
        index = device.index if isinstance(device, Device) else self.cuda.device_index if device in (None, "cuda") else int(device)
        t = Tensor(shape if not isinstance(shape, int) else (shape,), dtype, index, strides, self.cuda.now, clear)
        self.made.append(t)
        return t

    def empty(self, shape, dtype=None, device=None):
        return self._make(shape, dtype, device)

    def zeros(self, shape, dtype=None, device=None):
        return self._make(shape, dtype, device, clear=True)

    def full(self, shape, value, dtype=None, device=None):
        return self._make(shape, dtype, device, clear=True)

    def empty_like(self, t, memory_format=torch.preserve_format):
        real = torch.empty_like(torch.empty_strided(t.shape, t.strides, dtype=t.dtype), memory_format=memory_format)
        return self._make(t.shape, t.dtype, t.device, real.stride())


class Library:
    """The C library: every call succeeds and is noted with its arguments; sizes are 32 KB."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_size"):
                return 1 << 15
            self.calls.append((name, args))
            return 0
        return call


def install(monkeypatch, sv, device=0):
    """Puts the stand-ins under the package's bindings. Returns (torch, library)."""
    from speculative_decoding_verification_target_gb300 import cache
    t, lib = Torch(device), Library()
    monkeypatch.setattr(sv, "torch", t)
    monkeypatch.setattr(sv, "load", lambda build_if_missing=False: lib)
    monkeypatch.setattr(cache, "torch", t)
    monkeypatch.setattr(cache, "_lib", lambda: lib)
    monkeypatch.setattr(cache, "_raw_stream", None)
    for module in (sv, cache):
        monkeypatch.setattr(module, "_current_device", t.cuda.current_device)
    return t, lib
