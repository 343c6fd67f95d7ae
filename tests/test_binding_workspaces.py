"""Which scratch memory the binding gives a call, without a GPU: the allocator,
the stream lookup and the library's entry point are stand-ins, and the
interleavings that a GPU would leave to chance are forced with barriers."""
import ctypes
import gc
import threading
import types
import weakref

import pytest
import torch

import tests.built  # noqa: F401  (binding loads the library)
from moe_experts_amd import binding

WAIT = 20  # seconds until a barrier gives up


class FakeTorch(types.SimpleNamespace):
    """What the workspace lookup takes from torch, on the CPU."""

    def __init__(self):
        self.uint8, self.device = torch.uint8, torch.device
        self.local = threading.local()  # the current device is a thread's own
        self.capturing = set()     # devices whose current stream is being captured
        self.taken = []            # (bytes, device index) of each allocation
        self._C = types.SimpleNamespace(
            _cuda_getDevice=lambda: self.current,
            _cuda_isCurrentStreamCapturing=lambda: self.current in self.capturing)
        fake = self

        class Device:
            def __init__(self, index):
                self.index = index

            def __enter__(self):
                self.before, fake.current = fake.current, self.index

            def __exit__(self, *exc):
                fake.current = self.before

        self.segments = []  # what the allocator reports of its memory
        self.cuda = types.SimpleNamespace(device=Device, current_device=lambda: self.current,
                                          memory_snapshot=lambda: self.segments)

    @property
    def current(self):
        return getattr(self.local, "index", 0)

    @current.setter
    def current(self, index):
        self.local.index = index

    def empty(self, n, dtype, device):
        self.taken.append((n, device.index))
        return torch.empty(n, dtype=dtype)


@pytest.fixture
def fake(monkeypatch):
    f = FakeTorch()
    monkeypatch.setattr(binding, "torch", f)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 0)
    return f


def in_threads(*work):
    """Runs the functions in a thread each; their results in order."""
    out, errors = [None] * len(work), []

    def go(i, f):
        try:
            out[i] = f()
        except BaseException as e:  # noqa: BLE001 - reported below
            errors.append(e)

    threads = [threading.Thread(target=go, args=(i, f)) for i, f in enumerate(work)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(WAIT)
    assert not errors, errors
    return out


@pytest.mark.parametrize("index", [0, 1])
def test_two_threads_on_one_stream(fake, index):
    """A call enqueues a kernel that leaves partial sums and one that adds them, with the
    interpreter's lock released: another thread's call may come between the two."""
    both = threading.Barrier(2)

    def entry(value):
        def f(ws, nbytes, stream):
            ctypes.memset(ws, value, nbytes)        # the first kernel
            both.wait(WAIT)                         # the other thread's first kernel
            seen = set(ctypes.string_at(ws, nbytes))  # the second kernel
            both.wait(WAIT)
            assert seen == {value}, f"partial sums of {value} were {seen}"
            return 0
        return lambda: binding._run(f, 4096, None, index)

    in_threads(entry(1), entry(2))


def test_two_threads_of_the_calls_that_ask_by_device(fake):
    both = threading.Barrier(2)

    def take():
        ws = binding.workspace(4096, torch.device("cuda", 0))
        both.wait(WAIT)
        return ws

    a, b = in_threads(take, take)
    assert a.data_ptr() != b.data_ptr()


def test_one_thread_keeps_its_buffer(fake):
    first = binding._workspace(4096, 0, 0)
    assert all(binding._workspace(n, 0, 0).data_ptr() == first.data_ptr() for n in (1, 4096, 64))
    assert binding._workspace(4096, 0, 7).data_ptr() != first.data_ptr()  # another stream
    grown = binding._workspace(first.numel() + 1, 0, 0)
    assert grown.numel() > first.numel()
    assert binding._workspace(16, 0, 0).data_ptr() == grown.data_ptr()


@pytest.mark.parametrize("current,asked", [(0, 1), (1, 0)])
def test_a_capture_on_another_device_than_the_current_one(fake, current, asked):
    """Whether a call is captured is asked of the device it runs on."""
    fake.current = current
    eager = binding.workspace(4096, torch.device("cuda", asked))
    assert binding.workspace(4096, torch.device("cuda", asked)) is eager
    fake.capturing = {asked}
    captured = binding.workspace(4096, torch.device("cuda", asked))
    assert captured.data_ptr() != eager.data_ptr() and fake.taken[-1] == (4096, asked)
    fake.capturing = {current}  # a capture that this call is not part of
    assert binding.workspace(4096, torch.device("cuda", asked)) is eager
    assert fake.current == current


@pytest.mark.parametrize("pool,kept", [((1, 0), False), ((0, 7), False), ((0, 0), True),
                                       (None, True)])
def test_memory_of_a_captured_call_lives_as_long_as_its_graph(fake, monkeypatch, pool, kept):
    """A graph's own pool holds the memory of its calls. A capture that was begun otherwise gets
    ordinary memory, which is free for others as soon as nothing refers to it."""
    fake.capturing = {0}
    fake.empty = lambda n, dtype, device: Buffer(n)
    if pool is not None:
        fake.segments = [
            {"device": 0, "address": 1 << 30, "total_size": 1 << 20, "segment_pool_id": (0, 0)},
            {"device": 1, "address": Buffer.AT, "total_size": 1 << 20, "segment_pool_id": (3, 3)},
            {"device": 0, "address": Buffer.AT - 512, "total_size": 1 << 20,
             "segment_pool_id": pool}]
    gone = weakref.ref(binding._workspace(4096, 0, 0))
    gc.collect()
    assert (gone() is not None) == kept


class Buffer:
    AT = 1 << 40

    def __init__(self, n):
        self.n = n

    def data_ptr(self):
        return self.AT

    def numel(self):
        return self.n
