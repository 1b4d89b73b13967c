"""The binding's streams and devices, on the CPU: host tensors that say they are on a GPU, a library
that notes what it is asked, and stand-ins for torch's current device and stream."""
import contextlib

import pytest
import torch

import io_aware_online_b200 as fa


class Tensor(torch.Tensor):
    """A host tensor on "cuda:1"; notes the streams that it is recorded for."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))

    def get_device(self):
        return 1

    def record_stream(self, stream):
        self.__dict__.setdefault("seen", []).append(stream.cuda_stream)


class Stream:
    def __init__(self, handle, device=torch.device("cuda", 1)):
        self.cuda_stream, self.device = handle, device


class Library:
    """Every entry point: notes (name, current device, stream) and returns 0, or a size."""

    def __init__(self, gpu):
        self.gpu, self.calls = gpu, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.gpu.device, self.gpu.stream.cuda_stream))
            return 256 if name.endswith("workspace_size") else 0
        return call


class GPU:
    def __init__(self):
        self.device, self.stream = 0, Stream(11)

    @contextlib.contextmanager
    def use(self, name, value):
        before = getattr(self, name)
        setattr(self, name, value)
        yield
        setattr(self, name, before)


@pytest.fixture
def gpu(monkeypatch):
    g = GPU()
    g.lib = Library(g)
    monkeypatch.setattr(fa, "load", lambda: g.lib)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: Stream(handle, device))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: g.stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: g.use("stream", s))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: g.device)
    monkeypatch.setattr(torch.cuda, "device", lambda d: g.use("device", d))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: g.stream.cuda_stream, raising=False)
    # host memory in place of the device's
    for name in ("empty", "empty_like"):
        plain = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _f=plain, device=None, **kw: _f(*a, **kw).as_subclass(Tensor))
    monkeypatch.setattr(Tensor, "new_empty", lambda self, shape, dtype=None: torch.empty(shape, dtype=dtype),
                        raising=False)
    return g


def tensor(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(Tensor)


def entry_points():
    """Each call that takes a stream, with its tensors."""
    def rows(*heads):
        return [tensor((2, 3, h, 64), torch.float16) for h in heads]

    def cache():
        return [tensor((4, 64, 2, 64), torch.int8) for _ in "kv"] + [tensor((4, 2, 64), torch.float32) for _ in "kv"]

    def ints(*shape):
        return tensor(shape, torch.int32)

    w = dict(q_weight=tensor((64,), torch.float32), cos=tensor((9, 32), torch.float32),
             sin=tensor((9, 32), torch.float32), positions=ints(2, 3))
    return [
        (fa.fa_qk_norm_rope, rows(4, 2), w),
        (fa.fa_qk_norm_rope_bwd, rows(4, 2, 4, 2), w),
        (fa.fa_kvcache_append_quant, cache() + rows(2, 2) + [ints(2)], dict(block_table=ints(2, 2))),
        (fa.fa_qk_norm_rope_append_quant, rows(4, 2, 2) + cache() + [ints(2)], dict(block_table=ints(2, 2), **w)),
        (fa.fa_kvcache_read_quant, cache() + [ints(3)], dict(block_table=ints(2, 2), total=5)),
        (fa.fa_fwd_kvcache_quant, rows(4) + cache(), dict(block_table=ints(2, 2), cache_seqlens=ints(2))),
    ]


IDS = [f.__name__ for f, _, _ in entry_points()]


@pytest.mark.parametrize("i", range(len(IDS)), ids=IDS)
@pytest.mark.parametrize("as_handle", [False, True])
def test_arguments_outlive_a_call_on_another_stream(gpu, i, as_handle):
    """Whoever frees an argument after the call frees it for work of the current stream: it has to be
    marked as used by the call's stream, as the results are for the current one."""
    fn, args, kw = entry_points()[i]
    result = fn(*args, **kw, stream=22 if as_handle else Stream(22))
    for t in [*args, *kw.values()]:
        if torch.is_tensor(t):
            assert t.__dict__.get("seen") == [22]
    for t in result if isinstance(result, tuple) else (result,):
        if t is not None:
            assert t.__dict__.get("seen") == [11]
    assert gpu.stream.cuda_stream == 11
    assert {c[2] for c in gpu.lib.calls if c[0] == fn.__name__} == {22}


@pytest.mark.parametrize("i", range(len(IDS)), ids=IDS)
def test_the_current_stream_needs_no_marks(gpu, i):
    for kw_stream in ({}, {"stream": Stream(11)}):
        fn, args, kw = entry_points()[i]
        fn(*args, **kw, **kw_stream)
        assert not any("seen" in t.__dict__ for t in [*args, *kw.values()] if torch.is_tensor(t))


@pytest.mark.parametrize("i", range(len(IDS)), ids=IDS)
def test_the_library_is_asked_on_the_tensors_device(gpu, i):
    """Sizes of workspaces depend on the current device's SMs, as the grid does."""
    fn, args, kw = entry_points()[i]
    fn(*args, **kw)
    assert fn.__name__ in [c[0] for c in gpu.lib.calls]
    assert {c[1] for c in gpu.lib.calls} == {1}
    assert gpu.device == 0


def test_strides_outlive_the_table_that_shares_them():
    """A thread that has its strides and is put aside while others fill the table twice over."""
    import ctypes
    mine = [fa._s3(8 * i, 1 << 40, 24 + i) for i in range(50)]
    for i in range(3 * 16384):
        fa._s3(i, 7, 7)
    for i, at in enumerate(mine):
        assert list((ctypes.c_int64 * 3).from_address(int(at))) == [8 * i, 1 << 40, 24 + i]
    assert len(fa._STRIDES) <= 16384
