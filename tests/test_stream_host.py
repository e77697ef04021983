"""What an entry point allocates belongs to the stream that it launches on:
an output or a workspace from another stream's pool could be handed out again,
or still be in use there, while the kernels work on it.  On the CPU, with the
library and torch.cuda stood in for: only where the allocations are made is
looked at."""

import contextlib

import pytest

torch = pytest.importorskip("torch")

import compressed_space_attention_b200 as isoq  # noqa: E402
from compressed_space_attention_b200 import binding  # noqa: E402


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class _Cuda:
    """torch.cuda of one device, whose current stream is recorded."""

    Stream = _Stream

    def __init__(self):
        self.now = _Stream(111)

    def current_device(self):
        return 0

    def current_stream(self, dev=None):
        return self.now

    def default_stream(self, dev=None):
        return _Stream(0)

    def ExternalStream(self, handle, device=None):  # noqa: N802
        assert handle != 0
        return _Stream(handle)

    def device(self, dev):
        return contextlib.nullcontext()

    @contextlib.contextmanager
    def stream(self, s):
        before, self.now = self.now, s
        yield
        self.now = before


class _OnDevice(torch.Tensor):
    """A CPU tensor that says it lies on device 0."""

    made = None
    is_cuda = True

    def get_device(self):
        return 0

    def new_empty(self, *a, **k):
        return _OnDevice.made(torch.Tensor.new_empty(self, *a, **k))


class _Torch:
    def __init__(self):
        self.cuda, self.streams, outer = _Cuda(), [], self

        class C:
            @staticmethod
            def _cuda_getCurrentRawStream(index):
                return outer.cuda.now.cuda_stream

        self._C = C
        _OnDevice.made = self._made

    def __getattr__(self, name):
        return getattr(torch, name)

    def _made(self, t):
        self.streams.append(self.cuda.now.cuda_stream)
        return t.as_subclass(_OnDevice)

    def empty(self, *a, **k):
        return self._made(torch.empty(*a, **{**k, "device": "cpu"}))

    def empty_like(self, t, **k):
        return self._made(torch.empty(t.shape, dtype=t.dtype))


class _Lib:
    """Records the stream of each launch; sizes are the library's own."""

    def __init__(self, real):
        self.real, self.streams = real, []

    def __getattr__(self, name):
        if "size" in name or "bytes" in name or "groups" in name:
            return getattr(self.real, name)

        def launch(*a):
            self.streams.append(a[-1])
            return 0
        return launch


def _d(*s, dtype=torch.float16):
    return torch.zeros(s, dtype=dtype).as_subclass(_OnDevice)


def _calls():
    u8, i32, f32 = torch.uint8, torch.int32, torch.float32
    b, hq, hkv, d, t = 2, 8, 2, 128, 8192
    q = _d(b, hq, d)
    cache = [_d(b, hkv, t, 48, dtype=u8), _d(b, hkv, t, 48, dtype=u8), _d(b, hkv, t), _d(b, hkv, t)]
    prefix = [_d(hkv, 64, 48, dtype=u8), _d(hkv, 64, 48, dtype=u8), _d(hkv, 64), _d(hkv, 64)]
    pages = [_d(9, hkv, 16, 48, dtype=u8), _d(9, hkv, 16, 48, dtype=u8), _d(9, hkv, 16), _d(9, hkv, 16)]
    lens, one, table = _d(b, dtype=i32), _d(1, dtype=i32), _d(b, 1024, dtype=i32)
    par = [_d(hkv, 32, 8, dtype=f32)] * 2
    qc, new = _d(b, 4, hq, d), _d(b, hkv, d)
    rotor = _d(hkv, isoq.isoq_rotor_groups(d), 4, dtype=f32)
    rows = isoq.isoq_rotor_packed_bytes(d, 3)
    return {
        "quantize": lambda s: isoq.isoq_quantize(_d(hkv, 5, d), par[0], 3, 0, stream=s),
        "dequantize": lambda s: isoq.isoq_dequantize(_d(hkv, 5, 48, dtype=u8), _d(hkv, 5), par[0], d, 3, 0, stream=s),
        "rotor_quantize": lambda s: isoq.isoq_rotor_quantize(_d(hkv, 5, d), rotor, 3, stream=s),
        "rotor_dequantize": lambda s: isoq.isoq_rotor_dequantize(_d(hkv, 5, rows, dtype=u8), _d(hkv, 5), rotor, d, 3, stream=s),
        "prefill": lambda s: isoq.isoq_prefill_attention(qc, *cache, lens, *par, 3, 0, stream=s),
        "decode": lambda s: isoq.isoq_decode_attention(q, *cache, lens, *par, 3, 0, stream=s),
        "decode_static": lambda s: binding.isoq_decode_attention_static(q, *cache, lens, *par, 3, 0, stream=s),
        "decode_step": lambda s: isoq.isoq_decode_step(q, new, new, *cache, lens, *par, 3, 0, stream=s),
        "window": lambda s: isoq.isoq_decode_attention_window(q, *cache, lens, *par, 3, 0, 8000, stream=s),
        "prefill_window": lambda s: isoq.isoq_prefill_attention_window(qc, *cache, lens, *par, 3, 0, 64, stream=s),
        "prefix": lambda s: isoq.isoq_decode_attention_prefix(q, *prefix, one, *cache, lens, *par, 3, 0, stream=s),
        "tables": lambda s: isoq.isoq_build_block_tables(lens, _d(b, dtype=i32), _d(64, dtype=i32), table, 16, 32, stream=s),
        "paged": lambda s: isoq.isoq_paged_decode_attention(q, *pages, table, lens, *par, 3, 0, stream=s),
    }


@pytest.mark.parametrize("name", list(_calls()))
@pytest.mark.parametrize("given", [None, "torch", "raw", "default"])
def test_allocations_belong_to_the_launch_stream(monkeypatch, name, given):
    fake, fake_lib = _Torch(), _Lib(isoq.lib())
    calls = _calls()
    monkeypatch.setattr(binding, "_torch", lambda: fake)
    monkeypatch.setattr(binding, "lib", lambda: fake_lib)
    stream = {None: None, "torch": _Stream(222), "raw": 222, "default": 0}[given]
    calls[name](stream)
    want = {None: 111, "torch": 222, "raw": 222, "default": 0}[given]
    assert fake_lib.streams == [want]
    assert fake.streams and set(fake.streams) == {want}
    assert fake.cuda.now.cuda_stream == 111
    allocated = {"window": 2, "prefix": 2, "paged": 2, "decode": 2, "decode_step": 2, "tables": 4, "quantize": 2,
                 "rotor_quantize": 2}
    assert len(fake.streams) == allocated.get(name, 1)
