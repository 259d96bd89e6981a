"""The binding's checks of tensors against one another, and the device and stream that it launches on,
without a GPU: tensors that say they are on a device, and a library that records its calls."""

import contextlib

import pytest

torch = pytest.importorskip("torch")
pa = pytest.importorskip("paged_kv_cache_286_gb300")


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on CUDA device `dev`."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    is_cuda = True

    def get_device(self):
        return self.dev


def on(shape, dtype, dev=0):
    t = torch.Tensor._make_subclass(OnDevice, torch.zeros(shape, dtype=dtype))
    t.dev = dev
    return t


class Library:
    def __init__(self, log):
        self.log = log

    def __getattr__(self, name):
        def call(*a):
            self.log.append((name, self.log.device[-1], a[-2] if name == "pa_check_error" else a[-1]))
            return 0
        return call


class Log(list):
    device = None


@pytest.fixture()
def log(monkeypatch):
    log = Log()
    log.device = [0]

    @contextlib.contextmanager
    def device(d):
        log.device.append(d)
        yield
        log.device.pop()

    monkeypatch.setattr(pa._lib, "load", lambda: Library(log))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: log.device[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: device(s.device_index))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    return log


class Stream:
    def __init__(self, dev):
        self.device_index, self.device, self.cuda_stream = dev, f"cuda:{dev}", 77


def step(v=None, dev=0, **kw):
    i32, bf = torch.int32, torch.bfloat16
    k = on((6, 2, 16, 64), bf, dev)
    a = dict(q=on((3, 4, 64), bf, dev), k_cache=k, v_cache=on((6, 2, 16, 64), bf, dev) if v is None else v,
             block_tables=on((2, 3), i32, dev), context_lens=on((2,), i32, dev), query_start_loc=on((3,), i32, dev),
             workspace=on((4096,), torch.uint8, dev), scale=0.1, max_context_len=40, max_query_len=2,
             out=on((3, 4, 64), torch.float32, dev))
    a.update(kw)
    return a


@pytest.mark.parametrize("shape", [(5, 2, 16, 64), (6, 1, 16, 64), (6, 2, 16, 128), (6, 2, 8, 64)])
def test_attention_refuses_pools_of_different_shapes(log, shape):
    """The descriptor comes from the keys: values of another shape would be read past their end."""
    with pytest.raises(ValueError, match="shapes differ"):
        pa.attention(**step(v=on(shape, torch.bfloat16)))
    with pytest.raises(ValueError, match="shapes differ"):
        pa.attention_key_weights(**step(v=on(shape, torch.bfloat16)), key_weights=on((2, 2, 40), torch.float32))
    with pytest.raises(ValueError, match="shapes differ"):
        mx = dict(k_cache=on((6, 2, 544), torch.uint8), v_cache=on((6, 2, 1088), torch.uint8))
        pa.attention(**step(**mx))
    assert log == []


def test_attention_takes_pools_of_one_shape(log):
    pa.attention(**step())
    assert [x[0] for x in log] == ["pa_attention"]
