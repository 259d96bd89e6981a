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
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: log.device[-1], raising=False)
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


@pytest.mark.parametrize("name", ["block_tables", "context_lens", "workspace", "out"])
def test_what_is_no_tensor_is_refused(log, name):
    with pytest.raises(TypeError):
        pa.attention(**step(**{name: [[1, 2]]}))
    assert log == []


def test_attention_takes_pools_of_one_shape(log):
    pa.attention(**step())
    assert [x[0] for x in log] == ["pa_attention"]


# ---- another device than the current one, and another stream -------------------------------------
def calls(dev, stream=None):
    i64, u8, bf = torch.int64, torch.uint8, torch.bfloat16
    pool = lambda: on((6, 2, 16, 64), bf, dev)  # noqa: E731
    new = lambda: on((3, 2, 64), bf, dev)  # noqa: E731
    pa.cache_append(new(), new(), on((3,), i64, dev), pool(), pool(), on((256,), u8, dev), stream=stream)
    pa.attention(**step(dev=dev), stream=stream)
    pa.attention_key_weights(**step(dev=dev), key_weights=on((2, 2, 40), torch.float32, dev), stream=stream)
    pa.evict_keys(pool(), pool(), *(on(s, torch.int32, dev) for s in ((2, 3), (2,), (2,))),
                  on((2, 2, 40), torch.float32, dev), on((256,), u8, dev), max_context_len=40, max_keep_len=4, recent=1,
                  kept=on((2, 2, 4), torch.int32, dev), new_lens=on((2,), torch.int32, dev), stream=stream)
    pa.check_error(on((256,), u8, dev), stream=stream)


NAMES = ["pa_cache_append", "pa_attention", "pa_attention_key_weights", "pa_evict_keys", "pa_check_error"]


@pytest.mark.parametrize("dev", [0, 1])
def test_calls_run_on_their_tensors_device(log, dev):
    calls(dev)
    assert log == [(name, dev, 1000 + dev) for name in NAMES]
    assert log.device == [0]


def test_calls_run_on_their_streams_device(log):
    calls(1, Stream(1))
    assert log == [(name, 1, 77) for name in NAMES]


@pytest.mark.parametrize("call", range(5))
def test_streams_of_another_device_are_refused(log, call):
    with pytest.raises(ValueError, match="stream of"):
        {0: lambda: pa.cache_append(*[on((3, 2, 64), torch.bfloat16)] * 2, on((3,), torch.int64),
                                    *[on((6, 2, 16, 64), torch.bfloat16)] * 2, on((256,), torch.uint8),
                                    stream=Stream(1)),
         1: lambda: pa.attention(**step(), stream=Stream(1)),
         2: lambda: pa.attention_key_weights(**step(), key_weights=on((2, 2, 40), torch.float32), stream=Stream(1)),
         3: lambda: calls(1, Stream(0)),
         4: lambda: pa.check_error(on((256,), torch.uint8), stream=Stream(1))}[call]()
    assert log == []


@pytest.mark.parametrize("name", ["k_cache", "v_cache", "block_tables", "context_lens", "query_start_loc", "workspace",
                                  "out"])
def test_tensors_on_two_devices_are_refused(log, name):
    args = step()
    args[name] = step(dev=1)[name]
    with pytest.raises(ValueError, match="different devices"):
        pa.attention(**args)
    with pytest.raises(ValueError, match="different devices"):
        pa.attention_key_weights(**args, key_weights=on((2, 2, 40), torch.float32))
    a = [on((3, 2, 64), torch.bfloat16) for _ in range(2)] + [on((3,), torch.int64)] + \
        [on((6, 2, 16, 64), torch.bfloat16) for _ in range(2)] + [on((256,), torch.uint8)]
    for i in range(1, 6):
        b = list(a)
        b[i] = on(tuple(a[i].shape), a[i].dtype, 1)
        with pytest.raises(ValueError, match="different devices"):
            pa.cache_append(*b)
    assert log == []
