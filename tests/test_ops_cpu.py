"""The 8-bit transformer operators' entry points without a device: a NULL
handle is refused before anything else, and the handle functions are
NULL-safe."""
import pytest

from dac_vocoder_decoding_amd import vocoder as V


def test_null_handles_are_refused():
    L = V.lib()
    assert L.vocoder_rms_norm(None, 0, 1, 1, None, 1, None, 0, None, 0, None, 0.0, None, 1, None, None) == \
        V.VOC_INVALID_PARAMS
    assert L.vocoder_quantize_rows(None, 0, 1, 1, None, 1, None, 1, None, None) == V.VOC_INVALID_PARAMS
    assert L.vocoder_matmul_int(None, 0, 1, 1, 1, None, 1, None, None, 1, None, None, 0, None, 1, None) == \
        V.VOC_INVALID_PARAMS
    assert L.vocoder_cache_append(None, None, None, 0, None, 0, 0, None, 0, 0, None) == V.VOC_INVALID_PARAMS
    assert L.vocoder_cache_attention(None, None, None, 0, 1, None, 0, 0, 1.0, 0, 0, None, 0, 0, None) == \
        V.VOC_INVALID_PARAMS
    assert L.voc_ops_create(0, None) == V.VOC_INVALID_PARAMS
    assert "NULL" in V.voc_ops_last_error(None)
    V.voc_ops_destroy(None)


def test_half_precision_is_no_decoder_dtype():
    cfg = V.voc_config_default()
    cfg.dtype = V.VOC_F16
    assert V.voc_config_validate(cfg) == V.VOC_INVALID_PARAMS


class OnGpu:
    """As much of a CUDA tensor (device -1: of one on the CPU) as the binding's
    checks look at."""

    def __init__(self, device, shape, dtype):
        import torch
        self._t, self._device = torch.empty(shape, dtype=dtype), device
        self.shape, self.dtype, self.is_cuda = self._t.shape, dtype, device >= 0
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")

    def __getattr__(self, name):
        return getattr(self._t, name)

    def get_device(self):
        return self._device


class Recorder:
    """In the library's place: the calls that would have been launched."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def recorded(monkeypatch):
    V._use_torch()
    library = Recorder()
    monkeypatch.setattr(V, "lib", lambda: library)
    monkeypatch.setattr(V, "_raw_stream", lambda device: 0)
    ops = V.voc_ops(1)
    ops.device = 1
    return ops, library.calls


def operator_calls(ops, place):
    """name -> (number of tensors, call with tensor i on device place(i))."""
    import torch
    f, i8, i32 = torch.float32, torch.int8, torch.int32

    def T(i, shape, dtype=f):
        return OnGpu(place(i), shape, dtype)

    def cache(i):
        return V.KVCache.from_tensors(T(i, (4, 2, 16, 32), i8), T(i, (4, 2, 32, 16), i8), T(i, (4, 2)), T(i, (4, 2)))

    def batch(i):
        return V.KVBatch(T(i, (1, 4), i32), T(i, (1,), i32), T(i, (2,), i32), 3, 3)

    return {
        "rms_norm": (6, lambda: V.rms_norm(ops, T(0, (3, 64)), T(1, (64,)), residual=T(2, (3, 64)), h=T(3, (3, 64)),
                                           q=T(4, (3, 64), i8), scale=T(5, (3,)))),
        "quantize_rows": (3, lambda: V.quantize_rows(ops, T(0, (3, 64)), q=T(1, (3, 64), i8), scale=T(2, (3,)))),
        "matmul_int": (6, lambda: V.matmul_int(ops, T(0, (3, 64), i8), T(1, (3,)), T(2, (5, 64), i8), T(3, (5,)),
                                               bias=T(4, (5,)), out=T(5, (3, 5)))),
        "cache_append": (4, lambda: V.cache_append(ops, cache(0), batch(1), T(2, (3, 2, 32)), T(3, (3, 2, 32)))),
        "cache_attention": (4, lambda: V.cache_attention(ops, cache(0), batch(1), T(2, (3, 4, 32)), out=T(3, (3, 4, 32)))),
    }


@pytest.mark.parametrize("name", ["rms_norm", "quantize_rows", "matmul_int", "cache_append", "cache_attention"])
def test_tensors_on_another_device_are_refused(recorded, name):
    """Every tensor of every call has to be on the handle's device: the kernels
    run there, and another device's memory may not be mapped."""
    ops, calls = recorded
    n, call = operator_calls(ops, lambda i: 1)[name]
    call()
    assert len(calls) == 1                                 # all on the handle's device: launched
    for wrong in range(n):
        for other in (0, 2, -1):
            with pytest.raises(ValueError):
                operator_calls(ops, lambda i: other if i == wrong else 1)[name][1]()
    assert len(calls) == 1


def test_parts_of_a_cache_and_a_batch_are_on_one_device():
    import torch
    T = OnGpu
    with pytest.raises(ValueError):
        V.KVCache.from_tensors(T(0, (4, 2, 16, 32), torch.int8), T(0, (4, 2, 32, 16), torch.int8), T(0, (4, 2), torch.float32),
                               T(1, (4, 2), torch.float32))
    with pytest.raises(ValueError):
        V.KVBatch(T(1, (1, 4), torch.int32), T(0, (1,), torch.int32), T(0, (2,), torch.int32), 3, 3)


@pytest.mark.parametrize("outer,inner", [("append", "attention"), ("attention", "append"), ("append", "append"),
                                         ("attention", "attention")])
def test_threads_may_share_a_batch(monkeypatch, outer, inner):
    """A call that another thread's call on the same batch overtakes, after its
    checks and before the library reads its arguments, keeps its own count of
    packed rows: the kernels take that count for the bound of its tensors."""
    import threading

    import torch
    V._use_torch()
    monkeypatch.setattr(V, "_raw_stream", lambda device: 0)
    cache = V.KVCache.from_tensors(OnGpu(0, (4, 2, 16, 32), torch.int8), OnGpu(0, (4, 2, 32, 16), torch.int8),
                                   OnGpu(0, (4, 2), torch.float32), OnGpu(0, (4, 2), torch.float32))
    batch = V.KVBatch(OnGpu(0, (1, 4), torch.int32), OnGpu(0, (1,), torch.int32), OnGpu(0, (2,), torch.int32), 9, 9)
    seen = {}

    def call(which, tokens):
        x = OnGpu(0, (tokens, 2, 32), torch.float32)
        if which == "append":
            V.cache_append(V.voc_ops(1), cache, batch, x, x)
        else:
            V.cache_attention(V.voc_ops(1), cache, batch, x, out=x)

    class Library:
        def __getattr__(self, name):
            def entry(ops, cache, ref, *args):
                if threading.current_thread() is threading.main_thread():
                    other = threading.Thread(target=call, args=(inner, 3))
                    other.start()
                    other.join()
                seen[threading.current_thread() is threading.main_thread()] = ref._obj.tokens
                return 0
            return entry

    monkeypatch.setattr(V, "lib", Library)
    call(outer, 7)
    assert seen == {True: 7, False: 3}
