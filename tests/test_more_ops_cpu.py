"""Head norms with rotation, the cache read back and the adapters beside the
8-bit product: the entry points and the binding's checks without a device."""
import pytest
import torch

from dac_vocoder_decoding_amd import vocoder as V
from test_ops_cpu import OnGpu, recorded  # noqa: F401 (a fixture)


def test_null_handles_are_refused():
    L = V.lib()
    assert L.vocoder_norm_rotate(None, 0, 1, 64, None, None, 0, 0, 0.0, *[1, None, 64, 64, None, None, 64, 64] * 2, None) == \
        V.VOC_INVALID_PARAMS
    assert L.vocoder_norm_rotate_append(None, None, None, 0, None, 0, 0, 0.0, 1, None, 0, 0, None, None, 0, 0, None, 0, 0, None,
                                        None, 0, 0, None) == V.VOC_INVALID_PARAMS
    assert L.vocoder_cache_read(None, None, None, 0, None, 0, 0, None, 0, 0, None) == V.VOC_INVALID_PARAMS
    assert L.vocoder_matmul_int_adapters(None, 0, 1, 1, 1, None, 1, None, None, 1, None, None, 0, None, None, None, 1, None) == \
        V.VOC_INVALID_PARAMS


class Held:
    """In the place of Adapters, whose constructor lays tensors out on a device."""

    def __init__(self, device):
        self.device, self.K, self.N, self.ref = device, 64, 5, None
        self.down = OnGpu(device, (1, 16, 64), torch.float16)
        self.tensors = ()


def calls(ops, place):
    """name -> (number of tensors, call with tensor i on device place(i))."""
    f, i8, i32 = torch.float32, torch.int8, torch.int32

    def T(i, shape, dtype=f):
        return OnGpu(place(i), shape, dtype)

    def cache(i):
        return V.KVCache.from_tensors(T(i, (4, 2, 16, 32), i8), T(i, (4, 2, 32, 16), i8), T(i, (4, 2)), T(i, (4, 2)))

    def batch(i):
        return V.KVBatch(T(i, (1, 4), i32), T(i, (1,), i32), T(i, (2,), i32), 3, 3)

    return {
        "norm_rotate": (8, lambda: V.norm_rotate(ops, T(0, (3, 4, 32)), T(1, (3, 2, 32)), position=T(2, (3,), i32), freq=T(3, (16,)),
                                                 q_weight=T(4, (32,)), k_weight=T(5, (32,)), q_out=T(6, (3, 4, 32)),
                                                 k_out=T(7, (3, 2, 32)))),
        "norm_rotate_append": (9, lambda: V.norm_rotate_append(
            ops, cache(0), batch(1), T(2, (3, 4, 32)), T(3, (3, 2, 32)), T(4, (3, 2, 32)), freq=T(5, (16,)), q_weight=T(6, (32,)),
            k_weight=T(7, (32,)), out=T(8, (3, 4, 32)))),
        "cache_read": (4, lambda: V.cache_read(ops, cache(0), batch(1), 3, k=T(2, (3, 2, 32)), v=T(3, (3, 2, 32)))),
        "matmul_int_adapters": (8, lambda: V.matmul_int_adapters(
            ops, T(0, (3, 64), i8), T(1, (3,)), T(2, (5, 64), i8), T(3, (5,)), Held(place(4)), T(5, (3,), i32), bias=T(6, (5,)),
            out=T(7, (3, 5)))),
    }


@pytest.mark.parametrize("name", ["norm_rotate", "norm_rotate_append", "cache_read", "matmul_int_adapters"])
def test_tensors_on_another_device_are_refused(recorded, name):  # noqa: F811
    ops, launched = recorded
    n, call = calls(ops, lambda i: 1)[name]
    call()
    assert len(launched) == 1
    for wrong in range(n):
        for other in (0, 2, -1):
            with pytest.raises(ValueError):
                calls(ops, lambda i: other if i == wrong else 1)[name][1]()
    assert len(launched) == 1


def test_shapes_that_do_not_fit_are_refused(recorded):  # noqa: F811
    ops, launched = recorded
    f, i8, i32 = torch.float32, torch.int8, torch.int32

    def T(shape, dtype=f):
        return OnGpu(1, shape, dtype)

    q, k = T((3, 4, 32)), T((3, 2, 32))
    cache = V.KVCache.from_tensors(T((4, 2, 16, 32), i8), T((4, 2, 32, 16), i8), T((4, 2)), T((4, 2)))
    batch = V.KVBatch(T((1, 4), i32), T((1,), i32), T((2,), i32), 3, 3)
    ids, a = T((3,), i32), T((3, 64), i8)
    for call in (
            lambda: V.norm_rotate(ops, q, q_out=q, freq=T((16,))),                                         # no positions
            lambda: V.norm_rotate(ops, q, q_out=q, position=ids, freq=T((17,))),
            lambda: V.norm_rotate(ops, q, q_out=q, position=T((2,), i32), freq=T((16,))),
            lambda: V.norm_rotate(ops, q, q_out=q, position=T((3,)), freq=T((16,))),
            lambda: V.norm_rotate(ops, q, q_out=q, q_weight=T((31,))),
            lambda: V.norm_rotate(ops, q, T((3, 2, 16)), q_out=q),
            lambda: V.norm_rotate(ops, q, T((2, 2, 32)), q_out=q),
            lambda: V.norm_rotate(ops, q, T((3, 2, 32), torch.float16), q_out=q),
            lambda: V.norm_rotate(ops, q, q_out=k),
            lambda: V.norm_rotate(ops, T((3, 32)), q_out=q),
            lambda: V.norm_rotate_append(ops, cache, batch, q, k, T((3, 3, 32)), out=q),
            lambda: V.norm_rotate_append(ops, cache, batch, T((2, 4, 32)), k, k, out=q),
            lambda: V.norm_rotate_append(ops, cache, batch, q, k, k, freq=T((17,)), out=q),
            lambda: V.norm_rotate_append(ops, cache, batch, q, k, k, out=T((3, 4, 64))),
            lambda: V.cache_read(ops, cache, batch, 3, k=T((3, 2, 64)), v=k),
            lambda: V.cache_read(ops, cache, batch, 3, k=k, v=T((3, 2, 32), torch.float16)),
            lambda: V.cache_read(ops, cache, batch, 4, k=k, v=k),
            lambda: V.cache_read(ops, cache, batch, 3, dtype=torch.float64, k=k, v=k),
            lambda: V.matmul_int_adapters(ops, a, T((3,)), T((6, 64), i8), T((6,)), Held(1), ids, out=T((3, 6))),
            lambda: V.matmul_int_adapters(ops, a, T((3,)), T((5, 64), i8), T((5,)), Held(1), T((2,), i32), out=T((3, 5))),
            lambda: V.matmul_int_adapters(ops, a, T((3,)), T((5, 64), i8), T((5,)), Held(1), T((3,)), out=T((3, 5)))):
        with pytest.raises(ValueError):
            call()
    assert not launched
    V.norm_rotate(ops, q, k, position=ids, freq=T((16,)), q_out=q, k_out=k)
    assert [name for name, _ in launched] == ["vocoder_norm_rotate"]


def test_adapters_that_do_not_fit_are_refused():
    h = torch.float16
    for down, up in ((torch.zeros(2, 4, 8, dtype=h), torch.zeros(2, 5, 4, dtype=h)),              # on the CPU
                     (OnGpu(0, (2, 4), h), OnGpu(0, (2, 5, 4), h)), (OnGpu(0, (2, 4, 8), h), OnGpu(0, (3, 5, 4), h)),
                     (OnGpu(0, (2, 4, 8), h), OnGpu(0, (2, 5, 3), h)), (OnGpu(0, (2, 4, 8), h), OnGpu(0, (2, 5, 4), torch.bfloat16)),
                     (OnGpu(0, (2, 4, 8), torch.float32), OnGpu(0, (2, 5, 4), torch.float32)),
                     (OnGpu(0, (2, 4, 8), h), OnGpu(1, (2, 5, 4), h)), (OnGpu(0, (0, 4, 8), h), OnGpu(0, (0, 5, 4), h)),
                     (OnGpu(0, (1, 257, 8), h), OnGpu(0, (1, 5, 257), h)), (OnGpu(0, (1, 0, 8), h), OnGpu(0, (1, 5, 0), h))):
        with pytest.raises(ValueError):
            V.Adapters(down, up)
