"""Thin ctypes binding of libvocoder.so (argument marshalling only).

Every function has the name of the C entry point it calls (include/vocoder.h)
and returns the C status code (0 = VOC_OK, negative = error) unless noted.
Device buffers are passed as torch CUDA tensors (their data_ptr()), streams
as torch streams or raw hipStream_t integers.  All computation happens in
the HIP library; this module fails loudly if the library is not built.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

# VOC_LIBRARY names another build of the same library (e.g. an ablation build).
LIB_PATH = os.environ.get("VOC_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libvocoder.so")

VOC_ABI_VERSION = 4
VOC_MAX_BLOCKS = 8
VOC_MAX_RES = 4

VOC_OK = 0
VOC_INVALID_PARAMS = -1
VOC_BAD_WEIGHTS = -2
VOC_OOM = -3
VOC_DEVICE_ERROR = -4
VOC_NOT_LOADED = -5
VOC_CANCELLED = -6

VOC_F32, VOC_BF16, VOC_F16 = 0, 1, 2
VOC_ACT_NONE, VOC_ACT_GELU = 0, 1
VOC_SNAKE, VOC_SNAKE_BETA = 0, 1

KERNEL_KINDS = ["conv_in", "convt", "res_k7", "res_k1", "head", "import", "export", "res_fused",
                "in_proj", "enc_down", "enc_out", "af_snake", "snake", "col2im", "tanh"]


class voc_config(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_int),
        ("latent_channels", ctypes.c_int),
        ("n_blocks", ctypes.c_int),
        ("width", ctypes.c_int * (VOC_MAX_BLOCKS + 1)),
        ("stride", ctypes.c_int * VOC_MAX_BLOCKS),
        ("in_kernel", ctypes.c_int),
        ("res_kernel", ctypes.c_int),
        ("out_kernel", ctypes.c_int),
        ("n_res", ctypes.c_int),
        ("dilation", ctypes.c_int * VOC_MAX_RES),
        ("act", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("snake_log_params", ctypes.c_int),
        ("convt_crop", ctypes.c_int),
        ("tile_frames", ctypes.c_int),
        ("in_proj", ctypes.c_int),
        ("causal", ctypes.c_int),
        ("enc_width", ctypes.c_int * (VOC_MAX_BLOCKS + 1)),
        ("af_snake", ctypes.c_int),
        ("out_channels", ctypes.c_int),
        ("operand_terms", ctypes.c_int),
    ]


class voc_tensor(ctypes.Structure):
    _fields_ = [
        ("name", ctypes.c_char_p),
        ("data", ctypes.POINTER(ctypes.c_float)),
        ("ndim", ctypes.c_int),
        ("shape", ctypes.c_int64 * 4),
    ]


class voc_profile_stat(ctypes.Structure):
    _fields_ = [
        ("launches", ctypes.c_int64),
        ("ms", ctypes.c_double),
        ("flops", ctypes.c_double),
        ("bytes", ctypes.c_double),
    ]


class voc_kv_cache(ctypes.Structure):
    _fields_ = [
        ("page_tokens", ctypes.c_int),
        ("kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("n_pages", ctypes.c_int64),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
    ]


class voc_kv_batch(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("tokens", ctypes.c_int64),
        ("max_new", ctypes.c_int64),
        ("max_total", ctypes.c_int64),
        ("starts", ctypes.c_void_p),
        ("past", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p),
        ("table_stride", ctypes.c_int64),
    ]


_lib = None

# int (*voc_cancel_fn)(void *user)
CANCEL_FN = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p)

# Per-context host state the C calls do not return: the rows of the streams
# started by vocoder_stream_reset, and the installed cancel callback (kept
# referenced while the library holds its pointer).
_stream_rows: dict = {}
_cancel_keep: dict = {}


def lib():
    """The loaded libvocoder.so.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m dac_vocoder_decoding_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        CFG = ctypes.POINTER(voc_config)
        sig = {
            "voc_config_default": (None, [CFG]),
            "voc_config_validate": (I, [CFG]),
            "voc_config_hop": (I64, [CFG]),
            "voc_config_halo": (I, [CFG]),
            "voc_config_max_frames": (I64, [CFG]),
            "vocoder_set_cancel": (I, [P, CANCEL_FN, P, I64]),
            "vocoder_create": (I, [CFG, I, ctypes.POINTER(P)]),
            "vocoder_load_weights": (I, [P, ctypes.POINTER(voc_tensor), I]),
            "vocoder_output_length": (I64, [P, I64]),
            "vocoder_decode": (I, [P, P, I64, I64, P, P]),
            "vocoder_decode_noalloc": (I, [P, P, I64, I64, P, P]),
            "vocoder_decode_windows": (I, [P, P, I64, I64, I64, I64, I64, I64, P, P]),
            "vocoder_windows_output_length": (I64, [P, I64, I64, I64, I64, I64]),
            "vocoder_stream_reset": (I, [P, I64]),
            "vocoder_encode": (I, [P, P, I64, I64, P, P]),
            "vocoder_stream_decode": (I, [P, P, I64, P, P]),
            "vocoder_last_error": (ctypes.c_char_p, [P]),
            "vocoder_destroy": (None, [P]),
            "vocoder_profile_enable": (I, [P, I]),
            "vocoder_profile_select": (I, [P, ctypes.c_uint32]),
            "vocoder_profile_reset": (I, [P]),
            "vocoder_profile_read": (I, [P, I, ctypes.POINTER(voc_profile_stat)]),
            "voc_dbg_stage_count": (I, [P]),
            "voc_dbg_stage_shape": (I, [P, I, I64, ctypes.POINTER(I64), ctypes.POINTER(I64),
                                        ctypes.POINTER(I64)]),
            "voc_dbg_run_stage": (I, [P, I, P, I64, I64, P, P]),
            "voc_dbg_copy": (I, [P, P, I64, P]),
            "voc_dbg_peak": (I, [I, I64, ctypes.POINTER(ctypes.c_double), P]),
            "voc_ops_create": (I, [I, ctypes.POINTER(P)]),
            "voc_ops_last_error": (ctypes.c_char_p, [P]),
            "voc_ops_destroy": (None, [P]),
            "voc_dbg_last_kernel": (ctypes.c_char_p, [P, ctypes.POINTER(I)]),
            "vocoder_rms_norm": (I, [P, I, I64, I64, P, I64, P, I64, P, I64, P, F, P, I64, P, P]),
            "vocoder_quantize_rows": (I, [P, I, I64, I64, P, I64, P, I64, P, P]),
            "vocoder_matmul_int": (I, [P, I, I64, I64, I64, P, I64, P, P, I64, P, P, I, P, I64, P]),
            "vocoder_cache_append": (I, [P, P, P, I, P, I64, I64, P, I64, I64, P]),
            "vocoder_cache_attention": (I, [P, P, P, I, I, P, I64, I64, F, I, I64, P, I64, I64, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


class VocError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"status {status}: {msg}")
        self.status = status


def _key(ctx):
    return ctx.value if isinstance(ctx, ctypes.c_void_p) else int(ctx or 0)


def expect_dim(what: str, shape, dim: int, want: int) -> None:
    """Raise ValueError unless shape[dim] == want (checked before any call
    that would let the library read or write past a buffer)."""
    if len(shape) != 3:
        raise ValueError(f"{what}: expected a 3-d tensor, got shape {tuple(shape)}")
    if shape[dim] != want:
        raise ValueError(f"{what}: dimension {dim} is {shape[dim]}, the context needs {want}")


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


# ------------------------------------------------------------------ config
def config_from_dict(d: dict) -> voc_config:
    """voc_config for an architecture dict (keys as in inputs.CONFIGS)."""
    c = voc_config()
    lib().voc_config_default(ctypes.byref(c))
    c.latent_channels = d["latent_channels"]
    c.n_blocks = len(d["strides"])
    for i, w in enumerate(d["widths"]):
        c.width[i] = w
    for i, s in enumerate(d["strides"]):
        c.stride[i] = s
    c.in_kernel = c.res_kernel = c.out_kernel = d.get("kernel", 7)
    c.n_res = len(d["dilations"])
    for i, dl in enumerate(d["dilations"]):
        c.dilation[i] = dl
    c.act = VOC_SNAKE_BETA if d["act"] == "snakebeta" else VOC_SNAKE
    c.dtype = VOC_BF16 if d["dtype"] == "bf16" else VOC_F32
    c.snake_log_params = d.get("snake_log_params", 0)
    c.tile_frames = d.get("tile_frames", 0)
    c.in_proj = d.get("in_proj", 0)
    c.causal = int(d.get("causal", 0))
    for i, w in enumerate(d.get("enc_widths") or ()):
        c.enc_width[i] = w
    c.af_snake = int(d.get("af_snake", 0))
    c.out_channels = int(d.get("out_channels", 1))
    c.operand_terms = int(d.get("operand_terms", 0))
    return c


def voc_config_default() -> voc_config:
    c = voc_config()
    lib().voc_config_default(ctypes.byref(c))
    return c


def voc_config_validate(cfg: voc_config) -> int:
    return lib().voc_config_validate(ctypes.byref(cfg))


def voc_config_hop(cfg: voc_config) -> int:
    return lib().voc_config_hop(ctypes.byref(cfg))


def voc_config_halo(cfg: voc_config) -> int:
    return lib().voc_config_halo(ctypes.byref(cfg))


def voc_config_max_frames(cfg: voc_config) -> int:
    return lib().voc_config_max_frames(ctypes.byref(cfg))


# ----------------------------------------------------------------- context
def vocoder_create(cfg: voc_config, device: int = 0):
    """Returns (status, ctx)."""
    ctx = ctypes.c_void_p()
    st = lib().vocoder_create(ctypes.byref(cfg), device, ctypes.byref(ctx))
    return st, ctx


def vocoder_load_weights(ctx, tensors: dict) -> int:
    """tensors: name -> float32 numpy array (host)."""
    arrs = {k: np.ascontiguousarray(v, dtype=np.float32) for k, v in tensors.items()}
    items = (voc_tensor * len(arrs))()
    keep = []
    for i, (k, v) in enumerate(arrs.items()):
        name = k.encode()
        keep.append(name)
        items[i].name = name
        items[i].data = v.ctypes.data_as(ctypes.POINTER(ctypes.c_float))
        items[i].ndim = v.ndim
        for j, s in enumerate(v.shape):
            items[i].shape[j] = s
    st = lib().vocoder_load_weights(ctx, items, len(arrs))
    del keep
    return st


def vocoder_output_length(ctx, T: int) -> int:
    return lib().vocoder_output_length(ctx, T)


def vocoder_decode(ctx, latent, B: int, T: int, pcm, stream=None) -> int:
    return lib().vocoder_decode(ctx, _ptr(latent), B, T, _ptr(pcm), _stream(stream))


def vocoder_decode_noalloc(ctx, latent, B: int, T: int, pcm, stream=None) -> int:
    return lib().vocoder_decode_noalloc(ctx, _ptr(latent), B, T, _ptr(pcm), _stream(stream))


def vocoder_decode_windows(ctx, latents, n: int, sides: int, L: int, L_last: int,
                           crop_left: int, crop_right: int, pcm, stream=None) -> int:
    return lib().vocoder_decode_windows(ctx, _ptr(latents), n, sides, L, L_last, crop_left,
                                        crop_right, _ptr(pcm), _stream(stream))


def vocoder_windows_output_length(ctx, n: int, L: int, L_last: int, crop_left: int,
                                  crop_right: int) -> int:
    return lib().vocoder_windows_output_length(ctx, n, L, L_last, crop_left, crop_right)


def vocoder_encode(ctx, audio, B: int, T: int, latent, stream=None) -> int:
    return lib().vocoder_encode(ctx, _ptr(audio), B, T, _ptr(latent), _stream(stream))


def encode(ctx, audio, latent_channels: int, stream=None):
    """latent [B, latent_channels, T] (new CUDA tensor) for CUDA fp32 audio
    [B, 1, T * hop]."""
    import torch
    assert audio.is_cuda and audio.dtype == torch.float32 and audio.is_contiguous()
    expect_dim("audio", audio.shape, 1, 1)
    b, _, n = audio.shape
    hop = vocoder_output_length(ctx, 1)
    assert n % hop == 0
    other, z = _output(stream, audio, b, latent_channels, n // hop)
    st = vocoder_encode(ctx, audio, b, n // hop, z, stream)
    _keep(other, audio, z)
    check(st, ctx)
    return z


def vocoder_stream_reset(ctx, rows: int) -> int:
    st = lib().vocoder_stream_reset(ctx, rows)
    _stream_rows[_key(ctx)] = rows if st == VOC_OK else 0
    return st


def vocoder_set_cancel(ctx, fn, group: int = 1) -> int:
    """Install fn() -> bool as the cancel hook (None removes it); see
    vocoder_set_cancel in vocoder.h for when it is polled."""
    if fn is None:
        cb = CANCEL_FN()
    else:
        cb = CANCEL_FN(lambda _user: 1 if fn() else 0)
    st = lib().vocoder_set_cancel(ctx, cb, None, group)
    if st == VOC_OK:
        _cancel_keep[_key(ctx)] = cb
    return st


def vocoder_stream_decode(ctx, latent, t: int, pcm, stream=None) -> int:
    return lib().vocoder_stream_decode(ctx, _ptr(latent), t, _ptr(pcm), _stream(stream))


def vocoder_last_error(ctx) -> str:
    r = lib().vocoder_last_error(ctx)
    return r.decode() if r else ""


def vocoder_destroy(ctx) -> None:
    lib().vocoder_destroy(ctx)
    _stream_rows.pop(_key(ctx), None)
    _cancel_keep.pop(_key(ctx), None)


def vocoder_profile_enable(ctx, enable: bool) -> int:
    return lib().vocoder_profile_enable(ctx, int(bool(enable)))


def vocoder_profile_select(ctx, kinds: int) -> int:
    """Time only the kernel kinds whose bit (1 << kind) is set; 0 = all."""
    return lib().vocoder_profile_select(ctx, int(kinds))


def vocoder_profile_reset(ctx) -> int:
    return lib().vocoder_profile_reset(ctx)


def vocoder_profile_read(ctx, kind: int):
    """Returns (status, dict(launches, ms, flops, bytes))."""
    s = voc_profile_stat()
    st = lib().vocoder_profile_read(ctx, kind, ctypes.byref(s))
    return st, dict(launches=s.launches, ms=s.ms, flops=s.flops, bytes=s.bytes)


def voc_dbg_stage_count(ctx) -> int:
    return lib().voc_dbg_stage_count(ctx)


def voc_dbg_stage_shape(ctx, stage: int, T_in: int):
    """Returns (status, c_in, c_out, t_out)."""
    a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    st = lib().voc_dbg_stage_shape(ctx, stage, T_in, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c))
    return st, a.value, b.value, c.value


def voc_dbg_run_stage(ctx, stage: int, x, B: int, T_in: int, out, stream=None) -> int:
    return lib().voc_dbg_run_stage(ctx, stage, _ptr(x), B, T_in, _ptr(out), _stream(stream))


def voc_dbg_copy(dst, src, nbytes: int, stream=None) -> int:
    return lib().voc_dbg_copy(_ptr(dst), _ptr(src), nbytes, _stream(stream))


def voc_dbg_peak(what: int, n: int, stream=None):
    """(status, value): measured HBM copy GB/s (what=0, n bytes) or MFMA
    TFLOP/s (what=1 fp32 / 2 bf16 with 16x16 MFMAs, 3 / 4 with 32x32 ones;
    n loop iterations)."""
    v = ctypes.c_double(0.0)
    st = lib().voc_dbg_peak(what, n, ctypes.byref(v), _stream(stream))
    return st, v.value


def check(st: int, ctx=None) -> None:
    """Raise VocError for a non-zero status, with the context's last error."""
    if st != VOC_OK:
        raise VocError(st, vocoder_last_error(ctx))


# ---------------------------------------------------- marshalling helpers
# With an explicit `stream` that is not the current one, the new tensor may be
# used and freed on the current one, and the input is kept until `stream` has
# passed the call; the order of the work on the two is the caller's.
def _output(stream, t, *shape):
    """(the stream of the call if it is not the current one, a new CUDA fp32
    tensor for the call's output beside its input t)."""
    if _empty is None:
        _use_torch()
    other = None if stream is None else _stream_of(stream, t)[1]
    return other, _new(other, shape, _float32, t.device)


def open_context(cfg_dict: dict, tensors: dict, device: int = 0, **overrides):
    """vocoder_create + vocoder_load_weights; raises VocError on failure."""
    cfg = config_from_dict({**cfg_dict, **overrides})
    st, ctx = vocoder_create(cfg, device)
    check(st)
    st = vocoder_load_weights(ctx, tensors)
    if st != VOC_OK:
        msg = vocoder_last_error(ctx)
        vocoder_destroy(ctx)
        raise VocError(st, msg)
    return ctx


def out_channels(ctx) -> int:
    """Output channels of the context's head (the last debug stage's c_out)."""
    st, _, c_out, _ = voc_dbg_stage_shape(ctx, voc_dbg_stage_count(ctx) - 1, 1)
    check(st, ctx)
    return c_out


def latent_channels(ctx) -> int:
    """Latent channels the context decodes (stage 0's c_in)."""
    st, c_in, _, _ = voc_dbg_stage_shape(ctx, 0, 1)
    check(st, ctx)
    return c_in


def decode(ctx, latent, stream=None):
    """pcm [B, out_channels, T*hop] (new CUDA tensor) for a CUDA fp32 latent [B, C, T]."""
    import torch
    assert latent.is_cuda and latent.dtype == torch.float32 and latent.is_contiguous()
    expect_dim("latent", latent.shape, 1, latent_channels(ctx))
    b, _, t = latent.shape
    other, pcm = _output(stream, latent, b, out_channels(ctx), vocoder_output_length(ctx, t))
    st = vocoder_decode(ctx, latent, b, t, pcm, stream)
    _keep(other, latent, pcm)
    check(st, ctx)
    return pcm


def decode_windows(ctx, windows, sides: int, last_frames: int, crop_left: int, crop_right: int,
                   stream=None):
    """Planar pcm [sides * out_channels, N] (new CUDA tensor) for CUDA fp32
    windows [n, sides * C, L] (vocoder_decode_windows)."""
    import torch
    assert windows.is_cuda and windows.dtype == torch.float32 and windows.is_contiguous()
    expect_dim("windows", windows.shape, 1, sides * latent_channels(ctx))
    n, _, L = windows.shape
    N = vocoder_windows_output_length(ctx, n, L, last_frames, crop_left, crop_right)
    if N < 0:
        raise VocError(VOC_INVALID_PARAMS, "bad window lengths or crops")
    other, pcm = _output(stream, windows, sides * out_channels(ctx), N)
    st = vocoder_decode_windows(ctx, windows, n, sides, L, last_frames, crop_left, crop_right,
                                pcm, stream)
    _keep(other, windows, pcm)
    check(st, ctx)
    return pcm


def stream_decode(ctx, latent, stream=None):
    """pcm [rows, out_channels, t*hop] (new CUDA tensor) for the next chunk
    [rows, C, t] of the streams started by vocoder_stream_reset."""
    import torch
    assert latent.is_cuda and latent.dtype == torch.float32 and latent.is_contiguous()
    expect_dim("latent", latent.shape, 0, _stream_rows.get(_key(ctx), 0))
    expect_dim("latent", latent.shape, 1, latent_channels(ctx))
    rows, _, t = latent.shape
    other, pcm = _output(stream, latent, rows, out_channels(ctx), vocoder_output_length(ctx, t))
    st = vocoder_stream_decode(ctx, latent, t, pcm, stream)
    _keep(other, latent, pcm)
    check(st, ctx)
    return pcm


def run_stage(ctx, stage: int, x, stream=None):
    """Output of debug stage `stage` for a CUDA fp32 input [B, C_in, T]."""
    import torch
    assert x.is_cuda and x.dtype == torch.float32 and x.is_contiguous()
    b, _, t = x.shape
    st, c_in, c_out, t_out = voc_dbg_stage_shape(ctx, stage, t)
    check(st, ctx)
    expect_dim("stage input", x.shape, 1, c_in)
    other, out = _output(stream, x, b, c_out, t_out)
    st = voc_dbg_run_stage(ctx, stage, x, b, t, out, stream)
    _keep(other, x, out)
    check(st, ctx)
    return out


# ------------------------------------------ 8-bit transformer operators
# The calls of vocoder.h take raw pointers and strides; the helpers below take
# CUDA tensors, read the strides off them, check the shapes that the library
# cannot see, and allocate what is not given.  All of them run on `stream`
# (default: torch's current stream).  With another stream than the current
# one, tensors that are read or written stay allocated until that stream has
# passed the call, and new ones are allocated on it and may be used and freed
# on the current one; the order of the work on the two is the caller's.

class voc_ops(ctypes.c_void_p):
    """A handle of the operators and the device that it belongs to."""
    device = 0


def voc_ops_create(device: int = 0):
    """Returns (status, ops)."""
    ops = voc_ops()
    st = lib().voc_ops_create(device, ctypes.byref(ops))
    ops.device = device
    if st == VOC_OK:
        _use_torch()
    return st, ops


def voc_ops_last_error(ops) -> str:
    r = lib().voc_ops_last_error(ops)
    return r.decode() if r else ""


def voc_ops_destroy(ops) -> None:
    lib().voc_ops_destroy(ops)


def voc_dbg_last_kernel(ops):
    """(name, shape) of the kernel that the last call on ops launched."""
    shape = (ctypes.c_int * 2)()
    return lib().voc_dbg_last_kernel(ops, shape).decode(), tuple(shape)


def open_ops(device: int = 0):
    """A handle of the operators (voc_ops_create); raises VocError on failure."""
    st, ops = voc_ops_create(device)
    if st != VOC_OK:
        raise VocError(st, voc_ops_last_error(None))
    return ops


# voc_dtype of torch dtypes, and the function that reads a device's current
# stream, filled in with the first handle (torch is imported only then).  A
# call takes about 5 us in the library; the checks here are written to cost
# little beside that.
_dtypes: dict = {}
_int8 = _float32 = _empty = _raw_stream = None


def _use_torch() -> None:
    global _int8, _float32, _empty, _raw_stream
    import torch
    _int8, _float32, _empty = torch.int8, torch.float32, torch.empty
    # The public torch.cuda.current_stream() builds a Stream object (3 us).
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
    _dtypes.update({torch.float32: VOC_F32, torch.bfloat16: VOC_BF16, torch.float16: VOC_F16})


def _stream_of(stream, t):
    """The address of `stream`, and the stream itself if it is not the current
    one of t's device."""
    device = t.get_device()
    here = _raw_stream(device)
    raw = stream if isinstance(stream, int) else stream.cuda_stream
    if raw == here:
        return raw, None
    if isinstance(stream, int):
        import torch
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    return raw, stream


def _new(other, shape, dtype, device):
    """An empty tensor for a call on `other` (None: on the current stream).

    One from the current stream's pool could be memory that work pending there
    still uses, and could be handed out again while `other` still writes it."""
    if other is None:
        return _empty(shape, dtype=dtype, device=device)
    import torch
    with torch.cuda.stream(other):
        t = _empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _keep(other, *tensors) -> None:
    """Keeps the memory of tensors (None among them) until `other` (None: the
    current stream, whose memory it is) has passed what was launched on it."""
    if other is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(other)


def _dtype(t) -> int:
    """voc_dtype of a torch dtype."""
    d = _dtypes.get(t)
    if d is None:
        raise ValueError(f"dtype {t}: float32, bfloat16 or float16 is needed")
    return d


def _check_ops(st: int, ops) -> None:
    if st != VOC_OK:
        raise VocError(st, voc_ops_last_error(ops))


def _elsewhere(what: str, t, device: int):
    where = f"CUDA device {t.get_device()}" if t.is_cuda else "the CPU"
    return ValueError(f"{what}: a tensor on the handle's CUDA device {device} is needed, this one is on {where}")


def _rows(what: str, t, shape, dtype, device: int) -> int:
    """Checks a matrix on `device` whose rows are contiguous; returns its row
    stride."""
    if t.shape != shape or len(shape) != 2 or t.dtype is not dtype:
        raise ValueError(f"{what}: a CUDA matrix {tuple(shape)} {dtype} is needed, got {tuple(t.shape)} {t.dtype}")
    if t.get_device() != device:
        raise _elsewhere(what, t, device)
    step, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{what}: rows have to be contiguous")
    return step if shape[0] > 1 else max(step, shape[1])


def _vector(what: str, t, n: int, device: int) -> int:
    """Checks n contiguous float32 values on `device`; returns their address."""
    if t.dtype is not _float32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous CUDA float32 values are needed")
    if t.get_device() != device:
        raise _elsewhere(what, t, device)
    return t.data_ptr()


def rms_norm(ops, x, weight, eps: float = 1e-6, residual=None, h=None, q=None, scale=None, stream=None):
    """(q int8 [rows, C], scale fp32 [rows], h) of the rows x [rows, C]
    (vocoder_rms_norm).  h = x + residual is stored into `h` (which may be x
    or residual itself), into a new tensor if that is None and there is a
    residual, and is x itself without one."""
    shape, dtype, device, at = x.shape, x.dtype, x.device, ops.device
    ldx = _rows("x", x, shape, dtype, at)
    raw, other = (_raw_stream(at), None) if stream is None else _stream_of(stream, x)
    rows, C = shape
    r = hp = None
    ldr = ldh = 0
    if residual is not None:
        ldr, r = _rows("residual", residual, shape, dtype, at), residual.data_ptr()
        if h is None:
            h, ldh = _new(other, shape, dtype, device), C
            hp = h.data_ptr()
    if h is not None and hp is None:
        ldh, hp = _rows("h", h, shape, dtype, at), h.data_ptr()
    if q is None:
        q, ldq = _new(other, shape, _int8, device), C
    else:
        ldq = _rows("q", q, shape, _int8, at)
    if scale is None:
        scale = _new(other, rows, _float32, device)
    st = lib().vocoder_rms_norm(ops, _dtype(dtype), rows, C, x.data_ptr(), ldx, r, ldr, hp, ldh,
                                _vector("weight", weight, C, at), eps, q.data_ptr(), ldq,
                                _vector("scale", scale, rows, at), raw)
    if other is not None:
        _keep(other, x, residual, h, weight, q, scale)
    if st:
        _check_ops(st, ops)
    return q, scale, x if h is None else h


def quantize_rows(ops, x, q=None, scale=None, stream=None):
    """(q int8 [rows, C], scale fp32 [rows]) of the rows x [rows, C]
    (vocoder_quantize_rows)."""
    shape, dtype, device, at = x.shape, x.dtype, x.device, ops.device
    ldx = _rows("x", x, shape, dtype, at)
    raw, other = (_raw_stream(at), None) if stream is None else _stream_of(stream, x)
    rows, C = shape
    if q is None:
        q, ldq = _new(other, shape, _int8, device), C
    else:
        ldq = _rows("q", q, shape, _int8, at)
    if scale is None:
        scale = _new(other, rows, _float32, device)
    st = lib().vocoder_quantize_rows(ops, _dtype(dtype), rows, C, x.data_ptr(), ldx, q.data_ptr(), ldq,
                                     _vector("scale", scale, rows, at), raw)
    if other is not None:
        _keep(other, x, q, scale)
    if st:
        _check_ops(st, ops)
    return q, scale


def matmul_int(ops, a, a_scale, b, b_scale, bias=None, gelu: bool = False, dtype=None, out=None, stream=None):
    """act((a b^T) * a_scale[:, None] * b_scale + bias) [M, N] for int8 a
    [M, K] and b [N, K] (vocoder_matmul_int), in `dtype` (default float16) or
    the dtype of `out`."""
    at = ops.device
    lda = _rows("a", a, a.shape, _int8, at)
    M, K = a.shape
    N = b.shape[0]
    ldb = _rows("b", b, (N, K), _int8, at)
    raw, other = (_raw_stream(at), None) if stream is None else _stream_of(stream, a)
    if out is None:
        if dtype is None:
            import torch
            dtype = torch.float16
        out, ldy = _new(other, (M, N), dtype, a.device), N
    else:
        if dtype is None:
            dtype = out.dtype
        ldy = _rows("out", out, (M, N), dtype, at)
    st = lib().vocoder_matmul_int(
        ops, _dtype(dtype), M, N, K, a.data_ptr(), lda, _vector("a_scale", a_scale, M, at), b.data_ptr(), ldb,
        _vector("b_scale", b_scale, N, at),
        None if bias is None else _vector("bias", bias, N, at),
        VOC_ACT_GELU if gelu else VOC_ACT_NONE, out.data_ptr(), ldy, raw)
    if other is not None:
        _keep(other, a, a_scale, b, b_scale, bias, out)
    if st:
        _check_ops(st, ops)
    return out


class KVCache:
    """A paged 8-bit cache (voc_kv_cache): k int8 [pages, kv_heads,
    page_tokens, head_dim], v int8 [pages, kv_heads, head_dim, page_tokens],
    k_scale and v_scale fp32 [pages, kv_heads]."""

    def __init__(self, pages: int, page_tokens: int, kv_heads: int, head_dim: int, device="cuda"):
        import torch
        self._set(torch.zeros(pages, kv_heads, page_tokens, head_dim, dtype=torch.int8, device=device),
                  torch.zeros(pages, kv_heads, head_dim, page_tokens, dtype=torch.int8, device=device),
                  torch.zeros(pages, kv_heads, device=device), torch.zeros(pages, kv_heads, device=device))

    @classmethod
    def from_tensors(cls, k, v, k_scale, v_scale):
        """A cache over tensors that the caller allocated."""
        c = cls.__new__(cls)
        c._set(k, v, k_scale, v_scale)
        return c

    def _set(self, k, v, k_scale, v_scale):
        import torch
        n, h, p, d = k.shape
        for t, shape, dt in ((k, (n, h, p, d), torch.int8), (v, (n, h, d, p), torch.int8),
                             (k_scale, (n, h), torch.float32), (v_scale, (n, h), torch.float32)):
            if tuple(t.shape) != shape or t.dtype != dt or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"cache: a contiguous CUDA {dt} tensor of shape {shape} is needed")
            if t.device != k.device:
                raise ValueError(f"cache: all of its tensors have to be on {k.device}, one is on {t.device}")
        self.device = k.get_device()
        self.k, self.v, self.k_scale, self.v_scale = self.tensors = k, v, k_scale, v_scale
        self.kv_heads, self.page_tokens, self.head_dim = h, p, d
        self.c = voc_kv_cache(p, h, d, n, k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())
        self.ref = ctypes.byref(self.c)


class KVBatch:
    """The sequences of one step (voc_kv_batch): page_table int32 [B, pages],
    past int32 [B], starts int32 [B + 1], and the host's bounds max_new (new
    tokens of a sequence) and max_total (past + new).  Calls leave it as it
    is, so that threads with handles of their own may share one."""

    def __init__(self, page_table, past, starts, max_new: int, max_total: int):
        import torch
        B = past.numel()
        for what, t, shape in (("page_table", page_table, (B, page_table.shape[-1])), ("past", past, (B,)),
                               ("starts", starts, (B + 1,))):
            if t.dtype != torch.int32 or not t.is_cuda or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{what}: a contiguous CUDA int32 tensor of shape {shape} is needed")
            if t.device != past.device:
                raise ValueError(f"{what}: the batch's tensors have to be on {past.device}, this one is on {t.device}")
        self.device = past.get_device()
        self.page_table, self.past, self.starts = self.tensors = page_table, past, starts
        self.c = voc_kv_batch(B, 0, max_new, max_total, starts.data_ptr(), past.data_ptr(), page_table.data_ptr(),
                              page_table.shape[1])
        self.ref = ctypes.byref(self.c)


def _heads(what: str, t, shape, dtype, device: int):
    """Checks a tensor [tokens, heads, dim] on `device` with contiguous dim;
    returns its token and head strides."""
    if t.shape != shape or len(shape) != 3 or t.dtype is not dtype:
        raise ValueError(f"{what}: a CUDA tensor {tuple(shape)} {dtype} is needed, got {tuple(t.shape)} {t.dtype}")
    if t.get_device() != device:
        raise _elsewhere(what, t, device)
    step, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{what}: the last dimension has to be contiguous")
    return step, head


def _with_tokens(batch: KVBatch, tokens: int) -> voc_kv_batch:
    """The batch for a call with `tokens` packed rows, a struct of that call's
    own: in a shared one another thread could change the number between this
    call's checks and its launch."""
    c = voc_kv_batch.from_buffer_copy(batch.c)
    c.tokens = tokens
    return c


def _apart(ops, cache: KVCache, batch: KVBatch):
    return ValueError(f"the cache is on CUDA device {cache.device}, the batch on {batch.device}, the handle on {ops.device}")


def cache_append(ops, cache: KVCache, batch: KVBatch, k, v, stream=None) -> None:
    """Append k and v [tokens, kv_heads, head_dim] to the cache
    (vocoder_cache_append)."""
    dtype, tokens, device = k.dtype, k.shape[0], ops.device
    shape = (tokens, cache.kv_heads, cache.head_dim)
    kt, kh = _heads("k", k, shape, dtype, device)
    vt, vh = _heads("v", v, shape, dtype, device)
    if not device == cache.device == batch.device:
        raise _apart(ops, cache, batch)
    c = _with_tokens(batch, tokens)
    raw, other = (_raw_stream(device), None) if stream is None else _stream_of(stream, k)
    st = lib().vocoder_cache_append(ops, cache.ref, ctypes.byref(c), _dtype(dtype), k.data_ptr(), kt, kh, v.data_ptr(), vt, vh,
                                    raw)
    if other is not None:
        _keep(other, k, v, *cache.tensors, *batch.tensors)
    if st:
        _check_ops(st, ops)


def cache_attention(ops, cache: KVCache, batch: KVBatch, q, scale: float | None = None, causal: bool = True,
                    window: int = 0, out=None, stream=None):
    """Attention of q [tokens, heads, head_dim] over the cache
    (vocoder_cache_attention); scale defaults to head_dim ** -0.5."""
    shape, dtype, dim, device = q.shape, q.dtype, cache.head_dim, ops.device
    qt, qh = _heads("q", q, shape, dtype, device)
    if shape[2] != dim:
        raise ValueError(f"q: head_dim {dim} is needed, got {shape[2]}")
    raw, other = (_raw_stream(device), None) if stream is None else _stream_of(stream, q)
    if out is None:
        out = _new(other, shape, dtype, q.device)
    ot, oh = _heads("out", out, shape, dtype, device)
    if not device == cache.device == batch.device:
        raise _apart(ops, cache, batch)
    c = _with_tokens(batch, shape[0])
    st = lib().vocoder_cache_attention(ops, cache.ref, ctypes.byref(c), _dtype(dtype), shape[1], q.data_ptr(), qt, qh,
                                       dim ** -0.5 if scale is None else scale, int(causal), window, out.data_ptr(), ot, oh,
                                       raw)
    if other is not None:
        _keep(other, q, out, *cache.tensors, *batch.tensors)
    if st:
        _check_ops(st, ops)
    return out
