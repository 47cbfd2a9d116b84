"""The 8-bit transformer operators' entry points without a device: a NULL
handle is refused before anything else, and the handle functions are
NULL-safe."""
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
